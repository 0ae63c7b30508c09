// Accumulated attention weight, 4-bit codes, fp16 scales.
#include "qda_paged_weights.cuh"

cudaError_t qda_paged_weights_b4_f1(const QdaWeightsParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s) {
  return qda::pw_pick<4, true>(p, D, GS, rows, ctas_per_sm, s);
}
