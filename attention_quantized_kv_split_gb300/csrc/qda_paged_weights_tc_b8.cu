// Accumulated attention weight for many query rows, 8-bit codes.
#include "qda_paged_weights_tc.cuh"

cudaError_t qda_paged_weights_tc_b8(const QdaWeightsParams* p, int D, bool prepare, cudaStream_t s) {
  return qda::pv_pick<8>(p, D, prepare, s);
}
