// Paged split kernel, 8-bit codes, fp16 caches.
#include "qda_paged_split.cuh"

cudaError_t qda_paged_split_b8_f1(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s) {
  return qda::ps_pick<8, true, false>(p, D, GS, rows, ctas_per_sm, s);
}
