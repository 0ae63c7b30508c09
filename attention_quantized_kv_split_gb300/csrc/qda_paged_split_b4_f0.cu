// Paged split kernel, 4-bit codes, bf16 caches.
#include "qda_paged_split.cuh"

cudaError_t qda_paged_split_b4_f0(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s) {
  return qda::ps_pick<4, false, false>(p, D, GS, rows, ctas_per_sm, s);
}
