// Paged split kernel, 8-bit codes, bf16 caches, with the rows' sums.
#include "qda_paged_split.cuh"

cudaError_t qda_paged_split_b8_f0_lse(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s) {
  return qda::ps_pick<8, false, true>(p, D, GS, rows, ctas_per_sm, s);
}
