// Paged split kernel, 4-bit codes, fp16 caches, with the rows' sums.
#include "qda_paged_split.cuh"

cudaError_t qda_paged_split_b4_f1_lse(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s) {
  return qda::ps_pick<4, true, true>(p, D, GS, rows, ctas_per_sm, s);
}
