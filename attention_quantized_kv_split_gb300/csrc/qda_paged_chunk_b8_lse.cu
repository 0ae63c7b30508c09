// Paged chunk kernel, 8-bit codes, with the rows' sums.
#include "qda_paged_chunk.cuh"

cudaError_t qda_paged_chunk_b8_lse(const QdaPagedParams* p, int D, int tiles, bool prepare, cudaStream_t s) {
  return qda::pc_pick<8, true>(p, D, tiles, prepare, s);
}
