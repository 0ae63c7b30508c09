// Paged chunk kernel, 4-bit codes.
#include "qda_paged_chunk.cuh"

cudaError_t qda_paged_chunk_b4(const QdaPagedParams* p, int D, int tiles, bool prepare, cudaStream_t s) {
  return qda::pc_pick<4, false>(p, D, tiles, prepare, s);
}
