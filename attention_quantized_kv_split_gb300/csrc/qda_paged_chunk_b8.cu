// Paged chunk kernel, 8-bit codes.
#include "qda_paged_chunk.cuh"

cudaError_t qda_paged_chunk_b8(const QdaPagedParams* p, int D, int tiles, bool prepare, cudaStream_t s) {
  return qda::pc_pick<8>(p, D, tiles, prepare, s);
}
