// Definitions shared by the host side and the kernels of the paged cache.
#pragma once

#include "qda_internal.h"

#define QDA_ERR_BIT_PAGED 8u   // device status: a page, slot or length outside its pool or table

// What a CTA of the attention kernels leaves for the merge: the tile that starts in its piece of the work and goes on
// behind it, and which of its two slots (a tile that started before its piece, and one that starts in it) hold a part.
struct QdaPagedSplitTile {
  int go, last;                     // there is such a tile; the last CTA that shares it
  int row0, rows, token0, unit;     // its query rows, the sequence's first token, the unit
  int first_filled, last_filled;
};

// Launch parameters of the paged attention kernels (passed by value as a __grid_constant__).
struct QdaPagedParams {
  const uint16_t* q;          // row t, head h at t * q_tstride + h * q_hstride
  const uint32_t* kp;         // [num_pages, Hkv, page, W]
  const uint16_t* ks;         // [num_pages, Hkv, page, NG]
  const uint16_t* kb;
  const uint32_t* vp;
  const uint16_t* vs;
  const uint16_t* vb;
  uint16_t* out;              // [total_q, H, D]
  const int* q_start;         // [B + 1]
  const int* kv_len;          // [B]
  const int* table;           // [B, max_pages]
  unsigned int* err;          // device error word
  long long q_tstride, q_hstride;
  int total_q, B, H, Hkv, nrep, num_pages, page_shift, max_pages, causal, D, GS, NG, W, f16;
  float qscale;               // log2(e) / sqrt(D)
  // how the call is shared among CTAs (qda_paged_sched.cuh)
  int ctas, min_keys;         // CTAs launched; fewest keys of a CTA's piece
  int units, parts;           // units of a sequence: Hkv * parts, unit u holds part u % parts of KV head u / parts's values
  QdaPagedSplitTile* split;   // [ctas]
  float* part_o;              // [2 * ctas, MT, D / parts] unnormalised partial outputs of split tiles
  float2* part_ml;            // [2 * ctas, MT] (reference in log2 units, sum of weights)
#ifdef QDA_BOUNDS_CHECK
  int stall_block;            // testing aid: the chunk kernel's first CTA gets no pages for this block of its own (-1: for all)
#endif
};

// Row of the pool arrays that holds row `r` of page `pg` of KV head `kvh`.
__host__ __device__ inline long long qda_pool_row(int pg, int kvh, int r, int Hkv, int page_shift) {
  return ((((long long)pg * Hkv) + kvh) << page_shift) + r;
}

// The split kernel (qda_paged_split.cuh), translation units per (bits, fp16): its instance for (D, GS, rows per tile).
// With ctas_per_sm the instance's resident CTAs per SM are stored there and nothing is launched; else p.ctas CTAs are.
cudaError_t qda_paged_split_b4_f0(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
cudaError_t qda_paged_split_b4_f1(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
cudaError_t qda_paged_split_b8_f0(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
cudaError_t qda_paged_split_b8_f1(const QdaPagedParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);

// The chunk kernel (qda_paged_chunk.cuh): 128 * tiles query rows per tile (tiles 1 or 2; 1 for D > 128), one CTA per SM.
// prepare sets the instance's shared memory limit on the current device and launches nothing.
cudaError_t qda_paged_chunk_b4(const QdaPagedParams* p, int D, int tiles, bool prepare, cudaStream_t s);
cudaError_t qda_paged_chunk_b8(const QdaPagedParams* p, int D, int tiles, bool prepare, cudaStream_t s);

// Merge of the split tiles' partial results, behind a kernel of `rows` rows per tile.
cudaError_t qda_launch_paged_merge(const QdaPagedParams& p, int rows, cudaStream_t s);
