// Definitions shared by the host side and the kernels of the paged cache.
#pragma once

#include "qda_internal.h"

#define QDA_ERR_BIT_PAGED 8u   // device status: a page, slot or length outside its pool or table

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
};

// Row of the pool arrays that holds row `r` of page `pg` of KV head `kvh`.
__host__ __device__ inline long long qda_pool_row(int pg, int kvh, int r, int Hkv, int page_shift) {
  return ((((long long)pg * Hkv) + kvh) << page_shift) + r;
}

cudaError_t qda_launch_paged_simple(const QdaPagedParams& p, int bits, cudaStream_t s);
