// Definitions shared by the host side and the kernels of the accumulated attention weight.
#pragma once

#include "qda_paged.h"

struct QdaWeightsParams {
  const uint16_t* q;          // row t, head h at t * q_tstride + h * q_hstride
  const uint32_t* kp;         // [num_pages, Hkv, page, W]
  const uint16_t* ks;         // [num_pages, Hkv, page, NG]
  const uint16_t* kb;
  const float* lse;           // [total_q, H]
  float* mass;                // [num_pages, Hkv, page]
  int* token;                 // [num_pages, Hkv, page]
  const int* q_start;         // [B + 1]
  const int* kv_len;          // [B]
  const int* table;           // [B, max_pages]
  const int* shift;           // [B], or nullptr
  unsigned int* err;
  long long q_tstride, q_hstride;
  int total_q, window, B, H, Hkv, nrep, num_pages, page_shift, max_pages, ctas, f16;
  float qscale;               // log2(e) / sqrt(D)
  float decay;
};

// Translation units per code width. With ctas_per_sm the instance's resident CTAs per SM are stored there and nothing is
// launched; else p.ctas CTAs are. rows: the bound on a KV head's query rows that choose the instance.
cudaError_t qda_paged_weights_b4(const QdaWeightsParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
cudaError_t qda_paged_weights_b8(const QdaWeightsParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
