// Definitions shared by the host side and the kernels of the accumulated attention weight.
#pragma once

#include "qda_paged.h"
#include "qda_ptx.cuh"

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
  // the kernel for many rows
  int D, NG, gs_shift;        // gs_shift: log2 of the group size
  char* chunks;               // [chunks of all sequences, Hkv] query rows as operands (qda_paged_weights_tc.cuh)
  int max_chunks;             // chunks that there is room for
  int stall;                  // testing aid of the checked build: the first CTA does not get this operand slice (-1: gets all)
};

#ifdef __CUDACC__
namespace qda {

// A sequence as these kernels see it.
struct PwSeq {
  int first, len;      // its first token's row in q, its new tokens
  int n, base;         // keys; keys before the first new token (negative where the lengths lie)
  int count;           // new tokens that count: the last ones
};

__device__ __forceinline__ PwSeq pw_seq(const QdaWeightsParams& p, int start, int end, int n) {
  PwSeq s;
  const int q0 = min(max(start, 0), p.total_q), q1 = min(max(end, q0), p.total_q);
  s.first = q0;
  s.len = q1 - q0;
  // (sums with a block's keys stay in range)
  s.n = (int)min((long long)max(n, 0), min((long long)min(p.max_pages, p.num_pages) << p.page_shift, 0x7ffffe00LL));
  s.base = n - s.len;
  s.count = p.window > 0 ? min(p.window, s.len) : s.len;
  return s;
}
__device__ __forceinline__ PwSeq pw_seq(const QdaWeightsParams& p, int b) {
  return pw_seq(p, p.q_start[b], p.q_start[b + 1], p.kv_len[b]);
}

// Where 16-byte chunk ch of row r of a tile's codes lies: chunks of a row are permuted by the row's bits in reverse, so that
// the eight rows that a warp reads at once fall into different banks for loads of 4, 8 and 16 bytes.
template <int RB>
__device__ __forceinline__ int pw_chunk(int r, int ch) {
  constexpr int CPR = RB / 16, N = CPR < 8 ? CPR : 8;
  const int x = r / (8 / N);
  const int f = N == 8 ? ((x & 1) << 2) | (x & 2) | ((x >> 2) & 1) : N == 4 ? ((x & 1) << 1) | ((x >> 1) & 1) : x & 1;
  return r * RB + ((ch ^ f) << 4);
}

__device__ __forceinline__ void pw_copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void pw_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void pw_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Whether a sequence's starts or length are not what they have to be.
__device__ __forceinline__ bool pw_bad(const QdaWeightsParams& p, int start, int end, int n, const PwSeq& s) {
  return start < 0 || end < start || end > p.total_q || (end > start && (n < 0 || n > s.n));
}

// Blocks of KEYS keys (none without new tokens).
template <int KEYS>
__device__ __forceinline__ int pw_blocks(const PwSeq& s) {
  return s.len > 0 ? (int)(((long long)s.n + KEYS - 1) / KEYS) : 0;
}

// Work of the first i blocks of KEYS keys under one KV head, in query rows: a block whose first key every counted token sees
// takes `whole`, one behind the causal edge `edge` and the rows of the tokens that see its first key (n - x KEYS of them).
template <int KEYS>
__device__ __forceinline__ int pw_flat(const PwSeq& s) {   // blocks of the first kind
  return s.n >= s.count ? (s.n - s.count) / KEYS + 1 : 0;
}
template <int KEYS>
__device__ __forceinline__ long long pw_prefix(const QdaWeightsParams& p, const PwSeq& s, int i, long long whole, int edge) {
  const long long flat = min(pw_flat<KEYS>(s), i), rest = i - flat;
  return flat * whole + rest * edge +
         p.nrep * (rest * s.n - KEYS * (((long long)i * (i - 1) - flat * (flat - 1)) / 2));
}

// First of `blocks` blocks that starts at or behind x, where prefix(i) is the place of block i.
template <typename F>
__device__ __forceinline__ int pw_block_at(int blocks, long long x, F&& prefix) {
  int lo = 0, hi = blocks;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix(mid) >= x) hi = mid; else lo = mid + 1;
  }
  return lo;
}

}  // namespace qda
#endif

// Translation units per code width and input type. With ctas_per_sm the instance's resident CTAs per SM are stored there and
// nothing is launched; else p.ctas CTAs are. rows: query rows that the instance holds, in eights (1, 2 or 4).
cudaError_t qda_paged_weights_b4_f0(const QdaWeightsParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
cudaError_t qda_paged_weights_b4_f1(const QdaWeightsParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
cudaError_t qda_paged_weights_b8_f0(const QdaWeightsParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);
cudaError_t qda_paged_weights_b8_f1(const QdaWeightsParams* p, int D, int GS, int rows, int* ctas_per_sm, cudaStream_t s);

// The kernel for many rows (D <= 256), and the one ahead of it that lays out the query rows. prepare sets the shared memory
// limit on the current device and launches nothing.
constexpr int kPvRows = 128;   // query rows of a chunk
cudaError_t qda_paged_weights_tc_b4(const QdaWeightsParams* p, int D, bool prepare, cudaStream_t s);
cudaError_t qda_paged_weights_tc_b8(const QdaWeightsParams* p, int D, bool prepare, cudaStream_t s);
cudaError_t qda_paged_weights_lay(const QdaWeightsParams& p, cudaStream_t s);
