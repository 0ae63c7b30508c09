// The paged cache (sm_103a): the step's tables, the append into pages, and the host side of the paged calls.
#include <algorithm>
#include <atomic>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qda_paged_check.h"
#include "qda_paged_sched.cuh"

namespace qda {

// ----------------------------------------------------------------------------------------------------- tables

constexpr int kMapThreads = 512;   // one thread per sequence in the scan (QDA_MAX_B)
static_assert(kMapThreads >= QDA_MAX_B, "one thread per sequence");

// Inclusive scan of a pair over the CTA's threads: shuffles in the warp, the warps' totals through shared memory.
__device__ __forceinline__ longlong2 block_scan2(longlong2 v, longlong2* tot) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long x = __shfl_up_sync(0xffffffffu, v.x, o), y = __shfl_up_sync(0xffffffffu, v.y, o);
    if (lane >= o) {
      v.x += x;
      v.y += y;
    }
  }
  if (lane == 31) tot[warp] = v;
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    v.x += tot[w].x;
    v.y += tot[w].y;
  }
  return v;
}

// Every CTA scans the B lengths for itself (at most QDA_MAX_B values, all in L2) and then writes its share of the
// tokens' slots and of the new pages: one launch, no CTA waits for another. A token on a new page takes its page id from
// the free list and not from the table, which another CTA may be writing. Bound by the latency of two dependent loads and
// the scan: 2.7 us for 64 sequences' tokens, 4.2 us for 512 sequences of 1 to 129 tokens (33000 slots, pages of 16), 7.1
// and 8.1 us with the host's part of a call.
__global__ void __launch_bounds__(kMapThreads)
    qda_paged_map_kernel(const int* __restrict__ old_len, const int* __restrict__ new_len, int* __restrict__ table,
                         const int* __restrict__ free_pages, int* __restrict__ q_start, int* __restrict__ kv_len,
                         int* __restrict__ slots, int* __restrict__ positions, int* __restrict__ used, int B,
                         int max_pages, int n_free, int page_shift, int max_tokens, unsigned int* err) {
  __shared__ longlong2 tot[kMapThreads / 32];
  __shared__ int s_start[QDA_MAX_B + 1], s_take[QDA_MAX_B + 1], s_old[QDA_MAX_B];
  const int tid = threadIdx.x;
  const int pmask = (1 << page_shift) - 1;
  const unsigned top_page = 0x7fffffffu >> page_shift;   // the pool's size is not known here: no id whose slots pass 32 bits
  int o = 0, n = 0;
  bool bad = false;
  if (tid < B) {
    o = old_len[tid];
    n = new_len[tid];
    bad = o < 0 || n < 0;
    o = max(o, 0);
    n = max(n, 0);
    if ((long long)o + n > 0x7fffffffLL) {
      bad = true;
      n = 0x7fffffff - o;
    }
  }
  const int had = (int)(((long long)o + pmask) >> page_shift), has = (int)(((long long)o + n + pmask) >> page_shift);
  const longlong2 in = block_scan2(make_longlong2(n, has - had), tot);
  constexpr long long kTop = 0x7fffffffLL;
  if (tid < B) {
    s_start[tid] = (int)min(in.x - n, kTop);
    s_take[tid] = (int)min(in.y - (has - had), kTop);
    s_old[tid] = o;
    if (tid == B - 1) {
      s_start[B] = (int)min(in.x, kTop);
      s_take[B] = (int)min(in.y, kTop);
      bad = bad || in.x > max_tokens;
    }
    if (blockIdx.x == 0) {
      q_start[tid] = (int)min(in.x - n, kTop);
      kv_len[tid] = o + n;
      if (tid == B - 1) {
        q_start[B] = (int)min(in.x, kTop);
        used[0] = (int)min(in.y, kTop);
      }
    }
  }
  __syncthreads();
  const int first = blockIdx.x * kMapThreads + tid, step = gridDim.x * kMapThreads;
  // the new pages, in the order of sequences and columns
  const int pages = s_take[B];
  for (long long i = first; i < pages; i += step) {
    const int b = qda_seq_of(s_take, B, (int)i);
    const long long col = (((long long)s_old[b] + pmask) >> page_shift) + (i - s_take[b]);
    if (col >= max_pages) {
      bad = true;
      continue;
    }
    const int pg = i < n_free ? free_pages[i] : -1;
    const bool have = (unsigned)pg <= top_page;
    bad = bad || !have;
    table[(size_t)b * max_pages + col] = have ? pg : -1;
  }
  const int total = s_start[B];
  for (long long t = first; t < max_tokens; t += step) {
    int slot = -1, pos = -1;
    if (t < total) {
      const int b = qda_seq_of(s_start, B, (int)t);
      const int ob = s_old[b];
      const long long at = (long long)ob + (t - s_start[b]);
      const long long col = at >> page_shift, old_cols = ((long long)ob + pmask) >> page_shift;
      pos = (int)at;
      int pg = -1;
      if (col < max_pages) {
        const long long nth = s_take[b] + (col - old_cols);
        if (col < old_cols) pg = table[(size_t)b * max_pages + col];
        else if (nth < n_free) pg = free_pages[nth];
      }
      if ((unsigned)pg <= top_page) slot = (pg << page_shift) | ((int)at & pmask);
      else bad = true;
    }
    slots[t] = slot;
    if (positions) positions[t] = pos;
  }
  if (bad) atomicOr(err, QDA_ERR_BIT_PAGED);
}

// ----------------------------------------------------------------------------------------------------- append

template <bool F16>
__device__ __forceinline__ uint32_t to_bits16(float x) {
  if constexpr (F16) return __half_as_ushort(__float2half_rn(x));
  else return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

template <bool F16>
__device__ __forceinline__ uint32_t to_bits16x2(float lo, float hi) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
}

// The quantizer's code of x.
__device__ __forceinline__ float exact_code(float x, float b, float s, float qmax) {
  return s == 0.f ? 0.f : fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x, b), s)), 0.f), qmax);
}

struct AppendParams {
  const void *k, *v;
  long long kt, kh, vt, vh;      // strides of k and v in elements
  const int* slots;
  uint32_t *kp, *vp;
  uint16_t *ks, *kb, *vs, *vb, *k_held, *v_held;
  uint32_t rows;                 // T * Hkv
  int Hkv, pool_slots, page_shift, GS;
  unsigned int* err;
};

// A row of D values takes D / E lanes of E = 8 consecutive values: 16 bytes or more per load and whole words of codes per
// lane (two warps at D = 512; 16 values a lane take 36.3 us there for the rows below, 8 take 34.9). A group spans GS / E
// lanes of one warp (minimum and maximum by shuffles). The arithmetic is the quantizer's, in IEEE fp32; a code is the
// nearest integer to a multiplication by 1 / s wherever the distance to a middle between two codes is beyond that product's
// error; next to a middle the remainder decides, and only scales and biases of extreme size are divided (17722 prompt
// tokens 143 us with a division per value, 95 so; 3500 tokens in fp32 at D = 512 34.9 either way). K and V of a row go to
// the same lanes, both loads in flight together. Bound by issue (39 instructions per value) and then by HBM: 17722 tokens
// of 8 heads of 256 values, bf16 -> 8-bit, 95 us (3.9 TB/s read and written, floor 55); 3500 tokens of 8 heads of 512
// values, fp32 -> 4-bit, 35 us (4.6 TB/s, floor 23.5); one token of 64 sequences 3.9.
template <int BITS, int E, int LANES, bool F16, int SRC>
__global__ void __launch_bounds__(256) qda_paged_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int D = LANES * E, PER = 32 / BITS, W = D / PER, WL = E / PER;
  constexpr float QMAX = (float)((1 << BITS) - 1);
  const uint32_t row = blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const bool live = row < p.rows;   // a warp may hold several rows: all its lanes stay for the shuffles
  const int lane = threadIdx.x % LANES;
  const uint32_t rr = live ? row : p.rows - 1, t = rr / (uint32_t)p.Hkv;
  const int h = (int)(rr - t * (uint32_t)p.Hkv);
  const int slot = p.slots[t];
  float x[2][E];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const long long at = w == 0 ? (long long)t * p.kt + h * p.kh : (long long)t * p.vt + h * p.vh;
    const void* src = w == 0 ? p.k : p.v;
    if constexpr (SRC == QDA_FP32) {
      const float4* s = reinterpret_cast<const float4*>(static_cast<const float*>(src) + at + lane * E);
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        const float4 a = __ldcs(s + i);
        x[w][4 * i] = a.x;
        x[w][4 * i + 1] = a.y;
        x[w][4 * i + 2] = a.z;
        x[w][4 * i + 3] = a.w;
      }
    } else {
      const uint4* s = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(src) + at + lane * E);
#pragma unroll
      for (int i = 0; i < E / 8; ++i) {
        const uint4 a = __ldcs(s + i);
        const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[w][8 * i + 2 * j] = half_bits_to_float<SRC == QDA_FP16>(u[j] & 0xffffu);
          x[w][8 * i + 2 * j + 1] = half_bits_to_float<SRC == QDA_FP16>(u[j] >> 16);
        }
      }
    }
  }
  if (live && slot >= p.pool_slots && lane == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
  const bool put = live && slot >= 0 && slot < p.pool_slots;
  const long long orow = qda_pool_row(slot >> p.page_shift, h, slot & ((1 << p.page_shift) - 1), p.Hkv, p.page_shift);
  const int lpg = p.GS / E, NG = D / p.GS;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    float lo = x[w][0], hi = x[w][0];
#pragma unroll
    for (int e = 1; e < E; ++e) {
      lo = fminf(lo, x[w][e]);
      hi = fmaxf(hi, x[w][e]);
    }
    for (int off = 1; off < lpg; off <<= 1) {
      lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, off));
      hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, off));
    }
    const uint32_t sb = to_bits16<F16>(__fdiv_rn(__fsub_rn(hi, lo), QMAX)), bb = to_bits16<F16>(lo);
    const float s = half_bits_to_float<F16>(sb), b = half_bits_to_float<F16>(bb);
    // code = clamp(rint(RN((x - b) / s))), without the division: the product with 1 / s is off by less than 2^-14 in the
    // codes' range (q 2^-23 and the quotient's own rounding, q < 258). Adding 1.5 * 2^23 rounds to the nearest integer,
    // ties to even, and leaves it in the low bits. A value within 2^-14 of the middle m between two codes (common: the
    // inputs are coarse) is decided by the remainder d - m s, whose sign a fused multiply-add gives exactly: |d - m s| up to
    // s times half a step of m means that the quotient rounds to m itself (it never lies halfway between two floats), a tie.
    constexpr float ROUND = 12582912.f, NEAR = 0.5f - 6.2e-5f;
    const bool plain = s >= 1e-30f && s <= 1e30f && fabsf(b) <= 1e30f;
    const float inv = plain ? __frcp_rn(s) : 0.f;
    float r[E];   // code + ROUND
    float off = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float q = fminf(fmaxf(__fmul_rn(__fsub_rn(x[w][e], b), inv), 0.f), QMAX);
      r[e] = __fadd_rn(q, ROUND);
      off = fmaxf(off, fabsf(__fsub_rn(q, __fsub_rn(r[e], ROUND))));
    }
    if (off > NEAR) {
      const float s24 = s * 5.9604644775390625e-8f;   // s 2^-24
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float d = __fsub_rn(x[w][e], b);
        const float q = fminf(fmaxf(__fmul_rn(d, inv), 0.f), QMAX), c = __fsub_rn(r[e], ROUND);
        const uint32_t side = __float_as_uint(__fsub_rn(q, c)) & 0x80000000u;
        const float m = c + __uint_as_float(0x3f000000u | side);                           // the nearest middle
        const float rest = __uint_as_float(__float_as_uint(__fmaf_rn(-m, s, d)) ^ side);   // > 0: beyond it
        const float step = s24 * __uint_as_float(__float_as_uint(m) & 0x7f800000u);
        // beyond by more than step: the next code; within: the even one of the two
        const float edge = __float_as_uint(r[e]) & 1u ? -step : step;
        if (rest > edge) r[e] = fminf(__fadd_rn(r[e], __uint_as_float(0x3f800000u | side)), ROUND + QMAX);
      }
    }
    if (!plain) {
#pragma unroll
      for (int e = 0; e < E; ++e) r[e] = __fadd_rn(exact_code(x[w][e], b, s, QMAX), ROUND);
    }
    if (put) {
      uint32_t word[WL];
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        word[i] = 0;
#pragma unroll
        for (int j = 0; j < PER; ++j) word[i] |= (__float_as_uint(r[i * PER + j]) & 0xffu) << (BITS * j);
      }
      uint32_t* dst = (w == 0 ? p.kp : p.vp) + orow * W + lane * WL;
      if constexpr (WL == 1) {
        dst[0] = word[0];
      } else if constexpr (WL == 2) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(word[0], word[1]);
      } else {
        *reinterpret_cast<uint4*>(dst) = make_uint4(word[0], word[1], word[2], word[3]);
      }
      if (lane % lpg == 0) {
        (w == 0 ? p.ks : p.vs)[orow * NG + lane / lpg] = (uint16_t)sb;
        (w == 0 ? p.kb : p.vb)[orow * NG + lane / lpg] = (uint16_t)bb;
      }
    }
    if (live && p.k_held != nullptr) {
      uint4* dst = reinterpret_cast<uint4*>((w == 0 ? p.k_held : p.v_held) + (size_t)rr * D + lane * E);
#pragma unroll
      for (int i = 0; i < E / 8; ++i) {
        uint32_t u[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          u[j] = to_bits16x2<F16>(fmaf(s, r[8 * i + 2 * j] - ROUND, b), fmaf(s, r[8 * i + 2 * j + 1] - ROUND, b));
        __stcs(dst + i, make_uint4(u[0], u[1], u[2], u[3]));
      }
    }
  }
}

template <int BITS, bool F16, int SRC>
cudaError_t launch_append(const AppendParams& p, int D, cudaStream_t s) {
  const int lanes = D / 8;
  const unsigned grid = (unsigned)(((long long)p.rows * lanes + 255) / 256);
  switch (D) {
    case 64: qda_paged_append_kernel<BITS, 8, 8, F16, SRC><<<grid, 256, 0, s>>>(p); break;
    case 128: qda_paged_append_kernel<BITS, 8, 16, F16, SRC><<<grid, 256, 0, s>>>(p); break;
    case 256: qda_paged_append_kernel<BITS, 8, 32, F16, SRC><<<grid, 256, 0, s>>>(p); break;
    default: qda_paged_append_kernel<BITS, 8, 64, F16, SRC><<<grid, 256, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

template <int BITS>
cudaError_t launch_append_types(const AppendParams& p, int D, bool f16, int src, cudaStream_t s) {
  if (f16)
    return src == QDA_BF16   ? launch_append<BITS, true, QDA_BF16>(p, D, s)
           : src == QDA_FP16 ? launch_append<BITS, true, QDA_FP16>(p, D, s)
                             : launch_append<BITS, true, QDA_FP32>(p, D, s);
  return src == QDA_BF16   ? launch_append<BITS, false, QDA_BF16>(p, D, s)
         : src == QDA_FP16 ? launch_append<BITS, false, QDA_FP16>(p, D, s)
                           : launch_append<BITS, false, QDA_FP32>(p, D, s);
}

// ------------------------------------------------------------------------------------------- merge of split tiles

// out = sum_c o_c 2^(m_c - M) / sum_c l_c 2^(m_c - M) over the CTAs c that share a tile, in CTA order. CTA (x, y) takes the
// tile that starts in piece x and goes on behind it (most CTAs find none and end), and 8 / WPR of its rows, WPR warps to a
// row: each folds every WPR-th part, then the warps' sums meet in shared memory. Launched with programmatic dependent
// launch, ahead of the end of the kernel before it. Bound by latency: a record, then its parts (behind the 64 sequences'
// tokens 6 us, behind 131072 keys 11, behind the long chunk 14). The kernels before it leave the records; when the merge
// found the shared tiles by scanning the lengths itself, it took 45 us more behind 64 sequences' tokens.
template <int D, int WPR, bool LSE>
__global__ void __launch_bounds__(256) qda_paged_merge_kernel(const __grid_constant__ QdaPagedParams p, int MT) {
  constexpr int E = D / 64;   // pairs of values per lane
  __shared__ float2 s_o[WPR > 1 ? 8 : 1][D / 2];
  __shared__ float2 s_ml[8];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
  if constexpr (WPR == 1) pdl_launch_dependents();   // behind the chunk kernel another kernel may follow
  if (blockIdx.x == 0 && blockIdx.y == 0) {          // what the call was given, looked over once
    bool bad = threadIdx.x == 0 && (p.q_start[0] < 0 || p.q_start[p.B] > p.total_q);
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
      const int rows = p.q_start[b + 1] - max(p.q_start[b], 0), n = p.kv_len[b];
      bad = bad || rows < 0 || (rows > 0 && (n < 0 || n > (long long)p.max_pages << p.page_shift));
    }
    if (bad) atomicOr(p.err, QDA_ERR_BIT_PAGED);
  }
  pdl_wait();
  const QdaPagedSplitTile t = p.split[c];
  if (!t.go || (int)blockIdx.y * (8 / WPR) >= t.rows) return;
  const int last = t.last;
  const int r = blockIdx.y * (8 / WPR) + warp / WPR, part = warp % WPR;
  const bool live = r < t.rows;
  float m = -INFINITY, l = 0.f;
  float2 o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = make_float2(0.f, 0.f);
  if (live) {
#pragma unroll 4
    for (int k = c + part; k <= last; k += WPR) {
      const QdaPagedSplitTile& rk = p.split[k];
      if (!(k == c ? rk.last_filled : rk.first_filled)) continue;
      const size_t at = (size_t)(2 * k + (k == c)) * MT + r;
      const float2 ml = p.part_ml[at];
      const float2* po = reinterpret_cast<const float2*>(p.part_o + at * D);
      float2 v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = po[e * 32 + lane];
      const float mn = fmaxf(m, ml.x);
      const float a = m == -INFINITY ? 0.f : exp2f(m - mn), w = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mn);
      m = mn;
      l = fmaf(l, a, ml.y * w);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        o[e].x = fmaf(o[e].x, a, v[e].x * w);
        o[e].y = fmaf(o[e].y, a, v[e].y * w);
      }
    }
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) s_o[warp][e * 32 + lane] = o[e];
    if (lane == 0) s_ml[warp] = make_float2(m, l);
    __syncthreads();
    if (part != 0 || !live) return;
    for (int w = 1; w < WPR; ++w) {
      const float2 ml = s_ml[warp + w];
      const float mn = fmaxf(m, ml.x);
      // (a part without a reference is zeros, or NaN that has to stay: of a query that is not a number)
      const float a = m == -INFINITY ? 0.f : exp2f(m - mn), x = ml.x == -INFINITY ? 0.f : exp2f(ml.x - mn);
      m = mn;
      l = fmaf(l, a, ml.y * x);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float2 v = s_o[warp + w][e * 32 + lane];
        o[e].x = fmaf(o[e].x, a, v.x * x);
        o[e].y = fmaf(o[e].y, a, v.y * x);
      }
    }
  }
  if (!live) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int row = t.row0 + r, tok = row / p.nrep;
  uint32_t* dst = reinterpret_cast<uint32_t*>(
      p.out + ((long long)(t.token0 + tok) * p.H + (t.unit / p.parts) * p.nrep + (row - tok * p.nrep)) * p.D +
      (t.unit % p.parts) * D);
#pragma unroll
  for (int e = 0; e < E; ++e)
    dst[e * 32 + lane] = p.f16 ? to_bits16x2<true>(o[e].x * inv, o[e].y * inv) : to_bits16x2<false>(o[e].x * inv, o[e].y * inv);
  if (LSE && lane == 0 && t.unit % p.parts == 0)
    qda_put_lse(p, t.token0 + tok, (t.unit / p.parts) * p.nrep + (row - tok * p.nrep), m, l, p.lse_unit);
}

template <int D>
cudaError_t launch_merge(const QdaPagedParams& p, int rows, cudaStream_t s) {
  // few rows per tile: a tile may be shared by many CTAs, so eight warps fold one row; many rows: a warp each
  const bool few = rows <= 16;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p.ctas, (unsigned)(few ? rows : rows / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (p.lse != nullptr)
    return few ? cudaLaunchKernelEx(&cfg, qda_paged_merge_kernel<D, 8, true>, p, rows)
               : cudaLaunchKernelEx(&cfg, qda_paged_merge_kernel<D, 1, true>, p, rows);
  return few ? cudaLaunchKernelEx(&cfg, qda_paged_merge_kernel<D, 8, false>, p, rows)
             : cudaLaunchKernelEx(&cfg, qda_paged_merge_kernel<D, 1, false>, p, rows);
}

// ----------------------------------------------------------------------------- rows beside keys that they do not see

// In the chunk kernel a block of 128 keys shares one power of two, chosen from the largest of them. Its fp16 operands are
// off by at most half a step of the subnormal numbers, 2^-19 of the largest with 4-bit codes and 2^-22 with 8-bit ones:
// next to nothing for a row that sees the largest, but a token in the middle of a causal chunk does not see the keys
// behind it, whatever they hold. This kernel, behind the merge of a causal call, looks for tokens whose own part of their
// last block holds less than 1 / FAR of the block's largest key, or value (so that the operands' error passes 2^-13 of
// what they see themselves), and does their rows anew in fp32: a CTA takes eight rows of a KV head at a time, a thread per
// key for the scores and a thread per dimension for the values, so that a key is read once for all eight. On ordinary
// inputs it finds none: a warp per KV head and block of new tokens reads their scales and biases. What it costs then: chunk
// over 32768 keys 858 -> 861 us, ragged chunks at D = 256 424 -> 430 us, 250 tokens at D = 512 99 -> 100 us (the same done
// by the chunk kernel's own warps costs it registers: 858 -> 915 us). 32 tokens of 8 heads done anew: 0.1 ms over 1024
// keys, 2.7 over 32768 (D 128, 4-bit; a row at a time it took 193), 7.8 at D 256, 8-bit.
constexpr int kFarThreads = 256, kFarWarps = kFarThreads / 32;
constexpr int kFarRows = 8;    // rows that are done at a time
constexpr int kFarParts = 16;  // CTAs at most that share a unit's rows

struct FarShared {
  long long first[QDA_MAX_B + 1];   // units (KV head, block of new tokens) before each sequence
  uint32_t found[kFarWarps][4];     // a bit per key of a warp's unit: the token there is done anew
  uint32_t row[kFarThreads];        // pool rows of the keys at hand (all ones: absent)
  float4 q[512][kFarRows / 4], w[kFarThreads][kFarRows / 4];   // queries by dimension, weights by key
  float red[kFarWarps][kFarRows], o[kFarThreads];
};

__device__ __forceinline__ int far_tokens(const QdaPagedParams& p, const PagedSeq& s) { return s.rows / p.nrep; }

// The blocks that hold a sequence's new tokens: *first and how many.
__device__ __forceinline__ int far_blocks(const QdaPagedParams& p, const PagedSeq& s, int* first) {
  const int end = min(s.n_all, s.base + far_tokens(p, s));   // keys that the last token sees
  *first = max(s.base, 0) / 128;
  return s.rows == 0 || end <= max(s.base, 0) ? 0 : (end - 1) / 128 - *first + 1;
}

// The largest that each of four keys (or values) from pool row `row` on can be; -1 for one that is not finite.
template <int BITS, int NG>
__device__ __forceinline__ void far_sizes(const uint16_t* scales, const uint16_t* biases, long long row, bool f16,
                                          float (&x)[4]) {
  constexpr float QMAX = (float)((1 << BITS) - 1);
  uint2 s[NG], b[NG];   // four rows of NG values, all on their way before the first is looked at
#pragma unroll
  for (int i = 0; i < NG; ++i) {
    s[i] = __ldg(reinterpret_cast<const uint2*>(scales + row * NG) + i);
    b[i] = __ldg(reinterpret_cast<const uint2*>(biases + row * NG) + i);
  }
  const uint32_t limit = f16 ? 0x7C00u : 0x7680u;   // the chunk kernel's: fp16 infinity; 2^110 in bf16
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t ts = 0, tb = 0;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      const int at = k * NG + g;
      auto half = [&](const uint2& w) { return (((at & 2) ? w.y : w.x) >> (16 * (at & 1))) & 0x7fffu; };
      ts = max(ts, half(s[at >> 2]));
      tb = max(tb, half(b[at >> 2]));
    }
    x[k] = max(ts, tb) < limit ? fmaf(half_bits_to_float_rt(ts, f16), QMAX, half_bits_to_float_rt(tb, f16)) : -1.f;
  }
}

// A warp: which keys of block j belong to tokens whose rows are to be done anew.
template <int BITS, int NG>
__device__ __forceinline__ void far_find(const QdaPagedParams& p, const PagedSeq& s, int b, int kvh, int j,
                                         uint32_t (&found)[4]) {
  constexpr float FAR = BITS == 4 ? 64.f : 512.f;
  const int lane = threadIdx.x & 31, pmask = (1 << p.page_shift) - 1;
  const int end = min((j + 1) * 128, min(s.n_all, s.base + far_tokens(p, s))), key0 = j * 128 + 4 * lane;
  const int pg = key0 < end ? __ldg(p.table + (size_t)b * p.max_pages + (key0 >> p.page_shift)) : -1;
  const bool have = (unsigned)pg < (unsigned)p.num_pages;   // four keys from a multiple of four on lie on one page
  const long long row = qda_pool_row(have ? pg : 0, kvh, key0 & pmask, p.Hkv, p.page_shift);
  float k[4], v[4];   // of this lane's four keys; then of all keys up to there
  far_sizes<BITS, NG>(p.ks, p.kb, row, p.f16, k);
  far_sizes<BITS, NG>(p.vs, p.vb, row, p.f16, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // a key counts if both parts of it are finite: else it is zero in the operands
    const bool counts = have && key0 + i < end && k[i] >= 0.f && v[i] >= 0.f;
    k[i] = counts ? k[i] : 0.f;
    v[i] = counts ? v[i] : 0.f;
    if (i > 0) {
      k[i] = fmaxf(k[i], k[i - 1]);
      v[i] = fmaxf(v[i], v[i - 1]);
    }
  }
  float kup = k[3], vup = v[3];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    kup = fmaxf(kup, __shfl_up_sync(0xffffffffu, kup, o));   // (lanes below o get their own)
    vup = fmaxf(vup, __shfl_up_sync(0xffffffffu, vup, o));
  }
  const float kall = __shfl_sync(0xffffffffu, kup, 31), vall = __shfl_sync(0xffffffffu, vup, 31);
  kup = __shfl_up_sync(0xffffffffu, kup, 1);
  vup = __shfl_up_sync(0xffffffffu, vup, 1);
  if (lane == 0) kup = vup = 0.f;
  // (zeros are exact in any unit: a token that sees nothing else of the block, padding for instance, is left as it is)
  auto far = [](float all, float own) { return own > 0.f && all > FAR * own; };
  uint32_t mine = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (key0 + i >= s.base && key0 + i < end && (far(kall, fmaxf(k[i], kup)) || far(vall, fmaxf(v[i], vup)))) mine |= 1u << i;
  // key 4 lane + i of the block is bit 4 lane + i of 128
#pragma unroll
  for (int y = 0; y < 4; ++y) found[y] = __reduce_or_sync(0xffffffffu, lane >> 3 == y ? mine << (4 * (lane & 7)) : 0u);
}

// A CTA: f(the threads' x) over all of them, for every thread and row.
template <typename F>
__device__ __forceinline__ void far_reduce(FarShared& sh, float (&x)[kFarRows], F f) {
#pragma unroll
  for (int r = 0; r < kFarRows; ++r) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) x[r] = f(x[r], __shfl_xor_sync(0xffffffffu, x[r], o));
  }
  __syncthreads();   // the last one's results are read
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int r = 0; r < kFarRows; ++r) sh.red[threadIdx.x >> 5][r] = x[r];
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kFarRows; ++r) {
    x[r] = sh.red[0][r];
#pragma unroll
    for (int w = 1; w < kFarWarps; ++w) x[r] = f(x[r], sh.red[w][r]);
  }
}

__device__ __forceinline__ void far_unpack(const float4 (&a)[kFarRows / 4], float (&x)[kFarRows]) {
#pragma unroll
  for (int i = 0; i < kFarRows / 4; ++i) {
    x[4 * i] = a[i].x;
    x[4 * i + 1] = a[i].y;
    x[4 * i + 2] = a[i].z;
    x[4 * i + 3] = a[i].w;
  }
}

// A CTA: output rows of up to kFarRows (token, query head) pairs of KV head kvh: heads[r] of the token in row tokens[r] of q
// over its keys n < seen[r] (0: no such row).
template <int BITS>
__device__ void far_rows(const QdaPagedParams& p, FarShared& sh, int b, int kvh, const int (&tokens)[kFarRows],
                         const int (&heads)[kFarRows], const int (&seen)[kFarRows]) {
  constexpr int PER = 32 / BITS;
  constexpr uint32_t MASK = (1u << BITS) - 1;
  const int tid = threadIdx.x, pmask = (1 << p.page_shift) - 1;
  const int* tab = p.table + (size_t)b * p.max_pages;
  __syncthreads();   // the last rows' queries and sums are read
#pragma unroll
  for (int r = 0; r < kFarRows; ++r) {
    const uint16_t* q = p.q + (long long)tokens[r] * p.q_tstride + (long long)heads[r] * p.q_hstride;
    for (int d = tid; d < p.D; d += kFarThreads)
      reinterpret_cast<float*>(&sh.q[d])[r] = seen[r] ? half_bits_to_float_rt(q[d], p.f16) : 0.f;
  }
  // values: a thread per dimension (two at D = 512) and key in turn
  const int part = p.D < kFarThreads ? tid / p.D : 0, parts = p.D < kFarThreads ? kFarThreads / p.D : 1;
  const int d0 = tid & (p.D - 1);
  int most = 0;
  float m[kFarRows], l[kFarRows], o[2][kFarRows];
#pragma unroll
  for (int r = 0; r < kFarRows; ++r) {
    m[r] = -INFINITY;
    l[r] = o[0][r] = o[1][r] = 0.f;
    most = max(most, seen[r]);
  }
  for (int n0 = 0; n0 < most; n0 += kFarThreads) {
    const int n = n0 + tid;
    const int pg = n < most ? __ldg(tab + (n >> p.page_shift)) : -1;
    const bool there = (unsigned)pg < (unsigned)p.num_pages;
    const uint32_t row = there ? (uint32_t)qda_pool_row(pg, kvh, n & pmask, p.Hkv, p.page_shift) : 0xffffffffu;
    __syncthreads();   // queries are there, the last weights and rows read
    sh.row[tid] = row;
    float x[kFarRows], top[kFarRows];
#pragma unroll
    for (int r = 0; r < kFarRows; ++r) x[r] = 0.f;
    if (there) {
      const uint4* codes = reinterpret_cast<const uint4*>(p.kp + (uint64_t)row * p.W);
      for (int d = 0; d < p.D; d += 4 * PER) {   // 16 bytes of codes, of one group
        const uint4 a = __ldg(codes + d / (4 * PER));
        const uint64_t g = (uint64_t)row * p.NG + d / p.GS;
        const float s = half_bits_to_float_rt(__ldg(p.ks + g), p.f16), z = half_bits_to_float_rt(__ldg(p.kb + g), p.f16);
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
#pragma unroll
          for (int e = 0; e < PER; ++e) {
            const float v = fmaf(s, (float)((w[i] >> (BITS * e)) & MASK), z);
            float q[kFarRows];
            far_unpack(sh.q[d + i * PER + e], q);
#pragma unroll
            for (int r = 0; r < kFarRows; ++r) x[r] = fmaf(q[r], v, x[r]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < kFarRows; ++r) top[r] = x[r] = there && n < seen[r] ? x[r] * p.qscale : -INFINITY;
    far_reduce(sh, top, [](float a, float c) { return fmaxf(a, c); });
    float w[kFarRows];
#pragma unroll
    for (int r = 0; r < kFarRows; ++r) {
      const float mn = fmaxf(m[r], top[r]);
      const float a = m[r] == -INFINITY ? 0.f : exp2f(m[r] - mn);
      w[r] = there && n < seen[r] ? exp2f(x[r] - (mn == -INFINITY ? 0.f : mn)) : 0.f;
      m[r] = mn;
      l[r] = l[r] * a + w[r];
      o[0][r] *= a;
      o[1][r] *= a;
    }
#pragma unroll
    for (int i = 0; i < kFarRows / 4; ++i) sh.w[tid][i] = make_float4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    __syncthreads();
    const int many = min(kFarThreads, most - n0);
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int d = d0 + y * kFarThreads;
      if (d >= p.D) break;
      const int at = d / PER, sh_bits = BITS * (d % PER), g = d / p.GS;
#pragma unroll 1
      for (int i0 = part; i0 < many; i0 += 4 * parts) {
        uint32_t c[4], rw[4], us[4], uz[4];   // four keys' loads on their way together
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = i0 + j * parts;
          rw[j] = i < many ? sh.row[i] : 0xffffffffu;
          const uint64_t ok = rw[j] == 0xffffffffu ? 0 : rw[j];
          c[j] = __ldg(p.vp + ok * p.W + at);
          us[j] = __ldg(p.vs + ok * p.NG + g);
          uz[j] = __ldg(p.vb + ok * p.NG + g);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (rw[j] == 0xffffffffu) continue;
          const float s = half_bits_to_float_rt(us[j], p.f16), z = half_bits_to_float_rt(uz[j], p.f16);
          const float v = fmaf(s, (float)((c[j] >> sh_bits) & MASK), z);
          float wt[kFarRows];
          far_unpack(sh.w[i0 + j * parts], wt);
#pragma unroll
          for (int r = 0; r < kFarRows; ++r)   // what a row does not see stays out, whatever it holds
            o[y][r] = wt[r] == 0.f ? o[y][r] : fmaf(wt[r], v, o[y][r]);
        }
      }
    }
  }
  far_reduce(sh, l, [](float x, float y) { return x + y; });
#pragma unroll 1
  for (int r = 0; r < kFarRows; ++r) {
    float mine[2] = {0.f, 0.f}, sum = 0.f, ref = 0.f;
    int t = 0, h = 0, see = 0;
#pragma unroll
    for (int k = 0; k < kFarRows; ++k)   // (registers have no index)
      if (k == r) {
        mine[0] = o[0][k];
        mine[1] = o[1][k];
        sum = l[k];
        ref = m[k];
        t = tokens[k];
        h = heads[k];
        see = seen[k];
      }
    __syncthreads();
    sh.o[tid] = mine[0];
    __syncthreads();
    if (part != 0 || see == 0) continue;
    for (int i = 1; i < parts; ++i) mine[0] += sh.o[tid + i * p.D];
    if (tid == 0 && p.lse != nullptr) qda_put_lse(p, t, h, ref, sum, 0.f);
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t* out = p.out + ((long long)t * p.H + h) * p.D;
#pragma unroll
    for (int y = 0; y < 2; ++y)
      if (d0 + y * kFarThreads < p.D)
        out[d0 + y * kFarThreads] = (uint16_t)(p.f16 ? to_bits16<true>(mine[y] * inv) : to_bits16<false>(mine[y] * inv));
  }
}

template <int BITS>
__global__ void __launch_bounds__(kFarThreads) qda_paged_far_kernel(const __grid_constant__ QdaPagedParams p) {
  __shared__ FarShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // units before each sequence: a warp scans the batch
  if (warp == 0) {
    long long carry = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int first;
      const long long n = b < p.B ? (long long)p.Hkv * far_blocks(p, paged_seq(p, b, 128), &first) : 0;
      long long up = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, up, o);
        if (lane >= o) up += x;
      }
      if (b < p.B) sh.first[b] = carry + up - n;
      carry += __shfl_sync(0xffffffffu, up, 31);
    }
    if (lane == 0) sh.first[p.B] = carry;
  }
  __syncthreads();
  const long long units = sh.first[p.B];
  // few units: several warps, of different CTAs, find the same one's rows and share them
  const int share = units == 0 ? 1 : (int)max(1LL, min((long long)kFarParts, (long long)gridDim.x * kFarWarps / units));
  const long long items = units * share;
  bool waited = false;
  // items i0, i0 + gridDim.x, ...: a warp each; item i is unit i % units and part i / units of its rows
  for (long long i0 = blockIdx.x; i0 < items; i0 += (long long)gridDim.x * kFarWarps) {
    auto unit = [&](long long item, int* b, int* kvh, int* j) {
      const long long u = item % units;
      *b = qda_seq_of(sh.first, p.B, u);
      const PagedSeq s = paged_seq(p, *b, 128);
      const int blocks = far_blocks(p, s, j);
      const long long i = u - sh.first[*b];
      *kvh = (int)(i / blocks);
      *j += (int)(i - (long long)*kvh * blocks);
      return s;
    };
    uint32_t found[4] = {0u, 0u, 0u, 0u};
    const long long mine = i0 + (long long)warp * gridDim.x;
    if (mine < items) {
      int b, kvh, j;
      const PagedSeq s = unit(mine, &b, &kvh, &j);
      switch (p.NG) {
        case 1: far_find<BITS, 1>(p, s, b, kvh, j, found); break;
        case 2: far_find<BITS, 2>(p, s, b, kvh, j, found); break;
        case 4: far_find<BITS, 4>(p, s, b, kvh, j, found); break;
        case 8: far_find<BITS, 8>(p, s, b, kvh, j, found); break;
        default: far_find<BITS, 16>(p, s, b, kvh, j, found); break;
      }
    }
    if (!__syncthreads_or(found[0] | found[1] | found[2] | found[3])) continue;
    // rare from here on
    if (lane == 0) {
#pragma unroll
      for (int y = 0; y < 4; ++y) sh.found[warp][y] = found[y];
    }
    __syncthreads();
    if (!waited) pdl_wait();   // the merge has written its rows
    waited = true;
    for (int w = 0; w < kFarWarps && i0 + (long long)w * gridDim.x < items; ++w) {
      int b, kvh, j;
      const long long item = i0 + (long long)w * gridDim.x;
      const PagedSeq s = unit(item, &b, &kvh, &j);
      const int part = (int)(item / units);
      int tokens[kFarRows], heads[kFarRows], seen[kFarRows], at = 0, group = 0;   // the rows of the next group, as they are met
      auto flush = [&]() {
        for (int r = at; r < kFarRows; ++r) tokens[r] = heads[r] = seen[r] = 0;
        if (at > 0 && group % share == part) far_rows<BITS>(p, sh, b, kvh, tokens, heads, seen);
        at = 0;
        ++group;
      };
      for (int key = 0; key < 128; ++key) {
        if (!((sh.found[w][key >> 5] >> (key & 31)) & 1u)) continue;
        const int pos = j * 128 + key;
        for (int r = 0; r < p.nrep; ++r) {
          tokens[at] = s.first + pos - s.base;
          heads[at] = kvh * p.nrep + r;
          seen[at] = pos + 1;
          if (++at == kFarRows) flush();
        }
      }
      if (at > 0) flush();
    }
    __syncthreads();
  }
  if (!waited) pdl_wait();   // what follows this kernel follows the merge
}

cudaError_t launch_far(const QdaPagedParams& p, int bits, int sms, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)sms);
  cfg.blockDim = dim3(kFarThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return bits == 4 ? cudaLaunchKernelEx(&cfg, qda_paged_far_kernel<4>, p)
                   : cudaLaunchKernelEx(&cfg, qda_paged_far_kernel<8>, p);
}

// The kernel a call takes, from what the host knows: the shape and the bound on a sequence's new tokens.
struct PagedPlan {
  bool chunk;              // the chunk kernel (else the split kernel)
  int rows, ctas, min_keys, parts;
  size_t o_bytes, ml_bytes, bytes;   // workspace: partial outputs, (reference, sum) pairs, all with the split tiles
};

using SplitFn = cudaError_t (*)(const QdaPagedParams*, int, int, int, int*, cudaStream_t);
SplitFn split_fn(int bits, bool f16, bool lse) {
  if (lse)
    return bits == 4 ? (f16 ? qda_paged_split_b4_f1_lse : qda_paged_split_b4_f0_lse)
                     : (f16 ? qda_paged_split_b8_f1_lse : qda_paged_split_b8_f0_lse);
  return bits == 4 ? (f16 ? qda_paged_split_b4_f1 : qda_paged_split_b4_f0)
                   : (f16 ? qda_paged_split_b8_f1 : qda_paged_split_b8_f0);
}

// Rows (new tokens times query heads of a KV head) up to which the split kernel takes a call. Its time grows with every 16
// rows (8 at D = 512), the chunk kernel's stays the same up to 128. Split against chunk kernel, 8 KV heads and about 90000
// keys in all: D 64, 8-bit, 32 rows 84 / 85 us (64 rows 100 / 97), D 128, 4-bit, 16 rows 65 / 99, 32 rows 107 / 100 (one
// sequence alone 82 / 86), D 256, 4-bit, 16 rows 98 / 130 (32 rows of 4 sequences' tokens 91 / 67), D 512, 4-bit, 16 rows
// 240 / 339, 32 rows 455 / 338 (of one short sequence 80 / 95). The rule knows neither lengths nor batch, which the device
// alone has, and takes one kernel for the whole call: 63 single tokens (98 us by themselves) and a chunk of 512 over 8000
// keys (93 us) take 375 us in one call with max_q = 512, where every token walks its keys as a tile of 256 rows.
constexpr long long split_rows(int D) { return D == 512 ? 24 : D == 256 ? 16 : 32; }

cudaError_t chunk_run(const QdaPagedParams* p, int D, int bits, int rows, bool lse, bool prepare, cudaStream_t s) {
  const auto run = bits == 4 ? (lse ? qda_paged_chunk_b4_lse : qda_paged_chunk_b4) : (lse ? qda_paged_chunk_b8_lse : qda_paged_chunk_b8);
  return run(p, D, rows / 128, prepare, s);
}

int paged_plan(int nrep, long long max_q, int D, int GS, int bits, bool f16, bool lse, int sms, PagedPlan* plan) {
  const long long rows = max_q * nrep;
  int dev = 0;
  const cudaError_t de = cudaGetDevice(&dev);
  if (de != cudaSuccess || dev < 0 || dev >= 64) return qda_cuda_fail(de == cudaSuccess ? cudaErrorInvalidDevice : de);
  const int di = D == 64 ? 0 : D == 128 ? 1 : D == 256 ? 2 : 3, gi = GS == 32 ? 0 : GS == 64 ? 1 : 2;
  plan->chunk = rows > split_rows(D);
  if (plan->chunk) {
    plan->rows = rows > 128 && D <= 128 ? 256 : 128;
    plan->min_keys = 512;
    plan->parts = D == 512 ? 2 : 1;
    plan->ctas = sms;
    static std::atomic<bool> ready[64][2][2][4][2] = {};
    std::atomic<bool>& r = ready[dev][lse][bits == 8][di][plan->rows == 256];
    if (!r.load()) {
      const cudaError_t e = chunk_run(nullptr, D, bits, plan->rows, lse, true, nullptr);
      if (e != cudaSuccess) return qda_cuda_fail(e);
      r.store(true);
    }
  } else {
    plan->rows = rows > 8 && D <= 256 ? 16 : 8;
    plan->min_keys = 176;
    plan->parts = 1;
    // resident CTAs per SM of an instance, 0 = not asked yet. The grid is the one of the instance without the rows' sums for
    // either, so that a call's outputs do not depend on whether it asks for them.
    static std::atomic<int> cache[64][2][2][2][4][3][2] = {};
    int occ = 0;
    for (int with = 0; with <= (lse ? 1 : 0); ++with) {
      std::atomic<int>& slot = cache[dev][with][bits == 8][f16][di][gi][plan->rows == 16];
      int n = slot.load();
      if (n == 0) {
        const cudaError_t e = split_fn(bits, f16, with != 0)(nullptr, D, GS, plan->rows, &n, nullptr);
        if (e != cudaSuccess) return qda_cuda_fail(e);
        n = std::max(n, 1);
        slot.store(n);
      }
      if (with == 0) occ = n;
    }
    plan->ctas = sms * occ;
  }
  const size_t n = (size_t)2 * plan->ctas * plan->rows;
  plan->o_bytes = (n * (D / plan->parts) * 4 + 255) & ~(size_t)255;
  plan->ml_bytes = (n * sizeof(float2) + 255) & ~(size_t)255;
  plan->bytes = plan->o_bytes + plan->ml_bytes + plan->ctas * sizeof(QdaPagedSplitTile);
  return QDA_OK;
}

}  // namespace qda

cudaError_t qda_launch_paged_merge(const QdaPagedParams& p, int rows, cudaStream_t s) {
  switch (p.D / p.parts) {
    case 64: return qda::launch_merge<64>(p, rows, s);
    case 128: return qda::launch_merge<128>(p, rows, s);
    case 256: return qda::launch_merge<256>(p, rows, s);
    default: return qda::launch_merge<512>(p, rows, s);
  }
}

extern "C" int qdecode_paged_map(const int32_t* old_len, const int32_t* new_len, int32_t* block_table,
                                 const int32_t* free_pages, int32_t* q_start, int32_t* kv_len, int32_t* slots,
                                 int32_t* positions, int32_t* used, int B, int max_pages, int n_free, int page,
                                 int max_tokens, void* stream) {
  using namespace qda;
  if (!old_len || !new_len || !block_table || !q_start || !kv_len || !used) return QDA_ERR_INVALID;
  if (B < 1 || max_pages < 1 || n_free < 0 || page < 1 || max_tokens < 0) return QDA_ERR_INVALID;
  if ((n_free > 0 && !free_pages) || (max_tokens > 0 && !slots)) return QDA_ERR_INVALID;
  if (kv_len == old_len || kv_len == new_len) return QDA_ERR_INVALID;
  if (!good_page(page) || B > QDA_MAX_B) return QDA_ERR_UNSUPPORTED;
  const void* ptrs[9] = {old_len, new_len, block_table, free_pages, q_start, kv_len, slots, positions, used};
  for (const void* p : ptrs)
    if (off4(p)) return QDA_ERR_ALIGN;
  int sms;
  unsigned int* err;
  const int st = qda_device(&sms, &err);
  if (st != QDA_OK) return st;
  const int grid = (int)std::min<long long>(sms, std::max(1LL, ((long long)max_tokens + kMapThreads - 1) / kMapThreads));
  qda_paged_map_kernel<<<grid, kMapThreads, 0, static_cast<cudaStream_t>(stream)>>>(
      old_len, new_len, block_table, free_pages, q_start, kv_len, slots, positions, used, B, max_pages, n_free,
      page_shift_of(page), max_tokens, err);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? QDA_OK : qda_cuda_fail(e);
}

extern "C" int qdecode_paged_append(const void* k, const void* v, long long k_tstride, long long k_hstride,
                                    long long v_tstride, long long v_hstride, const int32_t* slots, uint32_t* k_packed,
                                    void* k_scales, void* k_biases, uint32_t* v_packed, void* v_scales, void* v_biases,
                                    void* k_held, void* v_held, int T, int Hkv, int num_pages, int page, int D, int GS,
                                    int bits, int dtype, void* stream) {
  using namespace qda;
  if (!k_packed || !k_scales || !k_biases || !v_packed || !v_scales || !v_biases) return QDA_ERR_INVALID;
  if (T < 0 || Hkv < 1 || (k_held == nullptr) != (v_held == nullptr)) return QDA_ERR_INVALID;
  if (T > 0 && (!k || !v || !slots)) return QDA_ERR_INVALID;
  const int cache = dtype & 0xff, src_byte = (dtype >> 8) & 0xff;
  if ((dtype >> 16) != 0 || (cache != QDA_BF16 && cache != QDA_FP16)) return QDA_ERR_INVALID;
  if (src_byte != 0 && src_byte != QDA_BF16 && src_byte != QDA_FP16 && src_byte != QDA_FP32) return QDA_ERR_INVALID;
  int st = check_codec(D, GS, bits);
  if (st == QDA_OK) st = check_pool(num_pages, page);
  if (st != QDA_OK) return st;
  const int src = src_byte == 0 ? cache : src_byte;
  const long long unit = src == QDA_FP32 ? 4 : 8;   // elements in 16 bytes
  const void* ptrs[10] = {k, v, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, k_held, v_held};
  for (const void* p : ptrs)
    if (off16(p)) return QDA_ERR_ALIGN;
  if (off4(slots) || k_tstride % unit || k_hstride % unit || v_tstride % unit || v_hstride % unit) return QDA_ERR_ALIGN;
  // rows are counted in 32 bits (strides of 0 make more of them addressable), CTAs of 256 threads in 31
  if ((long long)T * Hkv > 0xffffff00LL || (long long)T * Hkv * (D / 8) > 0x7fffffffLL * 256) return QDA_ERR_UNSUPPORTED;
  if (T == 0) return QDA_OK;
  AppendParams p;
  std::memset(&p, 0, sizeof(p));
  int sms;
  st = qda_device(&sms, &p.err);
  if (st != QDA_OK) return st;
  p.k = k;
  p.v = v;
  p.kt = k_tstride;
  p.kh = k_hstride;
  p.vt = v_tstride;
  p.vh = v_hstride;
  p.slots = slots;
  p.kp = k_packed;
  p.vp = v_packed;
  p.ks = static_cast<uint16_t*>(k_scales);
  p.kb = static_cast<uint16_t*>(k_biases);
  p.vs = static_cast<uint16_t*>(v_scales);
  p.vb = static_cast<uint16_t*>(v_biases);
  p.k_held = static_cast<uint16_t*>(k_held);
  p.v_held = static_cast<uint16_t*>(v_held);
  p.rows = (uint32_t)((long long)T * Hkv);
  p.Hkv = Hkv;
  p.pool_slots = num_pages * page;
  p.page_shift = page_shift_of(page);
  p.GS = GS;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = bits == 4 ? launch_append_types<4>(p, D, cache == QDA_FP16, src, s)
                                  : launch_append_types<8>(p, D, cache == QDA_FP16, src, s);
  return e == cudaSuccess ? QDA_OK : qda_cuda_fail(e);
}

extern "C" int qdecode_paged_attn_workspace_bytes(int B, int H, int Hkv, int max_q, int D, int GS, int bits,
                                                  size_t* bytes) {
  using namespace qda;
  if (bytes == nullptr || B < 1 || H < 1 || Hkv < 1 || max_q < 1 || H % Hkv != 0) return QDA_ERR_INVALID;
  const int st = check_codec(D, GS, bits);
  if (st != QDA_OK) return st;
  if (B > QDA_MAX_B || H / Hkv > QDA_MAX_NREP) return QDA_ERR_UNSUPPORTED;
  int sms;
  unsigned int* err;
  int got = qda_device(&sms, &err);
  if (got != QDA_OK) return got;
  // a call may state a smaller max_q than this one, either dtype, and ask for the rows' sums or not
  size_t most = 0;
  for (int kind = 0; kind < 4; ++kind) {
    for (long long m : {1LL, split_rows(D) / (H / Hkv), 128LL / (H / Hkv), (long long)max_q}) {
      m = std::max(1LL, std::min(m, (long long)max_q));
      PagedPlan plan;
      got = paged_plan(H / Hkv, m, D, GS, bits, (kind & 1) != 0, (kind & 2) != 0, sms, &plan);
      if (got != QDA_OK) return got;
      most = std::max(most, plan.bytes);
    }
  }
  *bytes = most;
  return QDA_OK;
}

namespace qda {

// Both attention calls; lse == nullptr: not asked for.
static int paged_attn(const void* q, long long q_tstride, long long q_hstride, const uint32_t* k_packed,
                      const void* k_scales, const void* k_biases, const uint32_t* v_packed, const void* v_scales,
                      const void* v_biases, void* out, float* lse, const int32_t* q_start, const int32_t* kv_len,
                      const int32_t* block_table, int total_q, int max_q, int B, int H, int Hkv, int num_pages, int page,
                      int max_pages, int causal, int D, int GS, int bits, int dtype, void* stream) {
  if (!k_packed || !k_scales || !k_biases || !v_packed || !v_scales || !v_biases || !q_start || !kv_len ||
      !block_table)
    return QDA_ERR_INVALID;
  if (total_q < 0 || max_q < 1 || B < 1 || H < 1 || Hkv < 1 || max_pages < 1 || H % Hkv != 0) return QDA_ERR_INVALID;
  if (total_q > 0 && (!q || !out)) return QDA_ERR_INVALID;
  if (dtype != QDA_BF16 && dtype != QDA_FP16) return QDA_ERR_INVALID;
  int st = check_codec(D, GS, bits);
  if (st == QDA_OK) st = check_pool(num_pages, page);
  if (st != QDA_OK) return st;
  if (B > QDA_MAX_B || H / Hkv > QDA_MAX_NREP) return QDA_ERR_UNSUPPORTED;
  if ((long long)num_pages * page * Hkv >= 0xffffffffLL) return QDA_ERR_UNSUPPORTED;   // pool rows are 32-bit
  if ((long long)total_q * (H / Hkv) > 0x7fffff00LL) return QDA_ERR_UNSUPPORTED;       // and so are a sequence's query rows
  const void* ptrs[8] = {q, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, out};
  for (const void* p : ptrs)
    if (off16(p)) return QDA_ERR_ALIGN;
  if (off4(lse) || off4(q_start) || off4(kv_len) || off4(block_table) || q_tstride % 8 || q_hstride % 8) return QDA_ERR_ALIGN;
  if (total_q == 0) return QDA_OK;
  // a row of q may be read after its output is written: by the other part of its values (D = 512), or to be done anew
  long long lo = 0, hi = D;
  for (const long long span : {(total_q - 1) * q_tstride, (H - 1) * q_hstride}) {
    lo += std::min(span, 0LL);
    hi += std::max(span, 0LL);
  }
  const char *qc = static_cast<const char*>(q), *oc = static_cast<const char*>(out);
  const char *qb = qc + 2 * lo, *qe = qc + 2 * hi, *oe = oc + 2LL * total_q * H * D;
  if (qb < oe && oc < qe) return QDA_ERR_INVALID;
  // (the rows' sums are written while other rows' queries are still read, and beside outputs)
  const char *lc = reinterpret_cast<const char*>(lse), *le = lc + 4LL * total_q * H;
  if (lse != nullptr && ((qb < le && lc < qe) || (oc < le && lc < oe))) return QDA_ERR_INVALID;
  QdaPagedParams p;
  std::memset(&p, 0, sizeof(p));
  int sms;
  st = qda_device(&sms, &p.err);
  if (st != QDA_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.kp = k_packed;
  p.ks = static_cast<const uint16_t*>(k_scales);
  p.kb = static_cast<const uint16_t*>(k_biases);
  p.vp = v_packed;
  p.vs = static_cast<const uint16_t*>(v_scales);
  p.vb = static_cast<const uint16_t*>(v_biases);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.table = block_table;
  p.q_tstride = q_tstride;
  p.q_hstride = q_hstride;
  p.total_q = total_q;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.nrep = H / Hkv;
  p.num_pages = num_pages;
  p.page_shift = page_shift_of(page);
  p.max_pages = max_pages;
  p.causal = causal != 0;
  p.D = D;
  p.GS = GS;
  p.NG = D / GS;
  p.W = D * bits / 32;
  p.f16 = dtype == QDA_FP16;
  p.qscale = 1.4426950408889634f / sqrtf((float)D);
  PagedPlan plan;
  st = paged_plan(p.nrep, max_q, D, GS, bits, p.f16 != 0, lse != nullptr, sms, &plan);
  if (st != QDA_OK) return st;
  void* ws = nullptr;
  st = qda_workspace(plan.bytes, &ws);
  if (st != QDA_OK) return st;
  p.part_o = static_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(ws) + plan.o_bytes);
  p.split = reinterpret_cast<QdaPagedSplitTile*>(static_cast<char*>(ws) + plan.o_bytes + plan.ml_bytes);
  p.lse_unit = plan.chunk ? kPcWeightBits : 0.f;
  p.ctas = plan.ctas;
  p.parts = plan.parts;
  p.units = Hkv * plan.parts;
  p.min_keys = plan.min_keys;
#ifdef QDA_BOUNDS_CHECK
  p.stall_block = qda_stall_chunk();
#endif
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = plan.chunk ? chunk_run(&p, D, bits, plan.rows, lse != nullptr, false, s)
                             : split_fn(bits, p.f16 != 0, lse != nullptr)(&p, D, GS, plan.rows, nullptr, s);
  if (e == cudaSuccess) e = qda_launch_paged_merge(p, plan.rows, s);
  if (e == cudaSuccess && plan.chunk && p.causal) e = launch_far(p, bits, sms, s);
  return e == cudaSuccess ? QDA_OK : qda_cuda_fail(e);
}

}  // namespace qda

extern "C" int qdecode_paged_attn(const void* q, long long q_tstride, long long q_hstride, const uint32_t* k_packed,
                                  const void* k_scales, const void* k_biases, const uint32_t* v_packed,
                                  const void* v_scales, const void* v_biases, void* out, const int32_t* q_start,
                                  const int32_t* kv_len, const int32_t* block_table, int total_q, int max_q, int B,
                                  int H, int Hkv, int num_pages, int page, int max_pages, int causal, int D, int GS,
                                  int bits, int dtype, void* stream) {
  return qda::paged_attn(q, q_tstride, q_hstride, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, out, nullptr,
                         q_start, kv_len, block_table, total_q, max_q, B, H, Hkv, num_pages, page, max_pages, causal, D, GS,
                         bits, dtype, stream);
}

extern "C" int qdecode_paged_attn_lse(const void* q, long long q_tstride, long long q_hstride, const uint32_t* k_packed,
                                      const void* k_scales, const void* k_biases, const uint32_t* v_packed,
                                      const void* v_scales, const void* v_biases, void* out, float* lse,
                                      const int32_t* q_start, const int32_t* kv_len, const int32_t* block_table,
                                      int total_q, int max_q, int B, int H, int Hkv, int num_pages, int page,
                                      int max_pages, int causal, int D, int GS, int bits, int dtype, void* stream) {
  if (total_q > 0 && lse == nullptr) return QDA_ERR_INVALID;
  return qda::paged_attn(q, q_tstride, q_hstride, k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, out, lse,
                         q_start, kv_len, block_table, total_q, max_q, B, H, Hkv, num_pages, page, max_pages, causal, D, GS,
                         bits, dtype, stream);
}

extern "C" int qdecode_paged_packed(int op, const int64_t* args) {
  // per op: arguments; the first of the 32-bit ones; those behind them (a double, the stream)
  static const int counts[8] = {15, 24, 27, 0, 28, 27, 28, 28}, first_int[8] = {9, 15, 13, 0, 14, 16, 13, 14};
  static const int behind[8] = {1, 1, 1, 0, 1, 2, 2, 1};
  if (args == nullptr || op < 0 || op > 7 || counts[op] == 0) return QDA_ERR_INVALID;
  int64_t a[28];
  std::memcpy(a, args, sizeof(int64_t) * counts[op]);   // args may have any alignment
  for (int i = first_int[op]; i < counts[op] - behind[op]; ++i)
    if (a[i] < INT32_MIN || a[i] > INT32_MAX) return QDA_ERR_INVALID;
  auto ptr = [&](int i) { return reinterpret_cast<void*>(static_cast<intptr_t>(a[i])); };
  auto i32 = [&](int i) { return static_cast<int32_t*>(ptr(i)); };
  auto u32 = [&](int i) { return static_cast<uint32_t*>(ptr(i)); };
  auto f32 = [&](int i) { return static_cast<float*>(ptr(i)); };
  auto n = [&](int i) { return static_cast<int>(a[i]); };
  auto real = [&](int i) {
    double x;
    std::memcpy(&x, &a[i], sizeof(x));
    return x;
  };
  if (op == 0)
    return qdecode_paged_map(i32(0), i32(1), i32(2), i32(3), i32(4), i32(5), i32(6), i32(7), i32(8), n(9), n(10), n(11),
                             n(12), n(13), ptr(14));
  if (op == 1)
    return qdecode_paged_append(ptr(0), ptr(1), a[2], a[3], a[4], a[5], i32(6), u32(7), ptr(8), ptr(9), u32(10), ptr(11),
                                ptr(12), ptr(13), ptr(14), n(15), n(16), n(17), n(18), n(19), n(20), n(21), n(22), ptr(23));
  if (op == 4)
    return qdecode_paged_attn_lse(ptr(0), a[1], a[2], u32(3), ptr(4), ptr(5), u32(6), ptr(7), ptr(8), ptr(9), f32(10), i32(11),
                                  i32(12), i32(13), n(14), n(15), n(16), n(17), n(18), n(19), n(20), n(21), n(22), n(23),
                                  n(24), n(25), n(26), ptr(27));
  if (op == 5)
    return qdecode_rope(ptr(0), a[1], a[2], ptr(3), a[4], a[5], ptr(6), a[7], a[8], ptr(9), a[10], a[11], i32(12),
                        static_cast<const double*>(ptr(13)), i32(14), i32(15), n(16), n(17), n(18), n(19), n(20), n(21),
                        n(22), n(23), n(24), real(25), ptr(26));
  if (op == 6)
    return qdecode_paged_weights(ptr(0), a[1], a[2], u32(3), ptr(4), ptr(5), f32(6), f32(7), i32(8), i32(9), i32(10), i32(11),
                                 i32(12), n(13), n(14), n(15), n(16), n(17), n(18), n(19), n(20), n(21), n(22), n(23), n(24),
                                 n(25), real(26), ptr(27));
  if (op == 7)
    return qdecode_paged_evict(u32(0), ptr(1), ptr(2), u32(3), ptr(4), ptr(5), f32(6), i32(7), i32(8), i32(9), i32(10), i32(11),
                               i32(12), i32(13), n(14), n(15), n(16), n(17), n(18), n(19), n(20), n(21), n(22), n(23), n(24),
                               n(25), n(26), ptr(27));
  return qdecode_paged_attn(ptr(0), a[1], a[2], u32(3), ptr(4), ptr(5), u32(6), ptr(7), ptr(8), ptr(9), i32(10), i32(11),
                            i32(12), n(13), n(14), n(15), n(16), n(17), n(18), n(19), n(20), n(21), n(22), n(23), n(24),
                            n(25), ptr(26));
}
