// Rotary positions (sm_103a): queries and keys turned by their positions, ahead of the append and the attention.
#include <algorithm>
#include <cmath>
#include <cstdlib>
#include <cstring>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qda_paged_check.h"
#include "qda_ptx.cuh"

namespace qda {

constexpr int kRopeThreads = 256;   // at most
constexpr int kRopeAngles = 2048;   // cosines and sines that a CTA holds: 16 KB
constexpr int kRopeTokens = 8;      // tokens of a CTA, at most

struct RopeParams {
  const void* x[2];         // queries, keys
  void* y[2];
  long long xt[2], xh[2], yt[2], yh[2];   // strides in elements
  const int* positions;     // [T]
  const double* freqs;      // [rot / 2]
  const int* q_start;       // [B + 1], or nullptr
  const int* shift;         // [B]
  int T, B, heads[2], rot, tokens, head_step, inverse;
  int items, rows;          // a row's pairs of vectors; rows that the CTA's threads take at a time
  float scale;
};

template <typename T>
__device__ __forceinline__ float rope_get(T v);
template <>
__device__ __forceinline__ float rope_get(float v) { return v; }
template <>
__device__ __forceinline__ float rope_get(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float rope_get(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T rope_put(float v);
template <>
__device__ __forceinline__ float rope_put(float v) { return v; }
template <>
__device__ __forceinline__ __half rope_put(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 rope_put(float v) { return __float2bfloat16_rn(v); }

template <typename T, int V>
struct alignas(sizeof(T) * V) RopeVec {
  T v[V];
};

// Pair i of a token at position n turns by n f_i: (a, b) -> s (a cos - b sin, b cos + a sin). The angle is kept in turns as a
// 64-bit fraction, n * round(2^64 frac(f / 2 pi)) mod 2^64: whole turns drop out of the integer product exactly, so that a
// position of 2^31 costs no more than 2^-24 of a turn and no argument reduction, where a product in fp32 would be off by 0.06
// radians at 2^20. A CTA takes a few tokens: their cosines and sines go to shared memory, one thread each, and are used by every
// head. A thread has one place in a row, V pairs there (two 16-byte loads: the two halves' values, or 2 V values side by side
// when pairs are interleaved), and walks rows, so that it reads its cosines once a token and divides nowhere; the next two rows
// are on their way while two are turned, the first ones while the angles are computed (a row's place found by division, and loads
// behind the angles, took 22.6 us when this took 18.4). Limited by the latency of memory: 2048 tokens of 40 rows of 128 bf16 take
// 16.4 us where a plain copy of the same 42 MB takes 14.4; 1756 tokens of 24 rows of 512 fp32 30.7 us, 5.6 TB/s; 15934 of 24 rows
// of 256 fp16 with 64 turned 84 us, 4.6 TB/s (loads awaited, HBM at 53 %); 64 tokens 9.6 us, of which the kernel is 5.1.
template <typename T, int V, bool INTER>
__global__ void __launch_bounds__(kRopeThreads) qda_rope_kernel(const __grid_constant__ RopeParams p) {
  __shared__ __align__(16) float2 cs[kRopeAngles];
  __shared__ int s_pos[kRopeTokens];
  __shared__ int s_start[QDA_MAX_B + 1];
  using Vec = RopeVec<T, V>;
  const int tid = threadIdx.x, half = p.rot >> 1;
  const int t0 = blockIdx.x * p.tokens, nt = min(p.tokens, p.T - t0);
  const int x = tid % p.items, y = tid / p.items;
  const int hq = p.heads[0], h0 = blockIdx.y * p.head_step, nh = min(p.head_step, hq + p.heads[1] - h0);
  const int turned = half / V;   // places that turn; those behind them are copied
  const bool turns = x < turned;
  const int d0 = turns && !INTER ? x * V : 2 * x * V, d1 = d0 + (turns && !INTER ? half : V);
  constexpr int U = 2;
  struct Rows {
    Vec a[U], b[U];
    int t, h;                    // token of the CTA and first row of its heads
  };
  Rows now, next;
  auto place = [&](int h, int* w, int* hh) {
    *w = h0 + h >= hq;
    *hh = h0 + h - (*w ? hq : 0);
  };
  auto load = [&](Rows& r, int t, int h) {
    r.t = t;
    r.h = h;
    if (t >= nt) return;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = h + u * p.rows;
      if (i >= nh) continue;
      int w, hh;
      place(i, &w, &hh);
      const T* src = static_cast<const T*>(p.x[w]) + (long long)(t0 + t) * p.xt[w] + hh * p.xh[w];
      r.a[u] = *reinterpret_cast<const Vec*>(src + d0);
      r.b[u] = *reinterpret_cast<const Vec*>(src + d1);
    }
  };
  const bool busy = y < p.rows;
  if (busy) load(now, 0, y);
  else now.t = nt;
  if (p.shift != nullptr) {
    for (int i = tid; i <= p.B; i += blockDim.x) s_start[i] = p.q_start[i];
    __syncthreads();
  }
  for (int i = tid; i < nt; i += blockDim.x) {
    int pos = p.positions[t0 + i];
    if (pos >= 0 && p.shift != nullptr && t0 + i >= s_start[0] && t0 + i < s_start[p.B])
      pos += p.shift[qda_seq_of(s_start, p.B, t0 + i)];
    s_pos[i] = pos;
  }
  __syncthreads();
  for (int i = tid; i < nt * half; i += blockDim.x) {
    const int t = i / half, j = i - t * half;
    const double f = p.freqs[j] * 0.15915494309189533577;
    const unsigned long long step = (unsigned long long)__double2ll_rn((f - rint(f)) * 18446744073709551616.0);
    const int phase = (int)((step * (unsigned long long)(unsigned)s_pos[t]) >> 32);
    float s, c;
    sincospif((float)phase * 4.656612873077392578125e-10f, &s, &c);   // half turns: phase 2^-31
    cs[i] = make_float2(p.scale * c, p.inverse ? -p.scale * s : p.scale * s);
  }
  __syncthreads();
  float2 k[V];
  int held = -1;                 // the token whose cosines are in k
  while (now.t < nt) {
    {
      const int h = now.h + U * p.rows;
      if (h < nh) load(next, now.t, h);
      else load(next, now.t + 1, y);
    }
    if (s_pos[now.t] >= 0) {
      if (turns && held != now.t) {
        held = now.t;
        const float2* c = cs + now.t * half + x * V;
        if constexpr (V >= 2) {
#pragma unroll
          for (int i = 0; i < V; i += 2) {
            const float4 f = *reinterpret_cast<const float4*>(c + i);   // (half is a multiple of V)
            k[i] = make_float2(f.x, f.y);
            k[i + 1] = make_float2(f.z, f.w);
          }
        } else {
          k[0] = c[0];
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int h = now.h + u * p.rows;
        if (h >= nh) continue;
        int w, hh;
        place(h, &w, &hh);
        const long long at = (long long)(t0 + now.t) * p.yt[w] + hh * p.yh[w];
        T* dst = static_cast<T*>(p.y[w]) + at;
        if (!turns && p.x[w] == p.y[w]) continue;   // in place: the rest stands there already
        if (turns) {
          if constexpr (INTER) {
            float v[2 * V];
#pragma unroll
            for (int i = 0; i < V; ++i) {
              v[i] = rope_get(now.a[u].v[i]);
              v[V + i] = rope_get(now.b[u].v[i]);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float e = v[2 * i], o = v[2 * i + 1];
              v[2 * i] = fmaf(e, k[i].x, -o * k[i].y);
              v[2 * i + 1] = fmaf(o, k[i].x, e * k[i].y);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) {
              now.a[u].v[i] = rope_put<T>(v[i]);
              now.b[u].v[i] = rope_put<T>(v[V + i]);
            }
          } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
              const float e = rope_get(now.a[u].v[i]), o = rope_get(now.b[u].v[i]);
              now.a[u].v[i] = rope_put<T>(fmaf(e, k[i].x, -o * k[i].y));
              now.b[u].v[i] = rope_put<T>(fmaf(o, k[i].x, e * k[i].y));
            }
          }
        }
        *reinterpret_cast<Vec*>(dst + d0) = now.a[u];
        *reinterpret_cast<Vec*>(dst + d1) = now.b[u];
      }
    }
    now = next;
  }
}

template <typename T, int V>
cudaError_t rope_run(const RopeParams& p, bool inter, dim3 grid, int threads, cudaStream_t s) {
  if (inter) qda_rope_kernel<T, V, true><<<grid, threads, 0, s>>>(p);
  else qda_rope_kernel<T, V, false><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t rope_pick(const RopeParams& p, int V, bool inter, dim3 grid, int threads, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (V == 8) return rope_run<T, 8>(p, inter, grid, threads, s);
  }
  return V == 4 ? rope_run<T, 4>(p, inter, grid, threads, s)
         : V == 2 ? rope_run<T, 2>(p, inter, grid, threads, s)
                  : rope_run<T, 1>(p, inter, grid, threads, s);
}

// Whether T tokens' rows of `heads` heads and D values of e bytes at a and at b touch the same memory. Exact for rows of one
// buffer that holds a token after the other (views of a fused projection); other spans that cross count as touching.
static bool rope_touch(const void* a, long long at, long long ah, int aheads, const void* b, long long bt, long long bh,
                       int bheads, int T, int D, int e) {
  auto token = [&](long long hs, int heads, __int128* lo, __int128* hi) {
    const __int128 last = (__int128)(heads - 1) * hs;
    *lo = last < 0 ? last * e : 0;
    *hi = ((last > 0 ? last : 0) + D) * e;
  };
  __int128 alo, ahi, blo, bhi;
  token(ah, aheads, &alo, &ahi);
  token(bh, bheads, &blo, &bhi);
  const __int128 pa = (__int128)reinterpret_cast<uintptr_t>(a), pb = (__int128)reinterpret_cast<uintptr_t>(b);
  const __int128 sa = (__int128)(T - 1) * at * e, sb = (__int128)(T - 1) * bt * e;
  if (pa + ahi + (sa > 0 ? sa : 0) <= pb + blo + (sb < 0 ? sb : 0) || pb + bhi + (sb > 0 ? sb : 0) <= pa + alo + (sa < 0 ? sa : 0))
    return false;
  const __int128 step = (__int128)at * e;
  if (at != bt || step <= 0 || ahi - alo > step || bhi - blo > step) return true;
  // a token's rows of b, seen from the token of a whose rows begin at or before them
  const __int128 off = (((pb + blo) - (pa + alo)) % step + step) % step;
  return off < ahi - alo || off + (bhi - blo) > step;
}

// Whether two of the rows that T tokens' `heads` heads have, D values at token * ts + head * hs, touch.
static bool rope_collide(long long ts, int T, long long hs, int heads, int D) {
  const __int128 t = ts < 0 ? -(__int128)ts : ts, h = hs < 0 ? -(__int128)hs : hs;
  if ((T > 1 && t < D) || (heads > 1 && h < D)) return true;
  if (T == 1 || heads == 1 || t >= (heads - 1) * h + D || h >= (T - 1) * t + D) return false;   // one lies within the other
  // dh heads on, the nearest tokens (of either direction: rows differ by dt tokens and dh heads, dt of any sign)
  for (int dh = 1; dh < heads; ++dh) {
    const __int128 off = dh * h, dt = off / t;
    if ((dt < T && off - dt * t < D) || (dt + 1 < T && (dt + 1) * t - off < D)) return true;
  }
  return false;
}

}  // namespace qda

extern "C" int qdecode_rope_freqs(int rot, double base, double factor, double context, double slow, double fast,
                                  double* freqs) {
  if (freqs == nullptr || rot < 2 || rot % 2 != 0) return QDA_ERR_INVALID;
  if (!(base > 0) || !(factor > 0) || !std::isfinite(base) || !std::isfinite(factor)) return QDA_ERR_INVALID;
  if (!(context >= 0) || !std::isfinite(context)) return QDA_ERR_INVALID;
  if (context > 0 && !(slow >= 0 && fast > slow && std::isfinite(fast))) return QDA_ERR_INVALID;
  for (int i = 0; i < rot / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / rot);
    double keep = 0;
    if (context > 0) keep = std::min(1.0, std::max(0.0, (context * f / 6.283185307179586477 - slow) / (fast - slow)));
    freqs[i] = f * (keep + (1 - keep) / factor);
  }
  return QDA_OK;
}

extern "C" int qdecode_rope(const void* q, long long q_tstride, long long q_hstride, const void* k, long long k_tstride,
                            long long k_hstride, void* q_out, long long qo_tstride, long long qo_hstride, void* k_out,
                            long long ko_tstride, long long ko_hstride, const int32_t* positions, const double* freqs,
                            const int32_t* q_start, const int32_t* shift, int T, int B, int H, int Hkv, int D, int rot,
                            int interleaved, int inverse, int dtype, double scale, void* stream) {
  using namespace qda;
  if (T < 0 || H < 0 || Hkv < 0 || H + (long long)Hkv < 1 || D < 1 || rot < 0) return QDA_ERR_INVALID;
  if (dtype != QDA_BF16 && dtype != QDA_FP16 && dtype != QDA_FP32) return QDA_ERR_INVALID;
  if (rot % 2 != 0 || rot < 2 || rot > D || !std::isfinite((float)scale)) return QDA_ERR_INVALID;
  if ((q_start == nullptr) != (shift == nullptr) || (shift != nullptr && B < 1)) return QDA_ERR_INVALID;
  if (T > 0 && ((H > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)) || !positions || !freqs)) return QDA_ERR_INVALID;
  if (D != 64 && D != 128 && D != 256 && D != 512) return QDA_ERR_UNSUPPORTED;
  if (shift != nullptr && B > QDA_MAX_B) return QDA_ERR_UNSUPPORTED;
  if (H + (long long)Hkv > QDA_ROPE_MAX_HEADS || T > 0x7ffff000) return QDA_ERR_UNSUPPORTED;
  const int e = dtype == QDA_FP32 ? 4 : 2;
  const void* ptrs[4] = {H ? q : nullptr, Hkv ? k : nullptr, H ? q_out : nullptr, Hkv ? k_out : nullptr};
  const long long strides[4][2] = {{q_tstride, q_hstride}, {k_tstride, k_hstride}, {qo_tstride, qo_hstride}, {ko_tstride, ko_hstride}};
  const int heads[4] = {H, Hkv, H, Hkv};
  for (int i = 0; i < 4; ++i)
    if (off16(ptrs[i]) || (heads[i] > 0 && (strides[i][0] % (16 / e) || strides[i][1] % (16 / e)))) return QDA_ERR_ALIGN;
  if (off4(positions) || off4(q_start) || off4(shift) || (reinterpret_cast<uintptr_t>(freqs) & 7u)) return QDA_ERR_ALIGN;
  if (T == 0) return QDA_OK;
  for (int i = 2; i < 4; ++i)
    if (heads[i] > 0 && rope_collide(strides[i][0], T, strides[i][1], heads[i], D)) return QDA_ERR_INVALID;
  auto touch = [&](int i, int j) {
    return heads[i] > 0 && heads[j] > 0 &&
           rope_touch(ptrs[i], strides[i][0], strides[i][1], heads[i], ptrs[j], strides[j][0], strides[j][1], heads[j], T, D, e);
  };
  for (int i = 0; i < 2; ++i) {   // an output is its input, or apart from it; and apart from the other tensor
    const bool same = ptrs[i] == ptrs[i + 2] && (T == 1 || strides[i][0] == strides[i + 2][0]) &&
                      (heads[i] == 1 || strides[i][1] == strides[i + 2][1]);   // (one token's stride means nothing)
    if (!same && touch(i, i + 2)) return QDA_ERR_INVALID;
  }
  if (touch(2, 1) || touch(3, 0) || touch(2, 3)) return QDA_ERR_INVALID;
  RopeParams p;
  std::memset(&p, 0, sizeof(p));
  int sms;
  unsigned int* err;
  const int st = qda_device(&sms, &err);
  if (st != QDA_OK) return st;
  for (int i = 0; i < 2; ++i) {
    p.x[i] = ptrs[i];
    p.y[i] = const_cast<void*>(ptrs[i + 2]);
    p.xt[i] = strides[i][0];
    p.xh[i] = strides[i][1];
    p.yt[i] = strides[i + 2][0];
    p.yh[i] = strides[i + 2][1];
    p.heads[i] = heads[i];
  }
  p.positions = positions;
  p.freqs = freqs;
  p.q_start = q_start;
  p.shift = shift;
  p.T = T;
  p.B = B;
  p.rot = rot;
  p.inverse = inverse != 0;
  p.scale = (float)scale;
  int V = 16 / e;
  while ((rot / 2) % V != 0) V /= 2;
  p.items = D / (2 * V);
  const int all = H + Hkv;
  // rows at a time: all heads in as few rounds as 256 threads allow, rounds of equal size
  const int rounds = (int)(((long long)all * p.items + kRopeThreads - 1) / kRopeThreads);
  p.rows = (all + rounds - 1) / rounds;
  // tokens to a CTA: up to eight rounds, fewer where that leaves SMs without CTAs; with few tokens the rounds are shared
  long long tokens = std::max(1, kRopeTokens / rounds);
  tokens = std::min(tokens, std::max(1LL, (long long)T / (6LL * sms)));
  tokens = std::min(tokens, (long long)(kRopeAngles / (rot / 2)));
  const int splits = tokens == 1 ? (int)std::min<long long>(rounds, std::max(1LL, 4LL * sms / T)) : 1;
  p.tokens = (int)tokens;
  p.head_step = (rounds + splits - 1) / splits * p.rows;
  const dim3 grid((unsigned)((T + tokens - 1) / tokens), (unsigned)((all + p.head_step - 1) / p.head_step));
  const int threads = (p.rows * p.items + 31) & ~31;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t ce = dtype == QDA_FP32   ? rope_pick<float>(p, V, interleaved != 0, grid, threads, s)
                         : dtype == QDA_FP16 ? rope_pick<__half>(p, V, interleaved != 0, grid, threads, s)
                                             : rope_pick<__nv_bfloat16>(p, V, interleaved != 0, grid, threads, s);
  return ce == cudaSuccess ? QDA_OK : qda_cuda_fail(ce);
}
