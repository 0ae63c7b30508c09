// Paged attention, plainest form (sm_103a): one warp per (token, query head), lanes along the head dimension, one key at a
// time with an online softmax in fp32. Right for every shape; reads the cache once per query row.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qda_paged.h"
#include "qda_ptx.cuh"

namespace qda {

template <int BITS, int E>
__global__ void __launch_bounds__(128) qda_paged_simple_kernel(const __grid_constant__ QdaPagedParams p) {
  constexpr int PER = 32 / BITS;
  const int lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (long long)p.total_q * p.H) return;
  const int t = (int)(row / p.H), h = (int)(row - (long long)t * p.H), kvh = h / p.nrep;
  if (t >= p.q_start[p.B]) return;
  int lo = 0, hi = p.B;   // the last sequence that starts at or before t is the one that holds it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.q_start[mid] <= t) lo = mid; else hi = mid;
  }
  const int b = lo, L = p.q_start[b + 1] - p.q_start[b];
  const int n_all = max(0, min(p.kv_len[b], (int)min((long long)p.max_pages << p.page_shift, 0x7fffffffLL)));
  const int seen = p.causal ? min(n_all, p.kv_len[b] - L + (t - p.q_start[b]) + 1) : n_all;
  float q[E], o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = half_bits_to_float_rt(p.q[t * p.q_tstride + h * p.q_hstride + lane * E + e], p.f16) * p.qscale;
    o[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int n = 0; n < seen; ++n) {
    const int pg = p.table[(size_t)b * p.max_pages + (n >> p.page_shift)];
    if ((unsigned)pg >= (unsigned)p.num_pages) {
      if (lane == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
      continue;
    }
    const long long r = qda_pool_row(pg, kvh, n & ((1 << p.page_shift) - 1), p.Hkv, p.page_shift);
    const int g = lane * E / p.GS;
    const float ks = half_bits_to_float_rt(p.ks[r * p.NG + g], p.f16), kb = half_bits_to_float_rt(p.kb[r * p.NG + g], p.f16);
    const float vs = half_bits_to_float_rt(p.vs[r * p.NG + g], p.f16), vb = half_bits_to_float_rt(p.vb[r * p.NG + g], p.f16);
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = lane * E + e;
      const uint32_t c = (p.kp[r * p.W + at / PER] >> (BITS * (at % PER))) & ((1u << BITS) - 1);
      s = fmaf(q[e], fmaf(ks, (float)c, kb), s);
    }
#pragma unroll
    for (int off = 16; off >= 1; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
    const float mn = fmaxf(m, s);
    const float a = m == -INFINITY ? 0.f : exp2f(m - mn), w = exp2f(s - mn);
    l = fmaf(l, a, w);
    m = mn;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const int at = lane * E + e;
      const uint32_t c = (p.vp[r * p.W + at / PER] >> (BITS * (at % PER))) & ((1u << BITS) - 1);
      o[e] = fmaf(o[e], a, w * fmaf(vs, (float)c, vb));
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    const float v = o[e] * inv;
    p.out[((size_t)t * p.H + h) * p.D + lane * E + e] =
        p.f16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
  }
}

}  // namespace qda

cudaError_t qda_launch_paged_simple(const QdaPagedParams& p, int bits, cudaStream_t s) {
  const unsigned grid = (unsigned)(((long long)p.total_q * p.H + 3) / 4);
  auto pick = [&](auto k4, auto k8) { bits == 4 ? k4<<<grid, 128, 0, s>>>(p) : k8<<<grid, 128, 0, s>>>(p); };
  switch (p.D) {
    case 64: pick(qda::qda_paged_simple_kernel<4, 2>, qda::qda_paged_simple_kernel<8, 2>); break;
    case 128: pick(qda::qda_paged_simple_kernel<4, 4>, qda::qda_paged_simple_kernel<8, 4>); break;
    case 256: pick(qda::qda_paged_simple_kernel<4, 8>, qda::qda_paged_simple_kernel<8, 8>); break;
    default: pick(qda::qda_paged_simple_kernel<4, 16>, qda::qda_paged_simple_kernel<8, 16>); break;
  }
  return cudaGetLastError();
}
