// Accumulated attention weight over the paged cache (sm_103a): for every key of a sequence under every KV head
//
//     mass[j] = decay * mass[j] + sum over the counted new tokens t and the KV head's query heads h of
//               exp(q[t, h] . k_hat[j] / sqrt(D) - lse[t, h])
//
// from the row sums that the attention call before it has left (lse), so that the keys are read once more and nothing is
// joined across CTAs: the query rows of a key block all meet in one CTA, in a fixed order, and no atomics are needed.
//
// Scores are exact to fp32 as in the split kernel: the codes go into m16n8k16 matrix instructions as fp16 subnormals
// (c 2^-24, one AND for two codes), a query row as fp16 scaled by a power of two to [2^14, 2^15), one accumulator per group,
// and S = sum_g s_g acc_g + b_g sum_g(q) in fp32. Keys are the instruction's 16 rows and query rows its 8 columns, so a
// lane's scale and bias serve both of its columns and a key's sum stays in a quad of lanes.
#pragma once

#include "qda_paged_weights.h"
#include "qda_ptx.cuh"

namespace qda {

constexpr int kPwWarps = 4;
constexpr int kPwKeys = 16 * kPwWarps;   // keys of a block

template <int BITS, int D, int GS, int NT>
struct PwGeom {
  static constexpr int NG = D / GS, W = D * BITS / 32;
  static constexpr int UPL = GS / 32;            // 8-value units of a group that a lane of a quad holds
  static constexpr int WPU = BITS / 4;           // words of such a unit
  static constexpr int UNITS = D / 32;           // units of a row per lane: two k-steps each
  static constexpr int ROWS = 8 * NT;
  static constexpr int MINB = D >= 512 ? 2 : NT == 1 ? 6 : 3;   // resident CTAs per SM
};

__device__ __forceinline__ float pw_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void pw_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A sequence as these kernels see it.
struct PwSeq {
  int first, len;      // its first token's row in q, its new tokens
  int n, base;         // keys; keys before the first new token (negative where the lengths lie)
  int count;           // new tokens that count: the last ones
  int blocks;          // key blocks (none without new tokens)
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
  s.blocks = s.len > 0 ? (int)(((long long)s.n + kPwKeys - 1) / kPwKeys) : 0;
  return s;
}

// Work of a key block beside its query rows (codes, mass, tokens), in query rows.
constexpr int kPwBlockCost = 24;

// Work of the first i key blocks under one KV head. A block's rows are those of the counted tokens that see its first key:
// min(count, n - i keys), all of them until the causal edge.
__device__ __forceinline__ long long pw_prefix(const QdaWeightsParams& p, const PwSeq& s, int i) {
  long long flat = s.n >= s.count ? ((long long)s.n - s.count) / kPwKeys + 1 : 0;
  flat = min(flat, (long long)i);
  const long long rest = i - flat;
  const long long rows = flat * s.count + rest * s.n - kPwKeys * (((long long)i * (i - 1) - flat * (flat - 1)) / 2);
  return (long long)i * kPwBlockCost + rows * p.nrep;
}

template <int BITS, int D, int GS, int NT>
__global__ void __launch_bounds__(kPwWarps * 32, PwGeom<BITS, D, GS, NT>::MINB)
    qda_paged_weights_kernel(const __grid_constant__ QdaWeightsParams p) {
  using G = PwGeom<BITS, D, GS, NT>;
  constexpr int NG = G::NG, UPL = G::UPL, WPU = G::WPU, ROWS = G::ROWS;
  __shared__ long long s_at[QDA_MAX_B + 1];   // sequences on the line of work
  __shared__ long long s_tot[kPwWarps];
  __shared__ uint4 s_q[NT][G::UNITS][32];     // B operands: unit u's two k-steps of a lane
  __shared__ float2 s_sum[NT][NG][4];         // a query row's sums per group, columns of a lane side by side
  __shared__ float2 s_mul[NT][4], s_lse[NT][4];
  __shared__ int2 s_last[NT][4];              // last key that the row sees; -1: no row
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c4 = lane & 3;

  // ---- the line of work: every CTA scans the lengths for itself
  long long carry = 0;
  if (tid == 0) s_at[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPwWarps * 32) {
    const int b = b0 + tid;
    long long v = 0;
    if (b < p.B) {
      const int start = p.q_start[b], end = p.q_start[b + 1], n = p.kv_len[b];
      const PwSeq s = pw_seq(p, start, end, n);
      v = p.Hkv * pw_prefix(p, s, s.blocks);
      if (blockIdx.x == 0 && (start < 0 || end < start || end > p.total_q || (end > start && (n < 0 || n > s.n))))
        atomicOr(p.err, QDA_ERR_BIT_PAGED);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) s_tot[warp] = v;
    __syncthreads();
    long long before = carry;
#pragma unroll
    for (int w = 0; w < kPwWarps; ++w) {
      if (w < warp) before += s_tot[w];
      carry += s_tot[w];
    }
    if (b < p.B) s_at[b + 1] = before + v;
    __syncthreads();
  }
  const long long total = carry, piece = (total + p.ctas - 1) / p.ctas;
  const long long from = min(total, piece * blockIdx.x), to = min(total, from + piece);
  if (from >= to) return;

  // ---- the first block that starts in this CTA's piece
  int b = qda_seq_of(s_at, p.B, from);
  PwSeq s = pw_seq(p, p.q_start[b], p.q_start[b + 1], p.kv_len[b]);
  long long head = pw_prefix(p, s, s.blocks);
  int kvh = (int)((from - s_at[b]) / head);
  long long at = s_at[b] + kvh * head;   // the KV head's place on the line
  int x = 0;
  {
    int hi = s.blocks;   // smallest x with at + prefix(x) >= from
    while (x < hi) {
      const int mid = (x + hi) >> 1;
      if (at + pw_prefix(p, s, mid) >= from) hi = mid; else x = mid + 1;
    }
  }
  const int pmask = (1 << p.page_shift) - 1;
  int have_b = -1, have_kvh = -1, have_row = -1;   // what the operands in shared memory hold
  while (true) {
    if (x >= s.blocks) {   // the next KV head, or sequence
      x = 0;
      at += head;
      if (++kvh >= p.Hkv) {
        kvh = 0;
        do {
          if (++b >= p.B) return;
          s = pw_seq(p, p.q_start[b], p.q_start[b + 1], p.kv_len[b]);
        } while (s.blocks == 0);
        head = pw_prefix(p, s, s.blocks);
      }
    }
    if (at + pw_prefix(p, s, x) >= to) return;

    // ---- this warp's sixteen keys: codes into registers
    const int key0 = x * kPwKeys + warp * 16;
    const int pg = key0 < s.n ? p.table[(size_t)b * p.max_pages + (key0 >> p.page_shift)] : -1;
    const bool there = (unsigned)pg < (unsigned)p.num_pages;
    if (key0 < s.n && !there && lane == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
    const long long row0 = there ? qda_pool_row(pg, kvh, key0 & pmask, p.Hkv, p.page_shift) : 0;
    uint32_t code[2][NG][UPL * WPU];
    float sc[2][NG], bi[2][NG];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const long long row = row0 + r8 + 8 * y;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        const uint32_t* src = p.kp + row * G::W + (g * 4 + c4) * (UPL * WPU);
        if constexpr (UPL * WPU >= 4) {
#pragma unroll
          for (int i = 0; i < UPL * WPU / 4; ++i) {
            const uint4 v = there ? __ldg(reinterpret_cast<const uint4*>(src) + i) : make_uint4(0, 0, 0, 0);
            code[y][g][4 * i] = v.x;
            code[y][g][4 * i + 1] = v.y;
            code[y][g][4 * i + 2] = v.z;
            code[y][g][4 * i + 3] = v.w;
          }
        } else if constexpr (UPL * WPU == 2) {
          const uint2 v = there ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0, 0);
          code[y][g][0] = v.x;
          code[y][g][1] = v.y;
        } else {
          code[y][g][0] = there ? __ldg(src) : 0;
        }
        sc[y][g] = there ? half_bits_to_float_rt(__ldg(p.ks + row * NG + g), p.f16) : 0.f;
        bi[y][g] = there ? half_bits_to_float_rt(__ldg(p.kb + row * NG + g), p.f16) : 0.f;
      }
    }
    float sum[2] = {0.f, 0.f};

    // ---- the query rows, ROWS at a time: those of the counted tokens that see the block's first key
    const int i_lo = max(s.len - s.count, max(x * kPwKeys - s.base, 0));
    const int r_hi = s.len * p.nrep;
    for (int row = i_lo * p.nrep; row < r_hi; row += ROWS) {
      if (have_b != b || have_kvh != kvh || have_row != row) {
        __syncthreads();   // the operands of before are read
        for (int r = warp; r < ROWS; r += kPwWarps) {
          const int tok = (row + r) / p.nrep, h = kvh * p.nrep + row + r - tok * p.nrep;
          const bool real = row + r < r_hi;
          const uint16_t* src = p.q + (long long)(s.first + tok) * p.q_tstride + (long long)h * p.q_hstride;
          constexpr int OCT = D / 8, OPL = (OCT + 31) / 32;   // octets of values, a lane's share
          float v[OPL][8];
          float top = 0.f;
#pragma unroll
          for (int i = 0; i < OPL; ++i) {
            const int o = i * 32 + lane;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (real && o < OCT) w = __ldg(reinterpret_cast<const uint4*>(src) + o);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = half2_bits_to_float2_rt(u[j], p.f16);
              v[i][2 * j] = f.x;
              v[i][2 * j + 1] = f.y;
              top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
          for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
          // 2^e times the row lies in [2^14, 2^15); what is 2^-39 of its largest and less loses bits (next to nothing)
          const int e = top > 0.f && top < INFINITY ? max(-100, min(14 - ilogbf(top), 100)) : 0;
          const float f = exp2f((float)e);
#pragma unroll
          for (int i = 0; i < OPL; ++i) {
            const int o = i * 32 + lane;
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              v[i][j] *= f;
              part += v[i][j];
            }
            // a group's octets lie side by side in lanes
            for (int k = 1; k < GS / 8; k <<= 1) part += __shfl_xor_sync(0xffffffffu, part, k);
            if (o >= OCT) continue;
            const int g = o / (GS / 8), in = o % (GS / 8);
            if (in == 0) reinterpret_cast<float*>(&s_sum[r >> 3][g][(r & 7) >> 1])[r & 1] = part * 5.9604644775390625e-8f;
            constexpr float HI = BITS == 4 ? 0.0625f : 1.f;   // (odd codes of a 4-bit word stand four bits higher)
            auto h2 = [](float a, float c) {
              const __half2 h = __floats2half2_rn(a, c);
              return *reinterpret_cast<const uint32_t*>(&h);
            };
            uint4 w;
            if constexpr (BITS == 4) {
              w = make_uint4(h2(v[i][0], v[i][4]), h2(v[i][1] * HI, v[i][5] * HI), h2(v[i][2], v[i][6]),
                             h2(v[i][3] * HI, v[i][7] * HI));
            } else {
              w = make_uint4(h2(v[i][0], v[i][2]), h2(v[i][1], v[i][3]), h2(v[i][4], v[i][6]), h2(v[i][5], v[i][7]));
            }
            s_q[r >> 3][g * UPL + in % UPL][(r & 7) * 4 + in / UPL] = w;
          }
          if (lane == 0) {
            const int nt = r >> 3, c = (r & 7) >> 1;
            reinterpret_cast<float*>(&s_mul[nt][c])[r & 1] = p.qscale * exp2f((float)(24 - e));
            reinterpret_cast<float*>(&s_lse[nt][c])[r & 1] =
                real ? p.lse[(long long)(s.first + tok) * p.H + h] * 1.4426950408889634f : 0.f;
            reinterpret_cast<int*>(&s_last[nt][c])[r & 1] = real ? s.base + tok : -1;
          }
        }
        __syncthreads();
        have_b = b;
        have_kvh = kvh;
        have_row = row;
      }
      if (!there) continue;
      float S[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) S[nt][0] = S[nt][1] = S[nt][2] = S[nt][3] = 0.f;
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        float acc[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
        for (int u = 0; u < UPL; ++u) {
          uint32_t a[8];   // two k-steps
          if constexpr (BITS == 4) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t w = code[y][g][u], z = w >> 8;
              a[y] = w & 0x000F000Fu;
              a[2 + y] = w & 0x00F000F0u;
              a[4 + y] = z & 0x000F000Fu;
              a[6 + y] = z & 0x00F000F0u;
            }
          } else {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const uint32_t w = code[y][g][2 * u + j];
                a[4 * j + y] = w & 0x00FF00FFu;
                a[4 * j + 2 + y] = (w >> 8) & 0x00FF00FFu;
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint4 bq = s_q[nt][g * UPL + u][lane];
            pw_mma(acc[nt], a[0], a[1], a[2], a[3], bq.x, bq.y);
            pw_mma(acc[nt], a[4], a[5], a[6], a[7], bq.z, bq.w);
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float2 qs = s_sum[nt][g][c4];
          S[nt][0] = fmaf(bi[0][g], qs.x, fmaf(sc[0][g], acc[nt][0], S[nt][0]));
          S[nt][1] = fmaf(bi[0][g], qs.y, fmaf(sc[0][g], acc[nt][1], S[nt][1]));
          S[nt][2] = fmaf(bi[1][g], qs.x, fmaf(sc[1][g], acc[nt][2], S[nt][2]));
          S[nt][3] = fmaf(bi[1][g], qs.y, fmaf(sc[1][g], acc[nt][3], S[nt][3]));
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float2 mul = s_mul[nt][c4], ls = s_lse[nt][c4];
        const int2 last = s_last[nt][c4];
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int key = key0 + r8 + 8 * y;
          const float e0 = pw_ex2(fmaf(S[nt][2 * y], mul.x, -ls.x)), e1 = pw_ex2(fmaf(S[nt][2 * y + 1], mul.y, -ls.y));
          sum[y] += key <= last.x ? e0 : 0.f;
          sum[y] += key <= last.y ? e1 : 0.f;
        }
      }
    }
    // ---- a key's sum over the quad's columns, and its new mass
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
      sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
    }
    if (there && c4 < 2) {
      const int key = key0 + r8 + 8 * c4;
      const long long row = row0 + r8 + 8 * c4;
      if (key < s.n) {
        const float add = c4 == 0 ? sum[0] : sum[1];
        if (key < s.base) {
          p.mass[row] = fmaf(p.decay, p.mass[row], add);
        } else {
          p.mass[row] = add;
          p.token[row] = key + (p.shift != nullptr ? p.shift[b] : 0);
        }
      }
    }
    ++x;
  }
}

template <int BITS, int D, int GS, int NT>
cudaError_t pw_run(const QdaWeightsParams* p, int* ctas_per_sm, cudaStream_t s) {
  auto kern = qda_paged_weights_kernel<BITS, D, GS, NT>;
  if (ctas_per_sm != nullptr) return cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, kern, kPwWarps * 32, 0);
  kern<<<p->ctas, kPwWarps * 32, 0, s>>>(*p);
  return cudaGetLastError();
}

template <int BITS>
cudaError_t pw_pick(const QdaWeightsParams* p, int D, int GS, int rows, int* occ, cudaStream_t s) {
#define QDA_PW(d, gs)                                                 \
  if (D == d && GS == gs) {                                           \
    if (rows > 8) return pw_run<BITS, d, gs, 4>(p, occ, s);           \
    return pw_run<BITS, d, gs, 1>(p, occ, s);                         \
  }
  QDA_PW(64, 32) QDA_PW(64, 64)
  QDA_PW(128, 32) QDA_PW(128, 64) QDA_PW(128, 128)
  QDA_PW(256, 32) QDA_PW(256, 64) QDA_PW(256, 128)
  QDA_PW(512, 32) QDA_PW(512, 64) QDA_PW(512, 128)
#undef QDA_PW
  return cudaErrorInvalidValue;
}

}  // namespace qda
