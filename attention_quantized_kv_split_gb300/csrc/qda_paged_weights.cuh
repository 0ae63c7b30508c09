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
constexpr int kPwCost = 24;              // work of a block beside its query rows (codes, mass, tokens), in query rows

template <int BITS, int D, int GS, int NT>
struct PwGeom {
  static constexpr int NG = D / GS, W = D * BITS / 32;
  static constexpr int UPL = GS / 32;            // 8-value units of a group that a lane of a quad holds
  static constexpr int WPU = BITS / 4;           // words of such a unit
  static constexpr int UNITS = D / 32;           // units of a row per lane: two k-steps each
  static constexpr int ROWS = 8 * NT;
  static constexpr int RB = W * 4, CPR = RB / 16;   // bytes and 16-byte chunks of a row of codes
  // a warp's stage: sixteen keys' codes, scales, biases, masses
  static constexpr int SC = 16 * NG * 2, STAGE = 16 * RB + 2 * SC + 64;
  static constexpr int STAGES = STAGE <= 3000 ? 4 : STAGE <= 6000 ? 3 : 2;
  static constexpr int RING = kPwWarps * STAGES * STAGE;
  static constexpr int OPS = NT * UNITS * 32 * 16;
  static constexpr int SMEM = RING + OPS;
  static constexpr int MINB = D >= 512 ? 2 : NT == 1 ? (D == 256 ? 4 : 6) : 3;   // resident CTAs per SM
};

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
__device__ __forceinline__ void pw_copy4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void pw_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void pw_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// BYTES (a power of two, up to 32) from shared memory into words.
template <int BYTES, int N>
__device__ __forceinline__ void pw_lds(const char* p, uint32_t (&v)[N]) {
  if constexpr (BYTES >= 16) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const uint4 x = *reinterpret_cast<const uint4*>(p + 16 * i);
      v[4 * i] = x.x;
      v[4 * i + 1] = x.y;
      v[4 * i + 2] = x.z;
      v[4 * i + 3] = x.w;
    }
  } else if constexpr (BYTES == 8) {
    const uint2 x = *reinterpret_cast<const uint2*>(p);
    v[0] = x.x;
    v[1] = x.y;
  } else if constexpr (BYTES == 4) {
    v[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    v[0] = *reinterpret_cast<const uint16_t*>(p);
  }
}

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

template <int NT, int NG>
struct PwRows {
  float2 sum[NT][NG][4];         // a query row's sums per group, columns of a lane side by side
  float2 mul[NT][4], lse[NT][4];
  int2 last[NT][4];              // last key that the row sees; -1: no row
};

// The CTA: operands and scalars of query rows row .. row + ROWS - 1 of sequence s under KV head kvh.
template <int BITS, int D, int GS, int NT>
__device__ __forceinline__ void pw_rows(const QdaWeightsParams& p, const PwSeq& s, int kvh, int row, uint4* ops,
                                        PwRows<NT, D / GS>& sh) {
  using G = PwGeom<BITS, D, GS, NT>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int r = warp; r < G::ROWS; r += kPwWarps) {
    const int tok = (row + r) / p.nrep, h = kvh * p.nrep + row + r - tok * p.nrep;
    const bool real = row + r < s.len * p.nrep;
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
#pragma unroll
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
#pragma unroll
      for (int k = 1; k < GS / 8; k <<= 1) part += __shfl_xor_sync(0xffffffffu, part, k);
      if (o >= OCT) continue;
      const int g = o / (GS / 8), in = o % (GS / 8);
      if (in == 0) reinterpret_cast<float*>(&sh.sum[r >> 3][g][(r & 7) >> 1])[r & 1] = part * 5.9604644775390625e-8f;
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
      ops[((r >> 3) * G::UNITS + g * G::UPL + in % G::UPL) * 32 + (r & 7) * 4 + in / G::UPL] = w;
    }
    if (lane == 0) {
      const int nt = r >> 3, c = (r & 7) >> 1;
      reinterpret_cast<float*>(&sh.mul[nt][c])[r & 1] = p.qscale * exp2f((float)(24 - e));
      reinterpret_cast<float*>(&sh.lse[nt][c])[r & 1] =
          real ? p.lse[(long long)(s.first + tok) * p.H + h] * 1.4426950408889634f : 0.f;
      reinterpret_cast<int*>(&sh.last[nt][c])[r & 1] = real ? s.base + tok : -1;
    }
  }
}

// Few query rows: every warp streams tiles of sixteen keys through a ring of its own in shared memory, asynchronous copies
// three tiles ahead, and the query rows of the CTA's (sequence, KV head) stay in shared memory as operands. With more rows
// than ROWS the CTA's warps take a block of tiles together and the rows pass by, ROWS at a time.
template <int BITS, int D, int GS, int NT>
__global__ void __launch_bounds__(kPwWarps * 32, PwGeom<BITS, D, GS, NT>::MINB)
    qda_paged_weights_kernel(const __grid_constant__ QdaWeightsParams p) {
  using G = PwGeom<BITS, D, GS, NT>;
  constexpr int NG = G::NG, UPL = G::UPL, WPU = G::WPU, ROWS = G::ROWS, S = G::STAGES;
  extern __shared__ __align__(16) char smem[];
  __shared__ long long s_at[QDA_MAX_B + 1];   // sequences on the line of work
  __shared__ long long s_tot[kPwWarps];
  __shared__ PwRows<NT, NG> rows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c4 = lane & 3;
  char* const ring = smem + warp * (S * G::STAGE);
  uint4* const ops = reinterpret_cast<uint4*>(smem + G::RING);

  // ---- the line of work: every CTA scans the lengths for itself
  auto work = [&](const PwSeq& s, int i) {
    return pw_prefix<kPwKeys>(p, s, i, kPwCost + (long long)s.count * p.nrep, kPwCost);
  };
  long long carry = 0;
  if (tid == 0) s_at[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPwWarps * 32) {
    const int b = b0 + tid;
    long long v = 0;
    if (b < p.B) {
      const int start = p.q_start[b], end = p.q_start[b + 1], n = p.kv_len[b];
      const PwSeq s = pw_seq(p, start, end, n);
      v = p.Hkv * work(s, pw_blocks<kPwKeys>(s));
      if (blockIdx.x == 0 && pw_bad(p, start, end, n, s)) atomicOr(p.err, QDA_ERR_BIT_PAGED);
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

  // ---- the CTA's piece, a (sequence, KV head) at a time: the blocks that start in it
  int b = qda_seq_of(s_at, p.B, from);
  PwSeq s = pw_seq(p, b);
  int blocks = pw_blocks<kPwKeys>(s);
  long long head = work(s, blocks);
  int kvh = (int)((from - s_at[b]) / head);
  long long at = s_at[b] + kvh * head;   // the KV head's place on the line
  auto block_at = [&](long long x) { return pw_block_at(blocks, x, [&](int i) { return at + work(s, i); }); };
  const int pmask = (1 << p.page_shift) - 1;
  int x0 = block_at(from);
  while (true) {
    const int x1 = at + head <= to ? blocks : block_at(to);
    if (x0 < x1) {
      const int* tab = p.table + (size_t)b * p.max_pages;
      const int t1 = min(x1 * kPwWarps, (s.n + 15) >> 4);
      auto page_of = [&](int t) { return t < t1 ? __ldg(tab + (t * 16 >> p.page_shift)) : -1; };
      auto row_of = [&](int t, int pg) { return qda_pool_row(pg, kvh, (t * 16) & pmask, p.Hkv, p.page_shift); };
      // sixteen keys on their way into a stage (a page outside the pool: nothing is read)
      auto fetch = [&](int t, int pg, int st) {
        if (t < t1 && (unsigned)pg < (unsigned)p.num_pages) {
          const long long row = row_of(t, pg);
          const uint32_t dst = smem_addr(ring + st * G::STAGE);
          const char* src = reinterpret_cast<const char*>(p.kp + row * G::W);
#pragma unroll
          for (int i = 0; i < (16 * G::CPR + 31) / 32; ++i) {
            const int c = i * 32 + lane;
            if (16 * G::CPR >= 32 || c < 16 * G::CPR)
              pw_copy16(dst + pw_chunk<G::RB>(c / G::CPR, c % G::CPR), src + 16 * c);
          }
          constexpr int CS = G::SC / 16;   // chunks of the scales, and of the biases
          if (lane < 2 * CS)
            pw_copy16(dst + 16 * G::RB + 16 * lane,
                      reinterpret_cast<const char*>((lane < CS ? p.ks : p.kb) + row * NG) + 16 * (lane < CS ? lane : lane - CS));
          if (2 * CS > 32 && lane + 32 < 2 * CS)
            pw_copy16(dst + 16 * G::RB + 16 * (lane + 32), reinterpret_cast<const char*>(p.kb + row * NG) + 16 * (lane + 32 - CS));
          if (lane < 16) pw_copy4(dst + 16 * G::RB + 2 * G::SC + 4 * lane, p.mass + row + lane);
        }
        pw_commit();
      };
      const int first = (s.len - s.count) * p.nrep, r_hi = s.len * p.nrep;
      int t = x0 * kPwWarps + warp;
      int pages[S];   // of the tiles in flight, and the next one's
#pragma unroll
      for (int i = 0; i < S; ++i) pages[i] = page_of(t + i * kPwWarps);
#pragma unroll
      for (int i = 0; i < S - 1; ++i) fetch(t + i * kPwWarps, pages[i], i);
      const bool many = r_hi - first > ROWS;
      if (!many) {
        __syncthreads();   // the operands of before are read
        pw_rows<BITS, D, GS, NT>(p, s, kvh, first, ops, rows);
        __syncthreads();
      }
      int st = 0;
      for (int step = x0; step < x1; ++step, t += kPwWarps) {
        {   // the stage before this one's is free again
          const int far = t + (S - 1) * kPwWarps;
          fetch(far, pages[S - 1], st == 0 ? S - 1 : st - 1);
        }
        pw_wait<S - 1>();
        __syncwarp();
        const int pg = pages[0];
        const bool there = t < t1 && (unsigned)pg < (unsigned)p.num_pages;
        if (t < t1 && !there && lane == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
#pragma unroll
        for (int i = 0; i < S - 1; ++i) pages[i] = pages[i + 1];
        pages[S - 1] = page_of(t + S * kPwWarps);
        const char* const stage = ring + st * G::STAGE;
        st = st == S - 1 ? 0 : st + 1;
        const int key0 = t * 16;
        float sum[2] = {0.f, 0.f};
        auto tile = [&]() {
          float sc[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) sc[nt][0] = sc[nt][1] = sc[nt][2] = sc[nt][3] = 0.f;
          uint32_t sw[2][(NG + 1) / 2], bw[2][(NG + 1) / 2];
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            pw_lds<NG * 2>(stage + 16 * G::RB + (r8 + 8 * y) * NG * 2, sw[y]);
            pw_lds<NG * 2>(stage + 16 * G::RB + G::SC + (r8 + 8 * y) * NG * 2, bw[y]);
          }
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            constexpr int LB = UPL * WPU * 4;   // a lane's bytes of a group
            uint32_t code[2][UPL * WPU];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              if constexpr (LB <= 16) {
                const int off = g * 4 * LB + c4 * LB;
                pw_lds<LB>(stage + pw_chunk<G::RB>(r8 + 8 * y, off >> 4) + (off & 15), code[y]);
              } else {
#pragma unroll
                for (int i = 0; i < LB / 16; ++i) {
                  const uint4 v = *reinterpret_cast<const uint4*>(
                      stage + pw_chunk<G::RB>(r8 + 8 * y, (g * 4 * LB + c4 * LB) / 16 + i));
                  code[y][4 * i] = v.x;
                  code[y][4 * i + 1] = v.y;
                  code[y][4 * i + 2] = v.z;
                  code[y][4 * i + 3] = v.w;
                }
              }
            }
            float acc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) acc[nt][0] = acc[nt][1] = acc[nt][2] = acc[nt][3] = 0.f;
#pragma unroll
            for (int u = 0; u < UPL; ++u) {
              uint32_t a[8];   // two k-steps
              if constexpr (BITS == 4) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  const uint32_t w = code[y][u], z = w >> 8;
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
                    const uint32_t w = code[y][2 * u + j];
                    a[4 * j + y] = w & 0x00FF00FFu;
                    a[4 * j + 2 + y] = (w >> 8) & 0x00FF00FFu;
                  }
                }
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint4 bq = ops[(nt * G::UNITS + g * UPL + u) * 32 + lane];
                pw_mma(acc[nt], a[0], a[1], a[2], a[3], bq.x, bq.y);
                pw_mma(acc[nt], a[4], a[5], a[6], a[7], bq.z, bq.w);
              }
            }
            const float s0 = half_bits_to_float_rt((sw[0][g / 2] >> (16 * (g & 1))) & 0xffffu, p.f16);
            const float s1 = half_bits_to_float_rt((sw[1][g / 2] >> (16 * (g & 1))) & 0xffffu, p.f16);
            const float b0 = half_bits_to_float_rt((bw[0][g / 2] >> (16 * (g & 1))) & 0xffffu, p.f16);
            const float b1 = half_bits_to_float_rt((bw[1][g / 2] >> (16 * (g & 1))) & 0xffffu, p.f16);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float2 qs = rows.sum[nt][g][c4];
              sc[nt][0] = fmaf(b0, qs.x, fmaf(s0, acc[nt][0], sc[nt][0]));
              sc[nt][1] = fmaf(b0, qs.y, fmaf(s0, acc[nt][1], sc[nt][1]));
              sc[nt][2] = fmaf(b1, qs.x, fmaf(s1, acc[nt][2], sc[nt][2]));
              sc[nt][3] = fmaf(b1, qs.y, fmaf(s1, acc[nt][3], sc[nt][3]));
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 mul = rows.mul[nt][c4], ls = rows.lse[nt][c4];
            const int2 last = rows.last[nt][c4];
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const int key = key0 + r8 + 8 * y;
              const float e0 = pw_ex2(fmaf(sc[nt][2 * y], mul.x, -ls.x)), e1 = pw_ex2(fmaf(sc[nt][2 * y + 1], mul.y, -ls.y));
              sum[y] += key <= last.x ? e0 : 0.f;
              sum[y] += key <= last.y ? e1 : 0.f;
            }
          }
        };
        // the counted tokens that see the block's first key
        int row = many ? max(first, max(step * kPwKeys - s.base, 0) * p.nrep) : first;
        do {
          if (many) {
            __syncthreads();   // the operands of before are read
            pw_rows<BITS, D, GS, NT>(p, s, kvh, row, ops, rows);
            __syncthreads();
          }
          if (there) tile();
          row += ROWS;
        } while (row < r_hi);
        // ---- a key's sum over the quad's columns, and its new mass
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
          sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
        }
        const int key = key0 + r8 + 8 * c4;
        if (there && c4 < 2 && key < s.n) {
          const long long row = row_of(t, pg) + r8 + 8 * c4;
          const float add = c4 == 0 ? sum[0] : sum[1];
          if (key < s.base) {
            const float old = *reinterpret_cast<const float*>(stage + 16 * G::RB + 2 * G::SC + 4 * (r8 + 8 * c4));
            p.mass[row] = fmaf(p.decay, old, add);
          } else {
            p.mass[row] = add;
            p.token[row] = key + (p.shift != nullptr ? p.shift[b] : 0);
          }
        }
        __syncwarp();   // the stage is read
      }
      pw_wait<0>();
      __syncwarp();
    }
    // ---- the next KV head, or sequence
    x0 = 0;
    at += head;
    if (++kvh >= p.Hkv) {
      kvh = 0;
      do {
        if (++b >= p.B) return;
        s = pw_seq(p, b);
        blocks = pw_blocks<kPwKeys>(s);
      } while (blocks == 0);
      head = work(s, blocks);
    }
    if (at >= to) return;
  }
}

template <int BITS, int D, int GS, int NT>
cudaError_t pw_run(const QdaWeightsParams* p, int* ctas_per_sm, cudaStream_t s) {
  using G = PwGeom<BITS, D, GS, NT>;
  auto kern = qda_paged_weights_kernel<BITS, D, GS, NT>;
  if (ctas_per_sm != nullptr) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, kern, kPwWarps * 32, G::SMEM);
    return e;
  }
  kern<<<p->ctas, kPwWarps * 32, G::SMEM, s>>>(*p);
  return cudaGetLastError();
}

template <int BITS>
cudaError_t pw_pick(const QdaWeightsParams* p, int D, int GS, int rows, int* occ, cudaStream_t s) {
#define QDA_PW(d, gs)                                                          \
  if (D == d && GS == gs) {                                                    \
    if (rows > 8) return pw_run<BITS, d, gs, 4>(p, occ, s);                    \
    return pw_run<BITS, d, gs, 1>(p, occ, s);                                  \
  }
  QDA_PW(64, 32) QDA_PW(64, 64)
  QDA_PW(128, 32) QDA_PW(128, 64) QDA_PW(128, 128)
  QDA_PW(256, 32) QDA_PW(256, 64) QDA_PW(256, 128)
  QDA_PW(512, 32) QDA_PW(512, 64) QDA_PW(512, 128)
#undef QDA_PW
  return cudaErrorInvalidValue;
}

}  // namespace qda
