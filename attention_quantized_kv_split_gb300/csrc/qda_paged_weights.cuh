// Accumulated attention weight over the paged cache (sm_103a): for every key of a sequence under every KV head
//
//     mass[j] = decay * mass[j] + sum over the counted new tokens t and the KV head's query heads h of
//               exp(q[t, h] . k_hat[j] / sqrt(D) - lse[t, h])
//
// from the row sums that the attention call before it has left (lse), so that the keys are read once more and nothing is
// joined across CTAs: the query rows of a key block all meet in one CTA, in a fixed order, and no atomics are needed.
//
// Keys enter as they are, as in the split kernel: the codes go into m16n8k16 matrix instructions as fp16 subnormals
// (c 2^-24, one AND for two codes), a query row as fp16 scaled by a power of two to [2^14, 2^15), one accumulator per group,
// and S = sum_g s_g acc_g + b_g sum_g(q) in fp32. A query's value is off by 2^-39 of its row's largest at most, and by 2^-35 in the
// odd dimensions of 4-bit keys, where it is held as a sixteenth. Keys are the instruction's 16 rows and query rows its 8 columns, so a
// lane's scale and bias serve both of its columns and a key's sum stays in a quad of lanes.
#pragma once

#include "qda_paged_weights.h"
#include "qda_ptx.cuh"

namespace qda {

constexpr int kPwWarps = 4;
constexpr int kPwCost = 24;    // work of 64 keys beside their query rows (codes, mass, tokens), in query rows

template <int BITS, int D, int GS, int NT>
struct PwGeom {
  static constexpr int NG = D / GS, W = D * BITS / 32;
  static constexpr int UPL = GS / 32;            // 8-value units of a group that a lane of a quad holds
  static constexpr int WPU = BITS / 4;           // words of such a unit
  static constexpr int UNITS = D / 32;           // units of a row per lane: two k-steps each
  static constexpr int ROWS = 8 * NT;
  static constexpr int T = NT <= 2 ? 2 : 1;      // sixteens of keys that a warp takes at a time
  static constexpr int KEYS = 16 * T * kPwWarps; // keys of a block
  static constexpr int RB = W * 4, CPR = RB / 16;   // bytes and 16-byte chunks of a row of codes
  // a warp's stage: its keys' codes, scales, biases, masses, sixteen by sixteen
  static constexpr int SC = 16 * NG * 2, SUB = 16 * RB + 2 * SC + 64, STAGE = T * SUB;
  static constexpr int STAGES = STAGE <= 3000 ? 4 : STAGE <= 6000 ? 3 : 2;
  static constexpr int RING = kPwWarps * STAGES * STAGE;
  static constexpr int OPS = NT * UNITS * 32 * 16;
  static constexpr int SMEM = RING + OPS;
  static constexpr int MINB = D >= 512 ? 2 : NT == 1 ? (D == 256 ? 4 : 5) : NT == 2 && D <= 128 ? 4 : 3;   // resident CTAs per SM
  static constexpr int COST = kPwCost * KEYS / 64;
};

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

// Half word i of words of 16-bit values, as a float.
template <bool F16, int N>
__device__ __forceinline__ float pw_half(const uint32_t (&w)[N], int i) {
  if constexpr (F16) {
    const __half2 h = *reinterpret_cast<const __half2*>(&w[i >> 1]);
    return i & 1 ? __high2float(h) : __low2float(h);
  } else {
    return __uint_as_float(i & 1 ? w[i >> 1] & 0xffff0000u : w[i >> 1] << 16);
  }
}

__device__ __forceinline__ float pw_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// c (+)= a b; without `more` the sums start from 0
__device__ __forceinline__ void pw_mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1, bool more) {
  if (more)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// ceil(total / n): 64-bit division only where it is needed.
__device__ __forceinline__ long long pw_share(long long total, int n) {
  if (total <= 0x7fffffffLL - n) return ((uint32_t)total + (uint32_t)n - 1) / (uint32_t)n;
  return (total + n - 1) / n;
}

template <int NT, int NG>
struct PwRows {
  float2 sum[NT][NG][4];         // a query row's sums per group, columns of a lane side by side
  float2 mul[NT][4], lse[NT][4];
  int2 last[NT][4];              // last key that the row sees; -1: no row
};

// The CTA: operands and scalars of query rows row .. row + ROWS - 1 of sequence s under KV head kvh.
template <int BITS, int D, int GS, int NT, bool F16>
__device__ __forceinline__ void pw_rows(const QdaWeightsParams& p, const PwSeq& s, int kvh, int row, uint4* ops,
                                        PwRows<NT, D / GS>& sh) {
  using G = PwGeom<BITS, D, GS, NT>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int OCT = D / 8, OPL = (OCT + 31) / 32;   // octets of values, a lane's share
  constexpr int RW = G::ROWS / kPwWarps, AT_ONCE = NT == 1 ? 1 : RW < 4 ? RW : 4;   // a warp's rows; those on their way together
#pragma unroll 1
  for (int r0 = 0; r0 < RW; r0 += AT_ONCE) {
    uint4 raw[AT_ONCE][OPL];
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int at = row + warp + (r0 + k) * kPwWarps, tok = at / p.nrep, h = kvh * p.nrep + at - tok * p.nrep;
      const uint16_t* src = p.q + (long long)(s.first + tok) * p.q_tstride + (long long)h * p.q_hstride;
#pragma unroll
      for (int i = 0; i < OPL; ++i) {
        raw[k][i] = make_uint4(0, 0, 0, 0);
        if (at < s.len * p.nrep && i * 32 + lane < OCT) raw[k][i] = __ldg(reinterpret_cast<const uint4*>(src) + i * 32 + lane);
      }
    }
#pragma unroll
    for (int k = 0; k < AT_ONCE; ++k) {
      const int r = warp + (r0 + k) * kPwWarps;
      const int tok = (row + r) / p.nrep, h = kvh * p.nrep + row + r - tok * p.nrep;
      const bool real = row + r < s.len * p.nrep;
      float v[OPL][8];
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < OPL; ++i) {
        const uint32_t u[4] = {raw[k][i].x, raw[k][i].y, raw[k][i].z, raw[k][i].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = pw_half<F16>(u, j);
          top = fmaxf(top, fabsf(v[i][j]));
        }
      }
#pragma unroll
      for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      // 2^e times the row lies in [2^14, 2^15): steps of 2^-24 below 2^-14
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
            real ? p.lse[(long long)(s.first + tok) * p.H + h] * 1.4426950408889634f : INFINITY;   // (no row weighs nothing)
        reinterpret_cast<int*>(&sh.last[nt][c])[r & 1] = real ? s.base + tok : -1;
      }
    }
  }
}

// Few query rows: every warp streams tiles of 16 T keys through a ring of its own in shared memory, asynchronous copies tiles
// ahead, and the query rows of the CTA's (sequence, KV head) stay in shared memory as operands. With more rows than ROWS the
// CTA's warps take a block of tiles together and the rows pass by, ROWS at a time.
//
// Neither unit is full: instruction issue 62 % of the slots at 20 warps per SM, HBM 44 %. One token of 64 sequences of 700 to
// 8200 keys, 4-bit, D 128, takes 51 us, 3.5 TB/s of codes, scales, biases and masses; 133 us with loads straight to registers,
// 72 with the ring, 55 with two sixteens of keys at a time, so that what a tile costs beside its products is paid half as
// often. One token over 131072 keys at D 256 takes 27 us (3.2 TB/s; starts and first loads are a third), over 512 keys 10
// (latency). Sixteen rows over four sequences of 8192 keys (8 KV heads, D 128, 4-bit) take 18.5 us with NT = 2 and 24.6 with NT
// = 4.
template <int BITS, int D, int GS, int NT, bool F16>
__global__ void __launch_bounds__(kPwWarps * 32, PwGeom<BITS, D, GS, NT>::MINB)
    qda_paged_weights_kernel(const __grid_constant__ QdaWeightsParams p) {
  using G = PwGeom<BITS, D, GS, NT>;
  constexpr int NG = G::NG, UPL = G::UPL, WPU = G::WPU, ROWS = G::ROWS, S = G::STAGES, T = G::T, RB = G::RB;
  extern __shared__ __align__(16) char smem[];
  __shared__ long long s_at[QDA_MAX_B + 1];   // sequences on the line of work
  __shared__ long long s_tot[kPwWarps];
  __shared__ PwRows<NT, NG> rows;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c4 = lane & 3;
  char* const ring = smem + warp * (S * G::STAGE);
  uint4* const ops = reinterpret_cast<uint4*>(smem + G::RING);

  // ---- the line of work: every CTA scans the lengths for itself
  auto work = [&](const PwSeq& s, int i) {
    return pw_prefix<G::KEYS>(p, s, i, G::COST + (long long)s.count * p.nrep, G::COST);
  };
  long long carry = 0;
  if (tid == 0) s_at[0] = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPwWarps * 32) {
    const int b = b0 + tid;
    long long v = 0;
    if (b < p.B) {
      const int start = p.q_start[b], end = p.q_start[b + 1], n = p.kv_len[b];
      const PwSeq s = pw_seq(p, start, end, n);
      v = p.Hkv * work(s, pw_blocks<G::KEYS>(s));
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
  const long long total = carry, piece = pw_share(total, p.ctas);
  const long long from = min(total, piece * blockIdx.x), to = min(total, from + piece);
  if (from >= to) return;

  // ---- the CTA's piece, a (sequence, KV head) at a time: the blocks that start in it. (One warp looks for the start: the
  // others' instructions would cost the SM's other CTAs more than they wait.)
  __shared__ int s_b, s_kvh, s_x0;
  if (warp == 0) {
    const int b = qda_seq_of(s_at, p.B, from);
    const PwSeq s = pw_seq(p, b);
    const int blocks = pw_blocks<G::KEYS>(s);
    const long long head = work(s, blocks);
    const int kvh = (int)((from - s_at[b]) / head);
    const long long at = s_at[b] + kvh * head;
    const int x0 = pw_block_at(blocks, from, [&](int i) { return at + work(s, i); });
    if (lane == 0) {
      s_b = b;
      s_kvh = kvh;
      s_x0 = x0;
    }
  }
  __syncthreads();
  int b = s_b, kvh = s_kvh;
  PwSeq s = pw_seq(p, b);
  int blocks = pw_blocks<G::KEYS>(s);
  long long head = work(s, blocks);
  long long at = s_at[b] + kvh * head;   // the KV head's place on the line
  auto block_at = [&](long long x) { return pw_block_at(blocks, x, [&](int i) { return at + work(s, i); }); };
  const int pmask = (1 << p.page_shift) - 1;
  int x0 = s_x0;
  constexpr int LPS = 32 / T;                 // lanes that fetch a sixteen of keys
  const int fsub = lane / LPS, fl = lane % LPS;
  // chunks of sixteen keys' scales, biases and masses, and where the first row's lie
  constexpr int CS = G::SC / 16, REST = 2 * CS + 4;
  auto rest_of = [&](int c) {
    return c < CS ? reinterpret_cast<const char*>(p.ks) + 16 * c
           : c < 2 * CS ? reinterpret_cast<const char*>(p.kb) + 16 * (c - CS) : reinterpret_cast<const char*>(p.mass) + 16 * (c - 2 * CS);
  };
  const char* const rest = rest_of(fl);
  const uint32_t rest_size = fl < 2 * CS ? NG * 2 : 4;
  while (true) {
    const int x1 = at + head <= to ? blocks : block_at(to);
    if (x0 < x1) {
      const int* tab = p.table + (size_t)b * p.max_pages;
      // sixteen keys `t` of the sequence: their page (-1: behind the sequence or this piece)
      const int t1 = min(x1 * (T * kPwWarps), (s.n + 15) >> 4);
      auto page_of = [&](int t) { return t < t1 ? __ldg(tab + (t * 16 >> p.page_shift)) : -1; };
      // (pool rows are below 2^32 - 1)
      auto row_of = [&](int t, int pg) {
        return (((uint32_t)pg * (uint32_t)p.Hkv + (uint32_t)kvh) << p.page_shift) + (uint32_t)((t * 16) & pmask);
      };
      // a tile on its way into a stage (a page outside the pool: nothing is read); pg: the page of this lane's sixteen
      auto fetch = [&](int t, int pg, int st) {
        if ((unsigned)pg < (unsigned)p.num_pages) {
          const uint32_t row = row_of(t + fsub, pg);
          const uint32_t dst = smem_addr(ring + st * G::STAGE + fsub * G::SUB);
          const char* src = reinterpret_cast<const char*>(p.kp) + (uint64_t)row * RB + 16 * fl;
#pragma unroll
          for (int i = 0; i < (16 * G::CPR + LPS - 1) / LPS; ++i) {
            const int c = i * LPS + fl;
            if (16 * G::CPR >= LPS || c < 16 * G::CPR)
              pw_copy16(dst + pw_chunk<RB>(c / G::CPR, c % G::CPR), src + 16 * LPS * i);
          }
          if constexpr (REST <= LPS) {
            if (fl < REST) pw_copy16(dst + 16 * RB + 16 * fl, rest + (uint64_t)row * rest_size);
          } else {
#pragma unroll
            for (int i = 0; i < (REST + LPS - 1) / LPS; ++i) {
              const int c = i * LPS + fl;
              if (c < REST) pw_copy16(dst + 16 * RB + 16 * c, rest_of(c) + (uint64_t)row * (c < 2 * CS ? NG * 2 : 4));
            }
          }
        }
        pw_commit();
      };
      const int first = (s.len - s.count) * p.nrep, r_hi = s.len * p.nrep;
      int t = x0 * (T * kPwWarps) + warp * T;
      int pages[S];   // of this lane's sixteen of the tiles in flight, and of the next one
#pragma unroll
      for (int i = 0; i < S; ++i) pages[i] = page_of(t + i * (T * kPwWarps) + fsub);
#pragma unroll
      for (int i = 0; i < S - 1; ++i) fetch(t + i * (T * kPwWarps), pages[i], i);
      const bool many = r_hi - first > ROWS;
      if (!many) {
        __syncthreads();   // the operands of before are read
        pw_rows<BITS, D, GS, NT, F16>(p, s, kvh, first, ops, rows);
        __syncthreads();
      }
      // keys up to here are seen by every counted row
      const int open = s.base + s.len - s.count;
      int st = 0;
#pragma unroll 1
      for (int step = x0; step < x1; ++step, t += T * kPwWarps) {
        fetch(t + (S - 1) * (T * kPwWarps), pages[S - 1], st == 0 ? S - 1 : st - 1);   // into the stage that was read last
        pw_wait<S - 1>();
        __syncwarp();
        const int pg = pages[0];
#pragma unroll
        for (int i = 0; i < S - 1; ++i) pages[i] = pages[i + 1];
        pages[S - 1] = page_of(t + S * (T * kPwWarps) + fsub);
        const bool mine = (unsigned)pg < (unsigned)p.num_pages;
        if (!mine && t + fsub < t1) atomicOr(p.err, QDA_ERR_BIT_PAGED);
        const bool any = __any_sync(0xffffffffu, mine);
        const char* const stage = ring + st * G::STAGE;
        st = st == S - 1 ? 0 : st + 1;
        const int key0 = t * 16;
        float sum[2 * T];   // of keys r8 and r8 + 8 of each sixteen, this lane's columns
#pragma unroll
        for (int i = 0; i < 2 * T; ++i) sum[i] = 0.f;
        auto tile = [&]() {
          float sc[NT][T][4];
          uint32_t sw[T][2][(NG + 1) / 2], bw[T][2][(NG + 1) / 2];
#pragma unroll
          for (int z = 0; z < T; ++z) {
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const char* q = stage + z * G::SUB + 16 * RB + (r8 + 8 * y) * NG * 2;
              pw_lds<NG * 2>(q, sw[z][y]);
              pw_lds<NG * 2>(q + G::SC, bw[z][y]);
            }
          }
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            constexpr int LB = UPL * WPU * 4;   // a lane's bytes of a group
            uint32_t code[T][2][UPL * WPU];
#pragma unroll
            for (int z = 0; z < T; ++z) {
#pragma unroll
              for (int y = 0; y < 2; ++y) {
                if constexpr (LB <= 16) {
                  const int off = g * 4 * LB + c4 * LB;
                  pw_lds<LB>(stage + z * G::SUB + pw_chunk<RB>(r8 + 8 * y, off >> 4) + (off & 15), code[z][y]);
                } else {
#pragma unroll
                  for (int i = 0; i < LB / 16; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4*>(
                        stage + z * G::SUB + pw_chunk<RB>(r8 + 8 * y, (g * 4 * LB + c4 * LB) / 16 + i));
                    code[z][y][4 * i] = v.x;
                    code[z][y][4 * i + 1] = v.y;
                    code[z][y][4 * i + 2] = v.z;
                    code[z][y][4 * i + 3] = v.w;
                  }
                }
              }
            }
            float acc[NT][T][4];
#pragma unroll
            for (int u = 0; u < UPL; ++u) {
              uint32_t a[T][8];   // two k-steps
#pragma unroll
              for (int z = 0; z < T; ++z) {
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                  if constexpr (BITS == 4) {
                    const uint32_t w = code[z][y][u], v = w >> 8;
                    a[z][y] = w & 0x000F000Fu;
                    a[z][2 + y] = w & 0x00F000F0u;
                    a[z][4 + y] = v & 0x000F000Fu;
                    a[z][6 + y] = v & 0x00F000F0u;
                  } else {
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                      const uint32_t w = code[z][y][2 * u + j];
                      a[z][4 * j + y] = w & 0x00FF00FFu;
                      a[z][4 * j + 2 + y] = (w >> 8) & 0x00FF00FFu;
                    }
                  }
                }
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint4 bq = ops[(nt * G::UNITS + g * UPL + u) * 32 + lane];
#pragma unroll
                for (int z = 0; z < T; ++z) {
                  pw_mma(acc[nt][z], a[z][0], a[z][1], a[z][2], a[z][3], bq.x, bq.y, u > 0);
                  pw_mma(acc[nt][z], a[z][4], a[z][5], a[z][6], a[z][7], bq.z, bq.w, true);
                }
              }
            }
#pragma unroll
            for (int z = 0; z < T; ++z) {
              const float s0 = pw_half<F16>(sw[z][0], g), s1 = pw_half<F16>(sw[z][1], g);
              const float b0 = pw_half<F16>(bw[z][0], g), b1 = pw_half<F16>(bw[z][1], g);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const float2 qs = rows.sum[nt][g][c4];
                float (&x)[4] = sc[nt][z];
                const float (&v)[4] = acc[nt][z];
                x[0] = fmaf(b0, qs.x, g == 0 ? s0 * v[0] : fmaf(s0, v[0], x[0]));
                x[1] = fmaf(b0, qs.y, g == 0 ? s0 * v[1] : fmaf(s0, v[1], x[1]));
                x[2] = fmaf(b1, qs.x, g == 0 ? s1 * v[2] : fmaf(s1, v[2], x[2]));
                x[3] = fmaf(b1, qs.y, g == 0 ? s1 * v[3] : fmaf(s1, v[3], x[3]));
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float2 mul = rows.mul[nt][c4], ls = rows.lse[nt][c4];
#pragma unroll
            for (int z = 0; z < T; ++z) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                sc[nt][z][j] = fmaf(sc[nt][z][j], j & 1 ? mul.y : mul.x, j & 1 ? -ls.y : -ls.x);
              if (many || key0 + 16 * T - 1 > open) {   // some row does not see some key
                const int2 last = rows.last[nt][c4];
                const int key = key0 + 16 * z + r8;
                if (key > last.x) sc[nt][z][0] = -INFINITY;
                if (key > last.y) sc[nt][z][1] = -INFINITY;
                if (key + 8 > last.x) sc[nt][z][2] = -INFINITY;
                if (key + 8 > last.y) sc[nt][z][3] = -INFINITY;
              }
              sum[2 * z] += pw_ex2(sc[nt][z][0]);
              sum[2 * z] += pw_ex2(sc[nt][z][1]);
              sum[2 * z + 1] += pw_ex2(sc[nt][z][2]);
              sum[2 * z + 1] += pw_ex2(sc[nt][z][3]);
            }
          }
        };
        // the counted tokens that see the block's first key
        int row = many ? max(first, max(step * G::KEYS - s.base, 0) * p.nrep) : first;
        do {
          if (many) {
            __syncthreads();   // the operands of before are read
            pw_rows<BITS, D, GS, NT, F16>(p, s, kvh, row, ops, rows);
            __syncthreads();
          }
          if (any) tile();
          row += ROWS;
        } while (row < r_hi);
        // ---- a key's sum over the quad's columns: with two sixteens each lane ends with one key's, its new mass
        float add;
        if constexpr (T == 2) {
          const float x = c4 & 2 ? sum[0] : sum[2], y = c4 & 2 ? sum[1] : sum[3];
          const float u = (c4 & 2 ? sum[2] : sum[0]) + __shfl_xor_sync(0xffffffffu, x, 2);
          const float v = (c4 & 2 ? sum[3] : sum[1]) + __shfl_xor_sync(0xffffffffu, y, 2);
          add = (c4 & 1 ? v : u) + __shfl_xor_sync(0xffffffffu, c4 & 1 ? u : v, 1);
        } else {
          const float x = (c4 & 1 ? sum[1] : sum[0]) + __shfl_xor_sync(0xffffffffu, c4 & 1 ? sum[0] : sum[1], 1);
          add = x + __shfl_xor_sync(0xffffffffu, x, 2);
        }
        const int z = T == 2 ? c4 >> 1 : 0, i = r8 + 8 * (c4 & 1), key = key0 + 16 * z + i;
        const int kpg = T == 2 ? __shfl_sync(0xffffffffu, pg, z * LPS) : pg;   // the page of this lane's key
        if ((T == 2 || c4 < 2) && key < s.n && (unsigned)kpg < (unsigned)p.num_pages) {
          const uint32_t at_row = row_of(t + z, kpg) + i;
          if (key < s.base) {
            p.mass[at_row] = fmaf(p.decay, *reinterpret_cast<const float*>(stage + z * G::SUB + 16 * RB + 2 * G::SC + 4 * i), add);
          } else {
            p.mass[at_row] = add;
            p.token[at_row] = key + (p.shift != nullptr ? p.shift[b] : 0);
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
        blocks = pw_blocks<G::KEYS>(s);
      } while (blocks == 0);
      head = work(s, blocks);
    }
    if (at >= to) return;
  }
}

template <int BITS, int D, int GS, int NT, bool F16>
cudaError_t pw_run(const QdaWeightsParams* p, int* ctas_per_sm, cudaStream_t s) {
  using G = PwGeom<BITS, D, GS, NT>;
  auto kern = qda_paged_weights_kernel<BITS, D, GS, NT, F16>;
  if (ctas_per_sm != nullptr) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, kern, kPwWarps * 32, G::SMEM);
    return e;
  }
  kern<<<p->ctas, kPwWarps * 32, G::SMEM, s>>>(*p);
  return cudaGetLastError();
}

template <int BITS, bool F16>
cudaError_t pw_pick(const QdaWeightsParams* p, int D, int GS, int rows, int* occ, cudaStream_t s) {
#define QDA_PW(d, gs)                                                                       \
  if (D == d && GS == gs)                                                                   \
    return rows == 1 ? pw_run<BITS, d, gs, 1, F16>(p, occ, s)                               \
           : rows == 2 ? pw_run<BITS, d, gs, 2, F16>(p, occ, s) : pw_run<BITS, d, gs, 4, F16>(p, occ, s);
  QDA_PW(64, 32) QDA_PW(64, 64)
  QDA_PW(128, 32) QDA_PW(128, 64) QDA_PW(128, 128)
  QDA_PW(256, 32) QDA_PW(256, 64) QDA_PW(256, 128)
  QDA_PW(512, 32) QDA_PW(512, 64) QDA_PW(512, 128)
#undef QDA_PW
  return cudaErrorInvalidValue;
}

}  // namespace qda
