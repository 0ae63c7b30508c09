// Paged attention for few query rows per KV head (sm_103a): single tokens, a few tokens per sequence, and every shape the
// chunk kernel does not take. Bound by HBM (the cache is read once per tile of 8 or 16 rows) and next to it by issue slots.
//
// Matrix instructions work on the codes themselves. A warp takes 16 keys at a time; the codes, straight from shared memory,
// become the 16-bit A operand of m16n8k16 products with fp32 sums (a few query rows are far too thin for the 128-row tiles
// of tcgen05, and its operands would have to be written back to shared or tensor memory first; here they never leave the
// registers):
//   scores   rows = keys, k = head dimension, columns = query rows. A code's bits as they are, masked out of the packed
//            word, are the fp16 subnormal c 2^-24 (16 c 2^-24 where a nibble is left unshifted, with q / 16 on the other
//            side): one AND makes two operand values, exact. q goes in as fp16 after an exact scaling of each row by a
//            power of two (bf16 has fewer significant bits and a wider range). Per group, s_g sum(c q) + b_g sum(q) is
//            formed in fp32: the scores are right to fp32.
//   values   rows = head dimension, k = keys, columns = query rows: the weight w = p s_g of each group is the B operand,
//            rounded to fp16 (11 significant bits: next to nothing beside a bf16 result, as much as the one rounding of an
//            fp16 one; w 2^-22 of the largest and less lose a bit with every factor of two); all sums of a query row are
//            taken in a unit 2^-vexp that follows the largest scale of the keys that the row sees and keeps w in range. To
//            centre the codes on the middle of their range (so that the rounding of w meets values no larger than half a
//            group's range), sum(w) of a group comes from one more product with A = the middle, or with many groups the
//            middle is taken off the codes; the rest, sum(p (b_g + mid s_g)), stays in fp32.
// Keys and query rows change places between the two products: one movmatrix per 8 x 8 weights.
//
// Memory: each warp fills its own ring of shared-memory stages with 16-byte asynchronous copies (no warp waits for
// another), the 16-byte pieces of a row XORed over the banks so that both operand reads are free of conflicts. The online
// softmax keeps a reference per query row that moves only when a score passes it by more than 4 (log2 units): one vote per
// 16 keys. Measured: one token of 64 sequences of 700 to 8200 keys (32 heads, 8 KV heads, D 128, 4-bit) 97 us, 3.4 TB/s of
// cache, half of a copy's rate: some 430 instructions per 16 keys keep the schedulers busy, and of the four CTAs of an SM
// the one launched last runs a third longer (pieces weighted against that: 96 us here, but 59 instead of 54 for one long
// sequence; not kept). One sequence of 131072 keys (16 heads, 4 KV heads, D 256) 55 us, 3.0 TB/s (lengths near it
// 60); 512 keys 14.4 us, latency.
// Hidden keys (behind the sequence, in a token's future, on a page outside the pool) get the weight 0 by selection and do
// not count for a row's unit, so that what their rows hold, NaN and large scales included, reaches nothing.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qda_paged_sched.cuh"

namespace qda {

constexpr int kPsWarps = 4;

template <int BITS, int D, int GS, int NT>
struct PsGeom {
  static constexpr int MT = 8 * NT;
  static constexpr int NG = D / GS;
  static constexpr int RB = D * BITS / 8;                 // bytes of codes per row
  static constexpr int KPS = RB <= 64 ? 32 : 16;          // keys per stage: at least 2 KB of codes of each kind
  static constexpr int CODE = KPS * RB;                   // bytes of K (or V) codes per stage
  static constexpr int SC = KPS * NG * 2;                 // bytes of one scale or bias array per stage
  static constexpr int STAGE = 2 * CODE + 4 * SC;
  static constexpr int STAGES = 3;
  static constexpr bool QSMEM = D * NT > 256;             // q operands in shared memory (else in registers)
  static constexpr bool SSMEM = NG * NT > 4;              // sums of q in shared memory
  static constexpr bool ONES = NG <= 4;                   // codes centred by a product with A = middle (else one by one)
  static constexpr int QF = QSMEM ? (D / 16) * NT * 256 : 0;
  static constexpr int QS = SSMEM ? NG * MT * 4 : 0;
  static constexpr int ROWS = QF + QS;
  static constexpr int RING = kPsWarps * STAGES * STAGE;
  static constexpr int COMB = kPsWarps * 8 * D * 4;   // the warps' results of 8 query rows
  static constexpr int SMEM = ROWS + (RING > COMB ? RING : COMB);
  static_assert(SMEM - ROWS >= (int)sizeof(PagedLine), "the line lies in the ring");
  static constexpr int OREGS = D / 4 * NT;
  // resident CTAs: as many as leave most instances without spills (the one of the batch above spills a few registers at 4)
  static constexpr int MINB = OREGS <= 32 ? (NG * NT > 2 ? 3 : 4) : 2;
};

__device__ __forceinline__ void ps_cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void ps_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ps_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ps_mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1, float c0, float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %11, "
      "%12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t ps_trans(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float ps_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t ps_bf2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ uint32_t ps_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t ps_sub2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// What a key row's bytes are XORed with within a stage's codes: 32-byte pieces move over the banks so that the operand
// reads (8 rows at one column, and 4 rows two apart at neighbouring columns) fall on distinct ones.
template <int RB>
__host__ __device__ constexpr uint32_t ps_turn(int row) {
  return (RB < 128 ? ((row * RB) >> 7) & 3 : (row & 3) ^ ((row >> 2) & 1)) << 5;
}

// N 16-bit values of a row's scales (or biases) from shared memory
template <int N>
__device__ __forceinline__ void ps_halves(uint32_t addr, uint32_t (&w)[(N + 1) / 2]) {
  if constexpr (N == 1) {
    unsigned short h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
    w[0] = h;
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (N == 4) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(addr + 16 * i));
  }
}
template <bool F16>
__device__ __forceinline__ float ps_half(const uint32_t* w, int g) {
  const uint32_t x = w[g >> 1];
  if constexpr (F16) {
    return __half2float(__ushort_as_half((unsigned short)((g & 1) ? x >> 16 : x & 0xffffu)));
  } else {
    return __uint_as_float((g & 1) ? x & 0xffff0000u : x << 16);
  }
}

// Largest 16-bit pattern of a scale below 2^k (fp16's subnormal ones count in steps of 2^-24, not in exponents)
template <bool F16>
__device__ __forceinline__ uint32_t ps_below(int k) {
  if constexpr (F16) return k > 15 ? 0x7BFFu : k > -15 ? ((uint32_t)(k + 15) << 10) - 1 : k > -25 ? (1u << (k + 24)) - 1 : 0u;
  else return k > 127 ? 0x7F7Fu : ((uint32_t)(k + 127) << 7) - 1;   // k stays far above the subnormal ones
}

// NW words of codes (NW = 0: half a word) from shared memory
template <int NW>
__device__ __forceinline__ void ps_words(uint32_t addr, uint32_t* w) {
  if constexpr (NW == 0) {
    unsigned short h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
    w[0] = h;
  } else if constexpr (NW == 1) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else if constexpr (NW == 2) {
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
#pragma unroll
    for (int i = 0; i < NW / 4; ++i)
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3])
                   : "r"(addr + 16 * i));
  }
}

// One output pair (two neighbouring values of the head dimension).
template <bool F16>
__device__ __forceinline__ uint32_t ps_out2(float a, float b) {
  if constexpr (F16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  } else {
    return ps_bf2(a, b);
  }
}

template <int BITS, int D, int GS, int NT, bool F16>
__global__ void __launch_bounds__(kPsWarps * 32, PsGeom<BITS, D, GS, NT>::MINB)
    qda_paged_split_kernel(const __grid_constant__ QdaPagedParams p) {
  using G = PsGeom<BITS, D, GS, NT>;
  constexpr int NG = G::NG, MT = G::MT, KPS = G::KPS, RB = G::RB, STAGES = G::STAGES;
  constexpr int GSB = GS * BITS / 8;          // bytes of a group's codes
  constexpr int KS = GS / 16;                 // products per group and key tile, on either side
  constexpr float MID = BITS == 4 ? 8.f : 128.f;
  constexpr uint32_t MID_LO = BITS == 4 ? 0x00080008u : 0x00800080u, MID_HI = 0x00800080u;   // middle codes as operands
  constexpr float TINY = 5.9604644775390625e-8f, GREAT = 16777216.f;                         // 2^-24, 2^24
  extern __shared__ __align__(128) unsigned char ps_smem[];
  __shared__ float s_ml[NT][kPsWarps][2][8];   // per 8 query rows and warp: reference, sum
  __shared__ PagedTile t;   // the tile at hand, and this CTA's piece of the line
  __shared__ long long s_x[2];
  __shared__ int s_more;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, r8 = lane >> 2, c4 = lane & 3;
  uint2* s_qf = reinterpret_cast<uint2*>(ps_smem);
  float* s_qs = reinterpret_cast<float*>(ps_smem + G::QF);   // [NG][MT] sums of q, times 2^-24
  const uint32_t ring = smem_addr(ps_smem + G::ROWS) + warp * STAGES * G::STAGE;
  float* comb = reinterpret_cast<float*>(ps_smem + G::ROWS);

  const uint32_t koff = (r8 * RB + c4 * (GSB / 4)) ^ ps_turn<RB>(r8), voff = (2 * c4 * RB + r8 * (GSB / 8)) ^ ps_turn<RB>(2 * c4);

  pdl_launch_dependents();
  PagedLine& line = *reinterpret_cast<PagedLine*>(comb);   // before the first copy lands there
  paged_line(p, MT, line);
  const long long total = line.at[p.B];
  const int cta = blockIdx.x;
  const PagedPieces pieces = paged_pieces(p, total);
  if (tid == 0) p.split[cta] = QdaPagedSplitTile{};
  if (cta >= pieces.ctas) return;
  if (tid == 0) {
    s_x[0] = paged_border(pieces, cta);
    s_x[1] = paged_border(pieces, cta + 1);
    t = paged_tile_at(p, line, MT, s_x[0]);
  }
  __syncthreads();
  const int pmask = (1 << p.page_shift) - 1;

  for (;;) {
    const int keys = paged_tile_keys(p, t, MT);
    const int nblk = (keys + KPS - 1) / KPS;
    const int j0 = paged_block_at(t, nblk, s_x[0]), j1 = paged_block_at(t, nblk, s_x[1]);
    const bool mine = s_x[0] <= t.lo;   // the CTA that starts the tile
    if (j0 < j1 || (nblk == 0 && mine)) {
      const int row0 = t.i * MT;
      // ---- this warp's key blocks j0 + warp, + kPsWarps, ... through its ring
      const int mine_n = j1 - j0 > warp ? (j1 - j0 - warp + kPsWarps - 1) / kPsWarps : 0;
      const int* tab = p.table + (size_t)t.b * p.max_pages;
      // the pages of a block's two 16-key halves (one half where a block is 16 keys), looked up one block ahead of the copies
      constexpr int HALVES = KPS / 16, STEP = kPsWarps * KPS;
      int pg[HALVES];
      int fill_n = (j0 + warp) * KPS, fill_left = mine_n, fill_stage = 0;   // next block to copy, blocks to copy, its stage
      auto look = [&]() {
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          const int n = fill_n + 16 * h;
          pg[h] = fill_left > 0 && n < keys ? __ldg(tab + (n >> p.page_shift)) : 0;
        }
      };
      bool saw_absent = false;
      uint32_t absent = 0;   // bit (stage * 2 + half): that half's page is outside the pool
      // this lane's 16 bytes of a block's scales and biases: NG * 2 pieces per array and half
      constexpr int PC = HALVES * NG * 2, SI = (4 * PC + 31) / 32;
      auto issue = [&]() {
        if (fill_left > 0) {
          const uint32_t base = ring + fill_stage * G::STAGE;
          uint32_t row[HALVES], gone = 0;   // pool rows (32 bits: the host checks)
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const bool ok = (unsigned)pg[h] < (unsigned)p.num_pages;
            gone |= ok ? 0u : 1u << h;
            row[h] = ((((uint32_t)(ok ? pg[h] : 0) * p.Hkv) + t.unit) << p.page_shift) + ((fill_n + 16 * h) & pmask);
          }
          if (gone | absent) {   // rare
            absent = (absent & ~(3u << (2 * fill_stage))) | gone << (2 * fill_stage);
            saw_absent = saw_absent || gone;
          }
          constexpr int PER = 16 * RB / 512;   // copies of 32 lanes per half
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {
            const char* ksrc = reinterpret_cast<const char*>(p.kp) + (uint64_t)row[h] * RB + lane * 16;
            const char* vsrc = reinterpret_cast<const char*>(p.vp) + (uint64_t)row[h] * RB + lane * 16;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
              const int at = ((h * PER + i) * 32 + lane) * 16, key = at / RB;
              const uint32_t dst = base + (at ^ ps_turn<RB>(key));
              ps_cp16(dst, ksrc + i * 512);
              ps_cp16(dst + G::CODE, vsrc + i * 512);
            }
          }
#pragma unroll
          for (int i = 0; i < SI; ++i) {
            const int id = i * 32 + lane, a = id / PC, k16 = id % PC;
            if (id < 4 * PC) {
              const uint16_t* arr = a == 0 ? p.ks : a == 1 ? p.kb : a == 2 ? p.vs : p.vb;
              const int h = HALVES == 2 ? k16 / (NG * 2) : 0;
              const char* src = reinterpret_cast<const char*>(arr) + (k16 - h * NG * 2) * 16 +
                                (uint64_t)(HALVES == 2 && h ? row[HALVES - 1] : row[0]) * (NG * 2);
              ps_cp16(base + 2 * G::CODE + a * G::SC + k16 * 16, src);
            }
          }
          fill_stage = fill_stage + 1 == STAGES ? 0 : fill_stage + 1;
          fill_n += STEP;
          --fill_left;
          look();
        }
        ps_commit();
      };

      look();
#pragma unroll
      for (int k = 0; k < STAGES - 1; ++k) issue();   // under way while the queries are prepared

      // ---- the tile's query rows: B operands, sums per group, and how far each sees
      uint2 qf[G::QSMEM ? 1 : D / 16 * NT];
      float qsum[G::SSMEM ? 1 : NG * NT][2];
      float qmul[NT][2];
      int seen[NT][2];
      int least = 0x7fffffff;   // keys that every row of the tile sees
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = row0 + nt * 8 + r8;
        const bool real = r < t.s.rows;
        const int tok = r / p.nrep;
        const uint16_t* qp = p.q + (long long)(t.s.first + tok) * p.q_tstride +
                             (long long)(t.unit * p.nrep + (r - tok * p.nrep)) * p.q_hstride;
        // lane c4 holds dimensions g GS + c4 GS / 4 ... of every group of row r8
        uint32_t raw[D / 8];
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int i = 0; i < GS / 32; ++i) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (real) v = *reinterpret_cast<const uint4*>(qp + g * GS + c4 * (GS / 4) + 8 * i);
            raw[g * (GS / 8) + 4 * i] = v.x;
            raw[g * (GS / 8) + 4 * i + 1] = v.y;
            raw[g * (GS / 8) + 4 * i + 2] = v.z;
            raw[g * (GS / 8) + 4 * i + 3] = v.w;
          }
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
          top = fmaxf(top, fmaxf(fabsf(ps_half<F16>(&raw[i], 0)), fabsf(ps_half<F16>(&raw[i], 1))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // largest value of the row to [2^8, 2^9): every product stays far inside fp32, values down to 2^-22 of it are normal
        // in fp16
        const int fe = min(262 - (int)((__float_as_uint(top) >> 23) & 255u), 253);
        const float up = __uint_as_float((uint32_t)fe << 23), down = __uint_as_float((uint32_t)(254 - fe) << 23);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
          float sum = 0.f;
#pragma unroll
          for (int i = 0; i < GS / 32; ++i) {
            // eight values of the row: 4-bit: two products (codes 0 4 | 1 5, and 2 6 | 3 7), 8-bit: (0 2 | 1 3, 4 6 | 5 7)
            float v[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) v[e] = ps_half<F16>(&raw[g * (GS / 8) + 4 * i], e) * up;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const float lo0 = BITS == 4 ? v[2 * h] : v[4 * h], lo1 = BITS == 4 ? v[2 * h + 4] : v[4 * h + 2];
              const float hi0 = BITS == 4 ? v[2 * h + 1] * 0.0625f : v[4 * h + 1];
              const float hi1 = BITS == 4 ? v[2 * h + 5] * 0.0625f : v[4 * h + 3];
              const __half2 a = __floats2half2_rn(lo0, lo1), b = __floats2half2_rn(hi0, hi1);
              const uint2 f = make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
              const int ks = (g * (GS / 32) + i) * 2 + h;
              if constexpr (G::QSMEM) {
                if (warp == 0) s_qf[(ks * NT + nt) * 32 + lane] = f;
              } else {
                qf[ks * NT + nt] = f;
              }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += v[e];
          }
          // over the four lanes of the row
          sum += __shfl_xor_sync(0xffffffffu, sum, 1);
          sum += __shfl_xor_sync(0xffffffffu, sum, 2);
          sum *= TINY;
          if constexpr (G::SSMEM) {
            if (warp == 0 && c4 == 0) s_qs[g * MT + nt * 8 + r8] = sum;
          } else {
            // scores hold query rows 2 c4, 2 c4 + 1 in this lane
#pragma unroll
            for (int j = 0; j < 2; ++j) qsum[g * NT + nt][j] = __shfl_sync(0xffffffffu, sum, (2 * c4 + j) * 4);
          }
        }
        const int sr = real ? paged_seen(p, t.s, r) : keys;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          qmul[nt][j] = __shfl_sync(0xffffffffu, down, (2 * c4 + j) * 4) * p.qscale * GREAT;
          seen[nt][j] = __shfl_sync(0xffffffffu, sr, (2 * c4 + j) * 4);
          least = min(least, seen[nt][j]);
        }
      }
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 1));
      least = min(least, __shfl_xor_sync(0xffffffffu, least, 2));
      if constexpr (G::QSMEM || G::SSMEM) __syncthreads();

      float o[NG * KS * NT][4], wsum[G::ONES ? NG * NT : 1][4], vb[NG * NT][2], l[NT][2], m[NT][2];
#pragma unroll
      for (int i = 0; i < NG * KS * NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
      if constexpr (G::ONES) {
#pragma unroll
        for (int i = 0; i < NG * NT; ++i) wsum[i][0] = wsum[i][1] = wsum[i][2] = wsum[i][3] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < NG * NT; ++i) vb[i][0] = vb[i][1] = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        l[nt][0] = l[nt][1] = 0.f;
        m[nt][0] = m[nt][1] = -INFINITY;
      }

      // each row's unit: everything that is summed for it is taken times 2^vexp, an integer that follows the value scales
      // that the row sees. most: 16-bit pattern of the largest scale that the units of this lane's rows all allow
      float vexp[NT][2];
      uint32_t most = 0, known = 0;   // known: bit 2 nt + j: the row has met a scale other than 0
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) vexp[nt][0] = vexp[nt][1] = 0.f;

      int st = 0, first = (j0 + warp) * KPS;   // the block's stage and first key
      for (int k = 0; k < mine_n; ++k) {
        issue();   // into the stage read one block ago
        ps_wait<STAGES - 1>();
        __syncwarp();   // every lane's pieces of the stage are in
        const uint32_t base = ring + st * G::STAGE;
#pragma unroll 1
        for (int h = 0; h < KPS / 16; ++h) {
          const int n0 = first + 16 * h;
          if (n0 >= keys) break;
          const bool gone = (absent >> (st * 2 + h)) & 1u;
          const bool edge = gone || n0 + 16 > least;
          // codes: key row r8 (and r8 + 8) at this lane's quarter of a group; key rows 2 c4, 2 c4 + 1 (and 8 behind) at its
          // eighth. Stages lie on 128-byte borders: what moves within 128 bytes is an XOR, the rest a sum
          const uint32_t kat = base + 16 * h * RB + koff, vat = base + G::CODE + 16 * h * RB + voff;
          constexpr uint32_t UP8 = RB == 32 ? 64 : 0, ODD = RB >= 128 ? 32 : RB, ODD_UP = RB >= 128 ? RB : 0;
          const uint32_t sc = base + 2 * G::CODE + (16 * h + r8) * NG * 2;   // this lane's key rows: r8 and r8 + 8
          // ---- scores
          float s[NT][4];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
          {
            uint32_t sw[2][(NG + 1) / 2], bw[2][(NG + 1) / 2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              ps_halves<NG>(sc + x * 8 * NG * 2, sw[x]);
              ps_halves<NG>(sc + G::SC + x * 8 * NG * 2, bw[x]);
            }
#pragma unroll
            for (int g = 0; g < NG; ++g) {
              constexpr int KW = GS * BITS / 128;   // words per lane, group and row
              uint32_t w0[KW], w1[KW];
              ps_words<KW>((kat ^ (g * GSB & 127)) + (g * GSB & ~127), w0);
              ps_words<KW>((kat ^ (g * GSB & 127) ^ UP8) + (g * GSB & ~127) + 8 * RB, w1);
              float acc[NT][4];
#pragma unroll
              for (int j = 0; j < KS; ++j) {
                uint32_t a0, a1, a2, a3;
                if constexpr (BITS == 4) {
                  const uint32_t u = (j & 1) ? w0[j / 2] >> 8 : w0[j / 2], v = (j & 1) ? w1[j / 2] >> 8 : w1[j / 2];
                  a0 = u & 0x000F000Fu;
                  a1 = v & 0x000F000Fu;
                  a2 = u & 0x00F000F0u;
                  a3 = v & 0x00F000F0u;
                } else {
                  a0 = w0[j] & 0x00FF00FFu;
                  a1 = w1[j] & 0x00FF00FFu;
                  a2 = (w0[j] >> 8) & 0x00FF00FFu;
                  a3 = (w1[j] >> 8) & 0x00FF00FFu;
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  uint2 f;
                  if constexpr (G::QSMEM) f = s_qf[((g * KS + j) * NT + nt) * 32 + lane];
                  else f = qf[(g * KS + j) * NT + nt];
                  if (j == 0) {
                    ps_mma(acc[nt], a0, a1, a2, a3, f.x, f.y, 0.f, 0.f, 0.f, 0.f);
                  } else {
                    ps_mma(acc[nt], a0, a1, a2, a3, f.x, f.y, acc[nt][0], acc[nt][1], acc[nt][2], acc[nt][3]);
                  }
                }
              }
              const float s0 = ps_half<F16>(sw[0], g), s1 = ps_half<F16>(sw[1], g);
              const float b0 = ps_half<F16>(bw[0], g), b1 = ps_half<F16>(bw[1], g);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float q0, q1;
                if constexpr (G::SSMEM) {
                  q0 = s_qs[g * MT + nt * 8 + 2 * c4];
                  q1 = s_qs[g * MT + nt * 8 + 2 * c4 + 1];
                } else {
                  q0 = qsum[g * NT + nt][0];
                  q1 = qsum[g * NT + nt][1];
                }
                s[nt][0] = fmaf(b0, q0, fmaf(s0, acc[nt][0], s[nt][0]));
                s[nt][1] = fmaf(b0, q1, fmaf(s0, acc[nt][1], s[nt][1]));
                s[nt][2] = fmaf(b1, q0, fmaf(s1, acc[nt][2], s[nt][2]));
                s[nt][3] = fmaf(b1, q1, fmaf(s1, acc[nt][3], s[nt][3]));
              }
            }
          }
          // ---- weights
          uint32_t sw[2][(NG + 1) / 2], bw[2][(NG + 1) / 2];   // the values' scales and biases
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            ps_halves<NG>(sc + 2 * G::SC + x * 8 * NG * 2, sw[x]);
            ps_halves<NG>(sc + 3 * G::SC + x * 8 * NG * 2, bw[x]);
          }
          uint32_t big = 0;   // largest scale of this lane's keys (a pattern per half word)
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            uint32_t y = sw[x][0] & 0x7fff7fffu;
#pragma unroll
            for (int i = 1; i < (NG + 1) / 2; ++i) y = __vmaxu2(y, sw[x][i] & 0x7fff7fffu);
            if (edge && (gone || n0 + r8 + 8 * x >= keys)) y = 0;   // rows behind the sequence may hold anything
            big = __vmaxu2(big, y);
          }
          big = max(big & 0xffffu, big >> 16);
          bool rise = big > most;
          uint32_t hidden = 0;   // bit 4 nt + j: score j of query rows nt is hidden
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int j = 0; j < 4; ++j) s[nt][j] *= qmul[nt][j & 1];
            if (edge) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (gone || n0 + r8 + (j >> 1) * 8 >= seen[nt][j & 1]) {
                  s[nt][j] = -INFINITY;
                  hidden |= 1u << (4 * nt + j);
                }
            }
            rise = rise || fmaxf(s[nt][0], s[nt][2]) > m[nt][0] + 4.f || fmaxf(s[nt][1], s[nt][3]) > m[nt][1] + 4.f;
          }
          if (__any_sync(0xffffffffu, rise)) {
            // a row's unit: the largest finite scale that it sees to [2^8, 2^9), good for scales up to 4 times that and
            // weights up to 2^4 (w stays below 2^15): as high as fp16 goes, so that small weights keep their bits
            constexpr uint32_t INF = F16 ? 0x7C00u : 0x7F80u;
            // the largest scale of either key of this lane, anew (rare: not worth a register elsewhere)
            uint32_t mine2[2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              uint32_t y = sw[x][0] & 0x7fff7fffu;
#pragma unroll
              for (int i = 1; i < (NG + 1) / 2; ++i) y = __vmaxu2(y, sw[x][i] & 0x7fff7fffu);
              y = max(y & 0xffffu, y >> 16);
              mine2[x] = y < INF ? y : 0u;
            }
            most = INF - 1;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                float x = fmaxf(s[nt][j], s[nt][j + 2]);
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                const float mn = fmaxf(m[nt][j], x);
                // the largest scale that the row sees here
                uint32_t top = max((hidden >> (4 * nt + j)) & 1u ? 0u : mine2[0],
                                   (hidden >> (4 * nt + j + 2)) & 1u ? 0u : mine2[1]);
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 4));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 8));
                top = max(top, __shfl_xor_sync(0xffffffffu, top, 16));
                float fo = 1.f;
                const bool none = m[nt][j] == -INFINITY;   // no key was visible before: sums are 0
                if (top > ((known >> (2 * nt + j)) & 1u ? ps_below<F16>(11 - (int)vexp[nt][j]) : 0u)) {
                  const uint32_t w = top;
                  const int e = (int)(__float_as_uint(ps_half<F16>(&w, 0)) >> 23) - 127;
                  const float ve = (float)max(-60, min(8 - e, 60));
                  fo = ps_ex2(ve - vexp[nt][j]);
                  vexp[nt][j] = ve;
                  known |= 1u << (2 * nt + j);
                }
                if (mn != -INFINITY) most = min(most, (known >> (2 * nt + j)) & 1u ? ps_below<F16>(11 - (int)vexp[nt][j]) : 0u);
                const float f = none ? 0.f : ps_ex2(m[nt][j] - mn) * fo;
                m[nt][j] = mn;
                l[nt][j] *= f;
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                  vb[g * NT + nt][j] *= f;
                  if constexpr (G::ONES) {
                    wsum[g * NT + nt][j] *= f;
                    wsum[g * NT + nt][j + 2] *= f;
                  }
                }
#pragma unroll
                for (int i = 0; i < NG * KS; ++i) {
                  o[i * NT + nt][j] *= f;
                  o[i * NT + nt][j + 2] *= f;
                }
              }
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const float m0 = (m[nt][0] == -INFINITY ? 0.f : m[nt][0]) - vexp[nt][0];
            const float m1 = (m[nt][1] == -INFINITY ? 0.f : m[nt][1]) - vexp[nt][1];
            s[nt][0] = ps_ex2(s[nt][0] - m0);
            s[nt][1] = ps_ex2(s[nt][1] - m1);
            s[nt][2] = ps_ex2(s[nt][2] - m0);
            s[nt][3] = ps_ex2(s[nt][3] - m1);
            l[nt][0] += s[nt][0] + s[nt][2];
            l[nt][1] += s[nt][1] + s[nt][3];
          }
          // ---- values
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            const float s0 = ps_half<F16>(sw[0], g), s1 = ps_half<F16>(sw[1], g);
            const float c0 = fmaf(MID, s0, ps_half<F16>(bw[0], g)), c1 = fmaf(MID, s1, ps_half<F16>(bw[1], g));
            uint32_t wt[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float w[4] = {s[nt][0] * s0, s[nt][1] * s0, s[nt][2] * s1, s[nt][3] * s1};
              if (!edge) {
                vb[g * NT + nt][0] = fmaf(s[nt][0], c0, fmaf(s[nt][2], c1, vb[g * NT + nt][0]));
                vb[g * NT + nt][1] = fmaf(s[nt][1], c0, fmaf(s[nt][3], c1, vb[g * NT + nt][1]));
              } else {   // a hidden key's scale and bias may be anything
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const bool no = (hidden >> (4 * nt + j)) & 1u;
                  w[j] = no ? 0.f : w[j];
                  vb[g * NT + nt][j & 1] += no ? 0.f : s[nt][j] * (j < 2 ? c0 : c1);
                }
              }
              wt[nt][0] = ps_trans(ps_h2(w[0], w[1]));
              wt[nt][1] = ps_trans(ps_h2(w[2], w[3]));
            }
            auto mul = [&](float (&acc)[4], int nt, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3) {
              ps_mma(acc, a0, a1, a2, a3, wt[nt][0], wt[nt][1], acc[0], acc[1], acc[2], acc[3]);
            };
            if constexpr (G::ONES) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mul(wsum[g * NT + nt], nt, MID_LO, MID_HI, MID_LO, MID_HI);
            }
            // this lane's codes: dimensions g GS + r8 GS / 8 ..., of keys 2 c4, 2 c4 + 1, 2 c4 + 8, 2 c4 + 9
            constexpr int VW = GS * BITS / 256;   // words per lane, group and key (0: half a word)
            uint32_t kw[4][VW ? VW : 1];
#pragma unroll
            for (int x = 0; x < 4; ++x)
              ps_words<VW>((vat ^ (g * GSB & 127) ^ ((x & 1) ? ODD : 0u) ^ ((x >> 1) ? UP8 : 0u)) + (g * GSB & ~127) +
                               (x & 1) * ODD_UP + (x >> 1) * 8 * RB, kw[x]);
            // pairs of keys: 16 bits of codes of either
            constexpr int PW = VW ? 2 * VW : 1;
            uint32_t pa[PW], pb[PW];   // keys (2 c4, 2 c4 + 1) and those 8 behind
#pragma unroll
            for (int i = 0; i < PW; ++i) {
              const uint32_t sel = VW && (i & 1) ? 0x7632u : 0x5410u;
              pa[i] = __byte_perm(kw[0][i / 2], kw[1][i / 2], sel);
              pb[i] = __byte_perm(kw[2][i / 2], kw[3][i / 2], sel);
            }
            // product j of the group: dimensions r8 GS / 8 + 2 j (rows 0-7) and + 2 j + 1 (rows 8-15)
#pragma unroll
            for (int j = 0; j < KS; ++j) {
              // 4-bit: a pair word holds four dimensions, two of them after a shift by 8; the odd ones count 16-fold (rows 8-15
              // are a dimension of their own: divided at the end). 8-bit: two dimensions
              uint32_t a[4];
              if constexpr (BITS == 4) {
                const uint32_t u = (j & 1) ? pa[j / 2] >> 8 : pa[j / 2], v = (j & 1) ? pb[j / 2] >> 8 : pb[j / 2];
                a[0] = u & 0x000F000Fu;
                a[1] = u & 0x00F000F0u;
                a[2] = v & 0x000F000Fu;
                a[3] = v & 0x00F000F0u;
              } else {
                a[0] = pa[j] & 0x00FF00FFu;
                a[1] = (pa[j] >> 8) & 0x00FF00FFu;
                a[2] = pb[j] & 0x00FF00FFu;
                a[3] = (pb[j] >> 8) & 0x00FF00FFu;
              }
              if constexpr (!G::ONES) {
#pragma unroll
                for (int x = 0; x < 4; ++x) a[x] = ps_sub2(a[x], (x & 1) ? MID_HI : MID_LO);
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mul(o[(g * KS + j) * NT + nt], nt, a[0], a[1], a[2], a[3]);
            }
          }
        }
        __syncwarp();   // the stage is read before it is filled again
        st = st + 1 == STAGES ? 0 : st + 1;
        first += STEP;
      }
      ps_wait<0>();

      // ---- the warps' results, 8 query rows at a time, through shared memory (the rings are empty now)
      const bool whole = j0 == 0 && j1 == nblk;
      const int slot = 2 * cta + (mine ? 1 : 0);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
#pragma unroll
          for (int sh = 4; sh <= 16; sh <<= 1) l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], sh);
          if (r8 == 0) {
            s_ml[nt][warp][0][2 * c4 + j] = m[nt][j];
            s_ml[nt][warp][1][2 * c4 + j] = l[nt][j] * ps_ex2(-vexp[nt][j]);
          }
        }
        __syncthreads();   // also: every warp is through with its ring (or with the last 8 rows)
        float f[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float M = -INFINITY;
#pragma unroll
          for (int w = 0; w < kPsWarps; ++w) M = fmaxf(M, s_ml[nt][w][0][2 * c4 + j]);
          f[j] = m[nt][j] == -INFINITY ? 0.f : ps_ex2(m[nt][j] - M - vexp[nt][j]);
        }
#pragma unroll
        for (int g = 0; g < NG; ++g) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float e = vb[g * NT + nt][j];
#pragma unroll
            for (int sh = 4; sh <= 16; sh <<= 1) e += __shfl_xor_sync(0xffffffffu, e, sh);
            e *= f[j];
            const float f0 = f[j] * GREAT, f1 = BITS == 4 ? f0 * 0.0625f : f0;
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              float* dst = comb + (warp * 8 + 2 * c4 + j) * D + g * GS + r8 * (GS / 8) + 2 * i;
              float x = o[(g * KS + i) * NT + nt][j], y = o[(g * KS + i) * NT + nt][j + 2];
              if constexpr (G::ONES) {
                x -= wsum[g * NT + nt][j];
                y -= wsum[g * NT + nt][j + 2];
              }
              *reinterpret_cast<float2*>(dst) = make_float2(fmaf(x, f0, e), fmaf(y, f1, e));
            }
          }
        }
        __syncthreads();
        // one warp per query row in turn: sum over the warps in order, lanes along the head dimension
        for (int q = warp; q < 8; q += kPsWarps) {
          const int r = nt * 8 + q;
          if (row0 + r >= t.s.rows) break;
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int w = 0; w < kPsWarps; ++w) M = fmaxf(M, s_ml[nt][w][0][q]);
#pragma unroll
          for (int w = 0; w < kPsWarps; ++w)
            L += s_ml[nt][w][0][q] == -INFINITY ? 0.f : s_ml[nt][w][1][q] * ps_ex2(s_ml[nt][w][0][q] - M);
          const int tok = (row0 + r) / p.nrep;
          uint32_t* dst = reinterpret_cast<uint32_t*>(
              p.out + ((long long)(t.s.first + tok) * p.H + t.unit * p.nrep + (row0 + r - tok * p.nrep)) * D);
          float* po = p.part_o + ((size_t)slot * MT + r) * D;
          const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
          for (int d = 0; d < D; d += 64) {
            float2 v = make_float2(0.f, 0.f);
#pragma unroll
            for (int w = 0; w < kPsWarps; ++w) {
              const float2 x = *reinterpret_cast<const float2*>(comb + (w * 8 + q) * D + d + 2 * lane);
              v.x += x.x;
              v.y += x.y;
            }
            if (whole) dst[(d >> 1) + lane] = ps_out2<F16>(v.x * inv, v.y * inv);
            else *reinterpret_cast<float2*>(po + d + 2 * lane) = v;
          }
          if (!whole && lane == 0) p.part_ml[(size_t)slot * MT + r] = make_float2(M, L);
        }
      }
      if (saw_absent && lane == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
    }
    __syncthreads();   // the tile and the combine area are read before the next tile overwrites them
    if (tid == 0 && (t.lo < s_x[0] || t.hi > s_x[1])) paged_record(p, pieces, t, MT, nblk, j0, j1, cta);
    if (tid == 0) s_more = s_x[1] > t.hi && paged_tile_next(p, MT, t);
    __syncthreads();
    if (!s_more) break;
  }
}

template <int BITS, int D, int GS, int NT, bool F16>
cudaError_t ps_run(const QdaPagedParams* p, int* ctas_per_sm, cudaStream_t s) {
  using G = PsGeom<BITS, D, GS, NT>;
  auto kern = qda_paged_split_kernel<BITS, D, GS, NT, F16>;
  if (ctas_per_sm != nullptr) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, G::SMEM);
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(ctas_per_sm, kern, kPsWarps * 32, G::SMEM);
    return e;
  }
  kern<<<p->ctas, kPsWarps * 32, G::SMEM, s>>>(*p);
  return cudaGetLastError();
}

template <int BITS, bool F16>
cudaError_t ps_pick(const QdaPagedParams* p, int D, int GS, int rows, int* occ, cudaStream_t s) {
#define QDA_PS(d, gs)                                                                   \
  if (D == d && GS == gs) {                                                             \
    if constexpr (d <= 256) {                                                           \
      if (rows > 8) return ps_run<BITS, d, gs, 2, F16>(p, occ, s);                      \
    }                                                                                   \
    return ps_run<BITS, d, gs, 1, F16>(p, occ, s);                                      \
  }
  QDA_PS(64, 32) QDA_PS(64, 64)
  QDA_PS(128, 32) QDA_PS(128, 64) QDA_PS(128, 128)
  QDA_PS(256, 32) QDA_PS(256, 64) QDA_PS(256, 128)
  QDA_PS(512, 32) QDA_PS(512, 64) QDA_PS(512, 128)
#undef QDA_PS
  return cudaErrorInvalidValue;
}

}  // namespace qda
