// Paged attention for many query rows per KV head (sm_103a): chunks of prompts, cross attention. Bound by the tensor cores.
//
// One CTA per SM takes a tile of 128 query rows of a KV head, or two of them side by side (D <= 128), and walks the tile's keys in blocks
// of 128: S = Q K^T and O += P V on tcgen05 (fp16 operands, fp32 sums in tensor memory), an online softmax in between. Rows are (token, query head)
// pairs, so all query heads of a KV head share a block's keys and values, which are turned from codes into operands once per block:
//   dequantising warps   codes -> fp16 tiles in shared memory (a ring of slots of 128 keys x 128 dimensions), next slot's codes in flight in registers;
//   softmax warps        one thread per query row: reads its row of S from tensor memory, writes P (fp16) over it;
//   MMA warp             one thread issues every product. With two tiles the products of one run while the softmax of the other does;
//                        with one tile S has two buffers and the next block's scores run during this block's softmax;
//   info warp            one block ahead: the block's pages, and how large its keys and values can be.
// Every link is an mbarrier; every wait is bounded and sets the device error word.
//
// Operands are fp16 for both input types (11 significant bits; for bf16 caches the operands then add almost nothing to the one
// rounding of the result, where bf16 operands would double it), and ranges are taken care of by powers of two: a query row is scaled so that its largest value
// lies in [2^8, 2^9), a block's keys and values so that none passes 2^-4 (2^-1 for 8-bit codes), from the block's scales and biases. The scale of the keys is undone with
// the softmax scale; that of the values only ever grows in a tile's walk and O is rescaled when it does. Small scale leaves no rounding behind: the
// codes enter the multiply-add as fp16 subnormals c 2^-24 (the code's bits as they are, one AND for two of them), so that one fused multiply-add with s 2^24 makes
// two operand values. The unpacked order of the dimensions is kept: q is stored in the same order and O read back in it.
// Hidden keys: beyond a row's sight -inf; behind the sequence, on an absent page, or not finite they are zero in the operands, so they reach nothing
// else, and a row that sees a key that is not finite becomes NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "qda_paged_sched.cuh"

namespace qda {

constexpr int kPcKeys = 128;     // keys per block
constexpr int kPcDeq = 8;        // dequantising warps
constexpr int kPcInfo = 8;       // blocks of info in flight

struct PcInfo {
  int pg[8];              // page of each 16 keys (-1: none or absent)
  float kmul;             // what undoes the keys' scale
  float kfac, vfac;       // the keys' and values' scale
  int kv;                 // values' scale is 2^-kv
  uint32_t flags;         // any bit of gone or bad
  uint32_t gone[4];       // keys on absent pages
  uint32_t bad[4];        // keys or values that are not finite
};

template <int D, int BITS, int NQ>
struct PcGeom {
  static constexpr int MT = 128 * NQ;
  static constexpr int SD = D < 128 ? D : 128;          // dimensions per slot
  static constexpr int DV = D < 256 ? D : 256;          // values' dimensions of a unit (TMEM holds O of no more)
  static constexpr int PARTS = D / DV;
  static constexpr int KSL = D / SD, VSL = DV / SD;     // slots of a block's keys and of its values
  static constexpr int SLOT = kPcKeys * SD * 2;
  static constexpr int QB = MT * D * 2;
  static constexpr int SLOTS0 = (226 * 1024 - 1024 - QB) / SLOT;
  static constexpr int SLOTS = SLOTS0 > 6 ? 6 : SLOTS0;
  static constexpr int SOFT = 4 * NQ;                   // softmax warps
  static constexpr int WARPS = SOFT + kPcDeq + 2;
  static constexpr int O_COL = 256;                     // O behind two S buffers of 128 columns
  static_assert(NQ == 1 || D <= 128, "two tiles need room for two O");
  static_assert(SLOTS >= 3 && O_COL + NQ * DV <= 512, "shared or tensor memory");
};

struct PcShared {
  PcInfo info[kPcInfo];
  uint64_t info_full[kPcInfo], info_empty[kPcInfo], full[6], empty[6], q_full, s_full[2], p_full[2], drain;
  uint64_t pv_done[2];   // one tile: values of even and odd blocks (a parity tells only neighbouring phases apart, and no more than two blocks are open)
  PagedTile t;
  long long x[2];
  uint32_t tmem;
  int abort, more;
};

template <int D, int BITS, int NQ>
constexpr int pc_smem() {
  using G = PcGeom<D, BITS, NQ>;
  return 1024 + G::QB + G::SLOTS * G::SLOT + (int)sizeof(PcShared);
}

__device__ __forceinline__ float pc_ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Shared-memory descriptor of a 128-byte swizzled operand (rows of 128 bytes, 8-row groups 1024 bytes apart); lbo: bytes between 64-element blocks of
// an operand whose rows run along K (values), unused for one whose rows hold K (keys, queries).
__device__ __forceinline__ uint64_t pc_desc(uint32_t saddr, uint32_t lbo) {
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)((lbo >> 4) & 0x3FFFu) << 16) | ((uint64_t)(1024u >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}

__device__ __forceinline__ void pc_mma_ss(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void pc_ld32(uint32_t taddr, float (&v)[32]) {
  uint32_t r[32];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
#pragma unroll
  for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void pc_st32(uint32_t taddr, const float (&v)[32]) {
  uint32_t a[16], b[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    a[i] = __float_as_uint(v[i]);
    b[i] = __float_as_uint(v[16 + i]);
  }
  tmem_st16(taddr, a);
  tmem_st16(taddr + 16, b);
}

__device__ __forceinline__ uint32_t pc_h2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ uint32_t pc_fma2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}

__device__ __forceinline__ float pc_half(uint32_t u16, bool f16) { return half_bits_to_float_rt(u16 & 0xffffu, f16); }

// Dimension at position i of 8 in the unpacked order.
template <int BITS>
__host__ __device__ constexpr int pc_dim(int i) {
  return BITS == 4 ? (i >> 1) + 4 * (i & 1) : (i & 4) + ((i & 3) >> 1) + 2 * (i & 1);
}

template <int D, int BITS, int NQ>
__global__ void __launch_bounds__(PcGeom<D, BITS, NQ>::WARPS * 32, 1)
    qda_paged_chunk_kernel(const __grid_constant__ QdaPagedParams p) {
  using G = PcGeom<D, BITS, NQ>;
  constexpr int MT = G::MT, SD = G::SD, DV = G::DV, KSL = G::KSL, VSL = G::VSL, SLOTS = G::SLOTS;
  constexpr float QMAX = (float)((1 << BITS) - 1);
  constexpr float FINITE = 1.329228e36f;   // 2^120: what is larger counts as not finite
  extern __shared__ __align__(1024) unsigned char pc_smem_raw[];
  unsigned char* base = pc_smem_raw + ((1024u - (smem_addr(pc_smem_raw) & 1023u)) & 1023u);
  unsigned char* q_s = base;
  unsigned char* ring = base + G::QB;
  PcShared& sh = *reinterpret_cast<PcShared*>(ring + SLOTS * G::SLOT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int W_DEQ = G::SOFT, W_MMA = G::SOFT + kPcDeq;   // and the info warp behind
  volatile int* abort = &sh.abort;

  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kPcInfo; ++i) {
      mbar_init(&sh.info_full[i], 1);
      mbar_init(&sh.info_empty[i], G::SOFT + kPcDeq);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&sh.full[i], kPcDeq);
      mbar_init(&sh.empty[i], 1);
    }
    mbar_init(&sh.q_full, G::SOFT);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 4);
      mbar_init(&sh.pv_done[i], 1);
    }
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_barrier_init();
  }
  PagedLine& line = *reinterpret_cast<PagedLine*>(ring);   // before the first slot is filled
  paged_line(p, MT, line);
  const long long total = line.at[p.B];
  if (total == 0) return;
  const int ctas = paged_ctas(total, p.ctas, p.min_keys), cta = blockIdx.x;
  if (cta >= ctas) return;
  if (warp == W_MMA) tmem_alloc(&sh.tmem, 512);
  if (tid == 0) {
    sh.x[0] = paged_border(total, ctas, cta);
    sh.x[1] = paged_border(total, ctas, cta + 1);
    sh.t = paged_tile_at(p, line, MT, sh.x[0]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int pmask = (1 << p.page_shift) - 1, Hkv = p.units / G::PARTS;
  uint32_t bc = 0, ic = 0, sc = 0, tc = 0;   // blocks, slots, s_full phases (two tiles) and tiles so far

  for (;;) {
    const PagedTile& t = sh.t;
    const int keys = paged_tile_keys(p, t, MT);
    const int nblk = (keys + kPcKeys - 1) / kPcKeys;
    const int j0 = paged_block_at(t, nblk, sh.x[0]), j1 = paged_block_at(t, nblk, sh.x[1]), n = j1 - j0;
    const bool mine = sh.x[0] <= t.lo;
    const int row0 = t.i * MT, kvh = t.unit / G::PARTS, part = t.unit % G::PARTS;
    // slots in the order of use: K(0), then K(j + 1), V(j)
    auto it_k = [&](int j) { return ic + (j == 0 ? 0 : KSL + (j - 1) * (KSL + VSL)); };
    auto it_v = [&](int j) { return ic + KSL + j * (KSL + VSL) + (j + 1 < n ? KSL : 0); };

    if (n > 0 || (nblk == 0 && mine)) {
      if (warp < G::SOFT) {
        // ================================================================================= softmax: a thread per row
        const int tq = warp >> 2;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const int rt = tq * 128 + 32 * (warp & 3) + lane;   // row of the tile
        const int r = row0 + rt;
        const bool real = r < t.s.rows;
        const int tok = r / p.nrep, head = kvh * p.nrep + (r - tok * p.nrep);
        const int seen = real ? paged_seen(p, t.s, r) : keys;
        float qmul = p.qscale;
        if (n > 0) {
          const uint4* qp = reinterpret_cast<const uint4*>(p.q + (long long)(t.s.first + tok) * p.q_tstride +
                                                           (long long)head * p.q_hstride);
          float top = 0.f;
          if (real) {
#pragma unroll 4
            for (int i = 0; i < D / 8; ++i) {
              const uint4 a = qp[i];
              const uint32_t u[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f = half2_bits_to_float2_rt(u[k], p.f16);
                top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
              }
            }
          }
          const int fe = min(262 - (int)((__float_as_uint(top) >> 23) & 255u), 253);
          const float up = __uint_as_float((uint32_t)fe << 23);
          qmul *= __uint_as_float((uint32_t)(254 - fe) << 23);
          unsigned char* dst = q_s + tq * 128 * D * 2 + (rt & 127) * 128;
#pragma unroll 4
          for (int i = 0; i < D / 8; ++i) {
            uint4 a = make_uint4(0, 0, 0, 0);
            if (real) a = qp[i];
            const uint32_t u[4] = {a.x, a.y, a.z, a.w};
            float v[8];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 f = half2_bits_to_float2_rt(u[k], p.f16);
              v[2 * k] = f.x * up;
              v[2 * k + 1] = f.y * up;
            }
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) w[k] = pc_h2(v[pc_dim<BITS>(2 * k)], v[pc_dim<BITS>(2 * k + 1)]);
            *reinterpret_cast<uint4*>(dst + (i >> 3) * 16384 + (((i & 7) ^ (rt & 7)) << 4)) =
                make_uint4(w[0], w[1], w[2], w[3]);
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.q_full);
        }
        float m = -INFINITY, l = 0.f;
        int kv = 0;
        bool poison = false;
        const uint32_t o_t = tmem + lanes + G::O_COL + tq * DV;
        for (int j = 0; j < n; ++j) {
          const uint32_t g = bc + j;
          const PcInfo& f = sh.info[g % kPcInfo];
          const int sb = NQ == 2 ? tq : (int)(g & 1);
          const uint32_t s_t = tmem + lanes + 128 * sb;
          mbar_wait_bounded(&sh.info_full[g % kPcInfo], (g / kPcInfo) & 1, abort, p.err, 1u);
          mbar_wait_bounded(&sh.s_full[sb], NQ == 2 ? (sc + j) & 1 : (g >> 1) & 1, abort, p.err, 1u);
          tc_fence_after();
          const float mult = qmul * f.kmul;
          const int kv_new = f.kv;
          const uint32_t flags = f.flags;
          const int key0 = (j0 + j) * kPcKeys;
          const bool edge = flags || __any_sync(0xffffffffu, key0 + kPcKeys > seen);
          float v[32];
          // a score that the row does not see becomes -inf
          auto mask = [&](int c) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (key0 + 32 * c + i >= seen) v[i] = -INFINITY;
            if (flags) {
              const uint32_t gone = f.gone[c], bad = f.bad[c];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                if ((gone >> i) & 1u) v[i] = -INFINITY;
                else if (((bad >> i) & 1u) && key0 + 32 * c + i < seen) poison = true;
              }
            }
          };
          float top = -INFINITY;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            pc_ld32(s_t + 32 * c, v);
            tmem_wait_ld();
            if (edge) mask(c);
#pragma unroll
            for (int i = 0; i < 32; i += 2) top = fmaxf(top, fmaxf(v[i], v[i + 1]));
          }
          top *= mult;   // mult > 0
          if (j == 0) kv = kv_new;
          if (__any_sync(0xffffffffu, top > m + 8.f) || kv_new != kv) {
            const float mn = fmaxf(m, top);
            const float a = mn == -INFINITY ? 1.f : pc_ex2(m - mn);
            m = mn;
            l *= a;
            if (j > 0) {
              if (NQ == 1) {   // the last block's values are in O (with two tiles the scores' barrier says so)
                mbar_wait_bounded(&sh.pv_done[(g - 1) & 1], ((g - 1) >> 1) & 1, abort, p.err, 1u);
                tc_fence_after();
              }
              const float x = a * pc_ex2((float)(kv - kv_new));
#pragma unroll 1
              for (int c = 0; c < DV / 32; ++c) {
                pc_ld32(o_t + 32 * c, v);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] *= x;
                pc_st32(o_t + 32 * c, v);
              }
            }
            kv = kv_new;
          }
          const float mm = m == -INFINITY ? 0.f : -m;
          float2 sum = make_float2(0.f, 0.f);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            pc_ld32(s_t + 32 * c, v);
            tmem_wait_ld();
            if (edge) mask(c);
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 e = __ffma2_rn(make_float2(v[2 * i], v[2 * i + 1]), make_float2(mult, mult), make_float2(mm, mm));
              const float2 x = make_float2(pc_ex2(e.x), pc_ex2(e.y));
              sum = __fadd2_rn(sum, x);
              w[i] = pc_h2(x.x, x.y);
            }
            tmem_st16(s_t + 16 * c, w);   // over scores that this thread has already read
          }
          l += sum.x + sum.y;
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.p_full[sb]);
            mbar_arrive(&sh.info_empty[g % kPcInfo]);
          }
        }
        // ---- the row's result
        const bool whole = j0 == 0 && j1 == nblk;
        float scale = 0.f;
        if (n > 0) {
          if (NQ == 2) {
            mbar_wait_bounded(&sh.s_full[tq], (sc + n) & 1, abort, p.err, 1u);
          } else {
            const uint32_t g = bc + n - 1;
            mbar_wait_bounded(&sh.pv_done[g & 1], (g >> 1) & 1, abort, p.err, 1u);
          }
          tc_fence_after();
          if (poison) l = __uint_as_float(0x7fc00000u);
          scale = pc_ex2((float)kv) * (whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f);
        }
        const size_t slot = (size_t)(2 * cta + (mine ? 1 : 0)) * MT + rt;
        uint4* out = reinterpret_cast<uint4*>(p.out + ((long long)(t.s.first + tok) * p.H + head) * D + part * DV);
        float4* po = reinterpret_cast<float4*>(p.part_o + slot * DV);
#pragma unroll 1
        for (int c = 0; c < DV / 32; ++c) {
          float v[32];
          if (n > 0) {
            pc_ld32(o_t + 32 * c, v);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
          float o[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float x = v[i];
            o[(i & ~7) + pc_dim<BITS>(i & 7)] = m == -INFINITY && !poison ? 0.f : x * scale;
          }
          if (!real) continue;
          if (whole) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float a = o[8 * k + 2 * i], b = o[8 * k + 2 * i + 1];
                if (p.f16) {
                  w[i] = pc_h2(a, b);
                } else {
                  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                  w[i] = *reinterpret_cast<const uint32_t*>(&h);
                }
              }
              out[4 * c + k] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) po[8 * c + k] = make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
        }
        if (real && !whole) p.part_ml[slot] = make_float2(m, l);
        tc_fence_before();
      } else if (warp < W_MMA) {
        // ======================================================================= codes -> fp16 tiles in shared memory
        constexpr int CPR = SD * BITS / 128;       // 16-byte pieces of codes per row of a slot
        constexpr int NCH = 128 * CPR / (kPcDeq * 32);
        constexpr int DPC = 128 / BITS;            // dimensions per piece
        constexpr int W = D * BITS / 32;
        const int id = tid - W_DEQ * 32;
        uint4 code[NCH];
        uint32_t sbv[NCH];                         // scale | bias << 16; both 0 where the key counts as zero
        int gshift = 31 - __clz(p.GS);
        const int items = n * (KSL + VSL);
        // item x of the walk: block, keys or values, slice of the dimensions
        auto what = [&](int x, int& j, bool& val, int& sl) {
          if (x < KSL) {
            j = 0;
            val = false;
            sl = x;
            return;
          }
          const int y = x - KSL, per = KSL + VSL;
          j = y / per;
          int z = y - j * per;
          if (j + 1 < n) {
            val = z >= KSL;
            sl = val ? z - KSL : z;
            if (!val) ++j;
          } else {
            val = true;
            sl = z;
          }
        };
        auto load = [&](int x) {
          int j, sl;
          bool val;
          what(x, j, val, sl);
          const uint32_t g = bc + j;
          mbar_wait_bounded(&sh.info_full[g % kPcInfo], (g / kPcInfo) & 1, abort, p.err, 1u);
          const PcInfo& f = sh.info[g % kPcInfo];
          const uint32_t* src = val ? p.vp : p.kp;
          const uint16_t *ss = val ? p.vs : p.ks, *bs = val ? p.vb : p.kb;
          const int d0 = val ? part * DV + sl * SD : sl * SD;
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const int at = i * (kPcDeq * 32) + id, row = at / CPR, q = at % CPR;
            const int key = (j0 + j) * kPcKeys + row, pg = f.pg[row >> 4];
            const bool ok = pg >= 0 && key < keys;
            const long long pr = qda_pool_row(ok ? pg : 0, kvh, ok ? key & pmask : 0, Hkv, p.page_shift);
            code[i] = __ldg(reinterpret_cast<const uint4*>(src + pr * W + d0 / (32 / BITS)) + q);
            const long long si = pr * p.NG + ((d0 + q * DPC) >> gshift);
            const uint32_t s = __ldg(ss + si), b = __ldg(bs + si);
            sbv[i] = ok ? s | b << 16 : 0u;
          }
        };
        if (items > 0) load(0);
        for (int x = 0; x < items; ++x) {
          int j, sl;
          bool val;
          what(x, j, val, sl);
          const uint32_t it = ic + x, slot = it % SLOTS, use = it / SLOTS;
          const float fac = val ? sh.info[(bc + j) % kPcInfo].vfac : sh.info[(bc + j) % kPcInfo].kfac;
          mbar_wait_bounded(&sh.empty[slot], (use & 1) ^ 1, abort, p.err, 1u);
          const uint32_t dst = smem_addr(ring) + slot * G::SLOT;
#pragma unroll
          for (int i = 0; i < NCH; ++i) {
            const int at = i * (kPcDeq * 32) + id, row = at / CPR, q = at % CPR;
            float s = pc_half(sbv[i], p.f16), b = pc_half(sbv[i] >> 16, p.f16);
            if (!(fmaf(fabsf(s), QMAX, fabsf(b)) < FINITE)) s = b = 0.f;
            const float s24 = s * fac * 16777216.f, bf = b * fac;
            const uint32_t s1 = pc_h2(s24, s24), s16 = pc_h2(s24 * 0.0625f, s24 * 0.0625f), b2 = pc_h2(bf, bf);
            const uint32_t cw[4] = {code[i].x, code[i].y, code[i].z, code[i].w};
            constexpr int PP = DPC / 8;   // 16-byte pieces of operand values
            // the order of the pieces differs between the halves of a row, so that eight lanes' stores meet all banks
            const int turn = SD == 128 ? (BITS == 4 ? (q >= 2 ? 2 : 0) : (q >= 4 ? 1 : 0)) : 0;
#pragma unroll
            for (int k = 0; k < PP; ++k) {
              uint32_t y[4];
              if constexpr (BITS == 4) {
                const uint32_t w = turn ? cw[k ^ 2] : cw[k];
                const uint32_t w8 = w >> 8;
                y[0] = pc_fma2(w & 0x000F000Fu, s1, b2);
                y[1] = pc_fma2(w & 0x00F000F0u, s16, b2);
                y[2] = pc_fma2(w8 & 0x000F000Fu, s1, b2);
                y[3] = pc_fma2(w8 & 0x00F000F0u, s16, b2);
              } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t w = turn ? cw[2 * (k ^ 1) + h] : cw[2 * k + h];
                  y[2 * h] = pc_fma2(w & 0x00FF00FFu, s1, b2);
                  y[2 * h + 1] = pc_fma2((w >> 8) & 0x00FF00FFu, s1, b2);
                }
              }
              const int piece = q * PP + (k ^ turn);
              const uint32_t a = dst + (piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                           : "memory");
            }
          }
          fence_proxy_async();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&sh.full[slot]);
            if (val && sl == VSL - 1) mbar_arrive(&sh.info_empty[(bc + j) % kPcInfo]);
          }
          if (x + 1 < items) load(x + 1);
        }
      } else if (warp == W_MMA) {
        // ============================================================================== one thread issues the products
        if (lane == 0 && n > 0) {
          const uint32_t id_qk = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | (8u << 24);                // M 128, N 128
          const uint32_t id_pv = (1u << 4) | (1u << 16) | ((uint32_t)(SD >> 3) << 17) | (8u << 24);   // M 128, N SD, B along N
          const uint32_t ring_a = smem_addr(ring), q_a = smem_addr(q_s);
          auto wait_slot = [&](uint32_t it) {
            mbar_wait_bounded(&sh.full[it % SLOTS], (it / SLOTS) & 1, abort, p.err, 1u);
            tc_fence_after();
          };
          // scores of tile tq from key slice sl in slot it
          auto qk = [&](int tq, int sl, uint32_t it, uint32_t d) {
#pragma unroll
            for (int k = 0; k < SD / 16; ++k) {
              const uint32_t off = (k >> 2) * 16384 + (k & 3) * 32;
              pc_mma_ss(d, pc_desc(q_a + tq * 128 * D * 2 + sl * 2 * 16384 + off, 16),
                        pc_desc(ring_a + (it % SLOTS) * G::SLOT + off, 16), id_qk, sl > 0 || k > 0);
            }
          };
          // O (+)= P V for value slice sl in slot it
          auto pv = [&](int sl, uint32_t it, uint32_t pt, uint32_t d, bool acc) {
#pragma unroll
            for (int k = 0; k < kPcKeys / 16; ++k)
              mma_f16_ts(d + sl * SD, pt + 8 * k, pc_desc(ring_a + (it % SLOTS) * G::SLOT + k * 2048, 16384), id_pv,
                         acc || k > 0);
          };
          mbar_wait_bounded(&sh.q_full, tc & 1, abort, p.err, 1u);
          tc_fence_after();
          if constexpr (NQ == 2) {
            wait_slot(it_k(0));
            for (int tq = 0; tq < 2; ++tq) {
              qk(tq, 0, it_k(0), tmem + 128 * tq);
              if (tq == 1) mma_commit(&sh.empty[it_k(0) % SLOTS]);
              mma_commit(&sh.s_full[tq]);
            }
            for (int j = 0; j < n; ++j) {
              for (int tq = 0; tq < 2; ++tq) {
                if (tq == 0) wait_slot(it_v(j));
                mbar_wait_bounded(&sh.p_full[tq], (bc + j) & 1, abort, p.err, 1u);
                tc_fence_after();
                pv(0, it_v(j), tmem + 128 * tq, tmem + G::O_COL + tq * DV, j > 0);
                if (tq == 1) mma_commit(&sh.empty[it_v(j) % SLOTS]);
                if (j + 1 < n) {
                  if (tq == 0) wait_slot(it_k(j + 1));
                  qk(tq, 0, it_k(j + 1), tmem + 128 * tq);
                  if (tq == 1) mma_commit(&sh.empty[it_k(j + 1) % SLOTS]);
                }
                mma_commit(&sh.s_full[tq]);   // the next scores are there, and this block's values in O
              }
            }
          } else {
            auto scores = [&](int j) {
              const uint32_t sb = (bc + j) & 1;
              for (int sl = 0; sl < KSL; ++sl) {
                wait_slot(it_k(j) + sl);
                qk(0, sl, it_k(j) + sl, tmem + 128 * sb);
                mma_commit(&sh.empty[(it_k(j) + sl) % SLOTS]);
              }
              mma_commit(&sh.s_full[sb]);
            };
            scores(0);
            for (int j = 0; j < n; ++j) {
              const uint32_t g = bc + j;
              if (j + 1 < n) scores(j + 1);
              mbar_wait_bounded(&sh.p_full[g & 1], (g >> 1) & 1, abort, p.err, 1u);
              tc_fence_after();
              for (int sl = 0; sl < VSL; ++sl) {
                wait_slot(it_v(j) + sl);
                pv(sl, it_v(j) + sl, tmem + 128 * (g & 1), tmem + G::O_COL, j > 0);
                mma_commit(&sh.empty[(it_v(j) + sl) % SLOTS]);
              }
              mma_commit(&sh.pv_done[g & 1]);
            }
          }
        }
        __syncwarp();
      } else {
        // ========================================================== pages and magnitudes of the blocks, a block ahead
        const int* tab = p.table + (size_t)t.b * p.max_pages;
        auto page_of = [&](int j) {   // lanes 0-7: the page of 16 keys
          const int k = (j0 + j) * kPcKeys + 16 * lane;
          return lane < 8 && j < n && k < keys ? __ldg(tab + (k >> p.page_shift)) : -1;
        };
        int next = n > 0 ? page_of(0) : -1;
        int kv_run = -126;
        const int nvec = 16 * p.NG;   // 16-byte pieces per array
        for (int j = 0; j < n; ++j) {
          const uint32_t g = bc + j;
          PcInfo& f = sh.info[g % kPcInfo];
          const int key0 = (j0 + j) * kPcKeys;
          int pg = next;
          next = page_of(j + 1);
          const bool asked = lane < 8 && key0 + 16 * lane < keys;
          const bool gone = asked && (unsigned)pg >= (unsigned)p.num_pages;
          if (gone) pg = -1;
          const uint32_t gone8 = __ballot_sync(0xffffffffu, gone);
          if (gone8 && lane == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
          mbar_wait_bounded(&sh.info_empty[g % kPcInfo], ((g / kPcInfo) & 1) ^ 1, abort, p.err, 1u);
          if (lane < 8) f.pg[lane] = pg;
          if (lane < 4) {
            f.gone[lane] = ((gone8 >> (2 * lane)) & 1u ? 0xffffu : 0u) | ((gone8 >> (2 * lane + 1)) & 1u ? 0xffff0000u : 0u);
            f.bad[lane] = 0u;
          }
          __syncwarp();
          float top[2] = {0.f, 0.f};
          bool any_bad = false;
#pragma unroll 2
          for (int v0 = 0; v0 < nvec; v0 += 32) {
            const int v = v0 + lane, g16 = min(v / (2 * p.NG), 7);
            const int pv = __shfl_sync(0xffffffffu, pg, g16);
            if (v < nvec && pv >= 0) {
              const int piece = v - g16 * 2 * p.NG;
              const long long row = qda_pool_row(pv, kvh, (key0 + 16 * g16) & pmask, Hkv, p.page_shift);
              const long long at = row * p.NG / 8 + piece;
              const uint4 a[4] = {__ldg(reinterpret_cast<const uint4*>(p.ks) + at), __ldg(reinterpret_cast<const uint4*>(p.kb) + at),
                                  __ldg(reinterpret_cast<const uint4*>(p.vs) + at), __ldg(reinterpret_cast<const uint4*>(p.vb) + at)};
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const uint32_t su[4] = {a[2 * x].x, a[2 * x].y, a[2 * x].z, a[2 * x].w};
                const uint32_t bu[4] = {a[2 * x + 1].x, a[2 * x + 1].y, a[2 * x + 1].z, a[2 * x + 1].w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int key = 16 * g16 + (piece * 8 + e) / p.NG;   // of the block
                  const float s = pc_half(su[e >> 1] >> (16 * (e & 1)), p.f16), b = pc_half(bu[e >> 1] >> (16 * (e & 1)), p.f16);
                  const float big = fmaf(fabsf(s), QMAX, fabsf(b));
                  if (key0 + key >= keys) continue;
                  if (big < FINITE) {
                    top[x] = fmaxf(top[x], big);
                  } else {
                    atomicOr(&f.bad[key >> 5], 1u << (key & 31));
                    any_bad = true;
                  }
                }
              }
            }
          }
          const uint32_t tk = __reduce_max_sync(0xffffffffu, __float_as_uint(top[0]));
          const uint32_t tv = __reduce_max_sync(0xffffffffu, __float_as_uint(top[1]));
          any_bad = __any_sync(0xffffffffu, any_bad);
          // largest magnitude to [2^T, 2^(T + 1)): the scale times 2^24 stays below 2^16
          constexpr int T = BITS == 4 ? -6 : -3;
          const int fk = max(1, min(254 + T - (int)(tk >> 23), 253)), fv = max(1, min(254 + T - (int)(tv >> 23), 253));
          kv_run = max(kv_run, 127 - fv);
          if (lane == 0) {
            f.kfac = __uint_as_float((uint32_t)fk << 23);
            f.kmul = __uint_as_float((uint32_t)(254 - fk) << 23);
            f.kv = kv_run;
            f.vfac = __uint_as_float((uint32_t)(127 - kv_run) << 23);
            f.flags = (gone8 != 0) | (any_bad ? 2u : 0u);
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh.info_full[g % kPcInfo]);
        }
      }
    }
    if (n > 0) {
      bc += n;
      ic += n * (KSL + VSL);
      sc += n + 1;
      ++tc;
    }
    __syncthreads();   // every warp is through with the tile
    if (tid == 0) sh.more = sh.x[1] > sh.t.hi && paged_tile_next(p, MT, sh.t);
    tc_fence_after();
    __syncthreads();
    if (!sh.more) break;
  }
  if (warp == W_MMA) {
    if (lane == 0) {   // no product is under way when the tensor memory goes back (after a wait that gave up some may be)
      volatile int none = 0;
      mma_commit(&sh.drain);
      mbar_wait_bounded(&sh.drain, 0, &none, p.err, 2u);
    }
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int BITS, int NQ>
cudaError_t pc_run(const QdaPagedParams* p, bool prepare, cudaStream_t s) {
  auto kern = qda_paged_chunk_kernel<D, BITS, NQ>;
  constexpr int smem = pc_smem<D, BITS, NQ>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  if (prepare) return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  kern<<<p->ctas, PcGeom<D, BITS, NQ>::WARPS * 32, smem, s>>>(*p);
  return cudaGetLastError();
}

template <int BITS>
cudaError_t pc_pick(const QdaPagedParams* p, int D, int tiles, bool prepare, cudaStream_t s) {
  switch (D) {
    case 64: return tiles == 2 ? pc_run<64, BITS, 2>(p, prepare, s) : pc_run<64, BITS, 1>(p, prepare, s);
    case 128: return tiles == 2 ? pc_run<128, BITS, 2>(p, prepare, s) : pc_run<128, BITS, 1>(p, prepare, s);
    case 256: return pc_run<256, BITS, 1>(p, prepare, s);
    case 512: return pc_run<512, BITS, 1>(p, prepare, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qda
