// Paged attention for many query rows per KV head (sm_103a): chunks of prompts, cross attention.
//
// One CTA per SM takes a tile of 128 query rows of a KV head, or two of them side by side (D <= 128), and walks the tile's
// keys in blocks of 128: S = Q K^T and O += P V on tcgen05 (fp16 operands, fp32 sums in tensor memory), an online softmax in
// between. Rows are (token, query head) pairs, so all query heads of a KV head share a block's keys and values, which are
// turned from codes into operands once per block:
//   dequantising warps   codes -> fp16 tiles in shared memory (a ring of slots of 128 keys x 128 dimensions), the next
//                        slot's codes in flight in registers;
//   softmax warps        eight: one thread per query row with two tiles, two threads (half of the keys, half of the values)
//                        with one. They read S from tensor memory and write P (fp16) over it;
//   MMA warp             one thread issues every product. With two tiles the products of one run while the softmax of the
//                        other does; with one tile S has two buffers and the next block's scores run during this block's
//                        softmax. Two threads per row took ragged chunks at D = 256 from 487 to 453 us (the lone softmax
//                        warp of a scheduler waited for itself);
//   info warps           blocks ahead: a block's pages, and how large its keys and values can be.
// Every link is an mbarrier; every wait is bounded and sets the device error word, and after one that gave up every role
// ends without an access that the call's arrays do not hold.
//
// Measured: 2048 tokens over 32768 keys (32 heads, 8 KV heads, D 128, 4-bit) 875 us, 1.22 PFLOP/s, 64 % of a large bf16
// product's rate. The tensor pipe and the issue slots are each busy half of the time there (52 and 54 %) and the warps wait
// for loads most (long_scoreboard 4.3 per issue): for scores from tensor memory and for codes, one item ahead. Ragged chunks
// at D 256, 8-bit, 432 us (0.56 PFLOP/s, tensor pipe 27 %, the same wait 5.6): one tile per CTA, so a block is dequantised for
// 128 rows only, and the cache is read from DRAM four times over. Cross attention at D 64 65 us (12 %, 6.9), 250 tokens over
// 4097 keys at D 512 100 us (21 %, 5.9).
//
// Operands are fp16 for both input types (11 significant bits; for bf16 caches the operands then add almost nothing to the
// one rounding of the result, where bf16 operands would double it), and ranges are taken care of by powers of two: a query
// row is scaled so that its largest value lies in [2^8, 2^9), a block's keys and values so that the largest that its scales
// and biases allow, scale * (2^bits - 1) + |bias|, lies in [2^-6, 2^-5) (4-bit codes) or [2^-3, 2^-2) (8-bit). Values down
// to 2^-8 (2^-11) of that keep their 11 bits, smaller ones lose a bit with every factor of two. The scale of the keys is
// undone with the softmax scale; that of the values only ever grows in a tile's walk and O is rescaled when it does. A small
// scale leaves no rounding behind: the codes enter the multiply-add as fp16 subnormals c 2^-24 (the code's bits as they are,
// one AND for two of them), so that one fused multiply-add with s 2^24 makes two operand values. The unpacked order of the
// dimensions is kept: q is stored in the same order and O read back in it.
// Hidden keys: beyond a row's sight -inf; behind the sequence, on an absent page, or not finite they are zero in the
// operands, so they reach nothing else, and a row that sees a key that is not finite becomes NaN. A finite key does choose
// the block's power of two for rows that do not see it: where that would cost them bits, the far kernel (qda_paged.cu) does
// those rows anew.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "qda_paged_sched.cuh"
#include "qda_paged_tc.cuh"

namespace qda {

constexpr int kPcKeys = 128;     // keys per block
constexpr int kPcInfo = 8;       // blocks of info in flight
constexpr int kPcTiles = 4;      // tiles in flight
constexpr int kPcInfoWarps = 3;  // info warps, taking blocks in turn (they fill up the last group of four warps)

constexpr uint32_t kPcNoRow = 0xffffffffu;

// Most powers of two that a query row, and a block's keys, are scaled up by. What undoes both, times the softmax scale
// (2^-4 and above), stays a normal number: hidden scores of -inf are multiplied by it, and zeros (a row, a block) would
// ask for any power. Values that these leave small make scores next to 0 with all that the other side may hold.
constexpr int kPcQUp = 63, kPcKUp = 57;

struct PcInfo {
  uint32_t row[8];        // pool row of each 16 keys (kPcNoRow: behind the sequence or on an absent page)
  float kmul;             // what undoes the keys' scale
  float kfac;             // the keys' scale
  int kv;                 // 2^-kv scales this block's values so; the walk takes the largest kv up to here
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
  static constexpr int SOFT = 8;                        // softmax warps
  static constexpr int DEQ = 8;                         // dequantising warps
  static constexpr int WARPS = SOFT + DEQ + 1 + kPcInfoWarps;
  // registers a thread: the launch's 96, dealt out anew among the warpgroups
  static constexpr int R_ALL = 96, R_SOFT = 136, R_DEQ = 72, R_LAST = 64;
  static_assert(SOFT * R_SOFT + DEQ * R_DEQ + 4 * R_LAST <= WARPS * R_ALL, "registers of the launch");
  // items of codes under way: a divisor of a block's items less one. More would cost the softmax warps their registers (453 us
  // of ragged chunks at D = 256 become 480 with 120 registers there, 720 with 104)
  static constexpr int AHEAD = 1;
  static constexpr int O_COL = 256;                     // O behind two S buffers of 128 columns
  static_assert(NQ == 1 || D <= 128, "two tiles need room for two O");
  static_assert(SLOTS >= 3 && O_COL + NQ * DV <= 512, "shared or tensor memory");
};

// A tile of this CTA's piece, and its part of the tile's key blocks.
struct PcTile {
  int n, j0;              // blocks j0 .. j0 + n - 1 (n = 0: a tile without keys, whose rows are zeros; -1: no more tiles)
  int keys;               // keys that the tile walks
  int whole, mine;        // all of the tile's blocks; the tile starts in this CTA's piece
  int row0, kvh, part, b;
  PagedSeq s;
};

struct PcShared {
  PcInfo info[kPcInfo];
  PcTile tile[kPcTiles];
  uint64_t info_full[kPcInfo], info_empty[kPcInfo], tile_full[kPcTiles], tile_empty[kPcTiles], full[6], empty[6], q_full,
      s_full[2], p_full[2], drain;
  uint64_t pv_done[2];    // two tiles: a tile's last values; one: values of even and odd blocks
  uint64_t pair[4];       // one tile: the two warps that share 32 rows
  float row[128];         // what they tell each other
  int rise[2][8];
  PagedTile t;
  long long x[2];
  uint32_t tmem;
  int abort, more;
};
// (A wait on a phase's parity tells neighbouring phases apart only: no barrier runs two phases ahead of a waiting role.)

template <int D, int BITS, int NQ>
constexpr int pc_smem() {
  using G = PcGeom<D, BITS, NQ>;
  return 1024 + G::QB + G::SLOTS * G::SLOT + (int)sizeof(PcShared);
}

// 8 columns of this thread's lane times x (rare; few registers, since the scores are being held)
__device__ __forceinline__ void pc_scale8(uint32_t taddr, float x) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * x);
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

__device__ __forceinline__ float pc_max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
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

// f(integral_constant<0>), ..., f(integral_constant<N - 1>)
template <int N, int I = 0, typename F>
__device__ __forceinline__ void pc_each(F&& f) {
  if constexpr (I < N) {
    f(std::integral_constant<int, I>{});
    pc_each<N, I + 1>(f);
  }
}

template <int D, int BITS, int NQ, bool LSE>
__global__ void __launch_bounds__(PcGeom<D, BITS, NQ>::WARPS * 32, 1)
    qda_paged_chunk_kernel(const __grid_constant__ QdaPagedParams p) {
  using G = PcGeom<D, BITS, NQ>;
  constexpr int DEQ = G::DEQ;
  constexpr int MT = G::MT, SD = G::SD, DV = G::DV, KSL = G::KSL, VSL = G::VSL, SLOTS = G::SLOTS;
  constexpr float QMAX = (float)((1 << BITS) - 1);
  constexpr float FINITE = 1.2980742e33f;   // 2^110: a scale or bias this large counts as not finite
  extern __shared__ __align__(1024) unsigned char pc_smem_raw[];
  unsigned char* base = pc_smem_raw + ((1024u - (smem_addr(pc_smem_raw) & 1023u)) & 1023u);
  unsigned char* q_s = base;
  unsigned char* ring = base + G::QB;
  PcShared& sh = *reinterpret_cast<PcShared*>(ring + SLOTS * G::SLOT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int W_DEQ = G::SOFT, W_MMA = G::SOFT + DEQ;   // the info warps behind
  volatile int* abort = &sh.abort;

  pdl_launch_dependents();
  if (tid == 0) {
    for (int i = 0; i < kPcInfo; ++i) {
      mbar_init(&sh.info_full[i], 1);
      mbar_init(&sh.info_empty[i], G::SOFT + DEQ);
    }
    for (int i = 0; i < SLOTS; ++i) {
      mbar_init(&sh.full[i], DEQ);
      mbar_init(&sh.empty[i], 1);
    }
    for (int i = 0; i < kPcTiles; ++i) {
      mbar_init(&sh.tile_full[i], 1);
      mbar_init(&sh.tile_empty[i], G::WARPS - 1);
      sh.tile[i].n = -1;
    }
    mbar_init(&sh.q_full, G::SOFT);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.s_full[i], 1);
      mbar_init(&sh.p_full[i], 8 / NQ);
      mbar_init(&sh.pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&sh.pair[i], 2);
    mbar_init(&sh.drain, 1);
    sh.abort = 0;
    fence_barrier_init();
  }
  // rows that a role may look up after a wait that gave up
  for (int i = tid; i < kPcInfo * 8; i += G::WARPS * 32) sh.info[i >> 3].row[i & 7] = kPcNoRow;
  PagedLine& line = *reinterpret_cast<PagedLine*>(ring);   // before the first slot is filled
  paged_line(p, MT, line);
  const int cta = blockIdx.x;
  const PagedPieces pieces = paged_pieces(p, line.at[p.B]);
  if (tid == 0) p.split[cta] = QdaPagedSplitTile{};
  if (cta >= pieces.ctas) return;
  if (warp == W_MMA) tmem_alloc(&sh.tmem, 512);
  if (tid == 0) {
    sh.x[0] = paged_border(pieces, cta);
    sh.x[1] = paged_border(pieces, cta + 1);
    sh.t = paged_tile_at(p, line, MT, sh.x[0]);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  const int pmask = (1 << p.page_shift) - 1, Hkv = p.units / G::PARTS;
  // blocks, slots and tiles with blocks so far: every role counts them for itself
  uint32_t bc = 0, ic = 0, tc = 0;
  auto wait = [&](uint64_t* bar, uint32_t phase) { return mbar_wait_bounded(bar, phase & 1u, abort, p.err, 1u); };
  // tile k of this CTA's piece (null behind the last); every warp hands it back with tile_done
  auto tile_at = [&](int k) -> const PcTile* {
    wait(&sh.tile_full[k % kPcTiles], k / kPcTiles);
    if (__any_sync(0xffffffffu, *abort != 0)) return nullptr;   // a wait gave up somewhere: every role ends
    const PcTile* t = &sh.tile[k % kPcTiles];
    return t->n < 0 ? nullptr : t;
  };
  auto tile_done = [&](int k) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh.tile_empty[k % kPcTiles]);
  };
  // slots of a tile of n blocks in the order of use: K(0), then K(j + 1), V(j)
  auto it_k = [&](int j) { return ic + (j == 0 ? 0 : KSL + (j - 1) * (KSL + VSL)); };
  auto it_v = [&](int j, int n) { return ic + KSL + j * (KSL + VSL) + (j + 1 < n ? KSL : 0); };

  if (warp < G::SOFT) {
    // =================================================================================== softmax: one or two threads per row
    pc_regs<G::R_SOFT, G::R_ALL>();
    // two tiles: a warpgroup each, a thread per row. One: two threads per row, in warps w and w + 4; each takes half of the
    // block's keys and half of the row's values
    const int tq = NQ == 2 ? warp >> 2 : 0, half = NQ == 2 ? 0 : warp >> 2;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int rt = tq * 128 + 32 * (warp & 3) + lane;   // row of the tile
    const uint32_t o_t = tmem + lanes + G::O_COL + tq * DV;
    uint32_t pairs = 0;
    auto pair_sync = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.pair[warp & 3]);
      wait(&sh.pair[warp & 3], pairs++);
    };
    // both threads of a row get f(the first one's x, the second one's)
    auto both = [&](float x, auto f) {
      if (half == 0) sh.row[rt] = x;
      pair_sync();
      if (half == 1) sh.row[rt] = x = f(sh.row[rt], x);
      pair_sync();
      return half == 0 ? sh.row[rt] : x;
    };
    // The warp's query rows into shared memory, in the codes' unpacked order, each row scaled by a power of two; returns what
    // undoes this thread's row's scale, times the softmax scale. With one tile a row is read by lanes side by side; with two
    // tiles (D <= 128) a thread reads its own row, which is slower by itself, but the other form costs the softmax loop
    // registers there (ragged chunks at D = 256: 575 against 622 us for the first form; chunk over 32768 keys at D = 128: 869
    // us with the second, 887 with the first).
    auto load_q = [&](const PcTile& t) {
      float mul = 0.f;
      // 8 values: their largest magnitude; and with `up` 16 bytes of operand
      auto values = [&](const uint4& a, float (&v)[8]) {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = half2_bits_to_float2_rt(w[k], p.f16);
          v[2 * k] = f.x;
          v[2 * k + 1] = f.y;
          top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        return top;
      };
      auto store = [&](const float (&v)[8], float up, int row, int piece) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) w[k] = pc_h2(v[pc_dim<BITS>(2 * k)] * up, v[pc_dim<BITS>(2 * k + 1)] * up);
        *reinterpret_cast<uint4*>(q_s + tq * 128 * D * 2 + (piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4)) =
            make_uint4(w[0], w[1], w[2], w[3]);
      };
      // exponent field of the power of two that brings `top` to [2^8, 2^9), as far as kPcQUp
      auto scale_of = [](float top) { return min(262 - (int)((__float_as_uint(top) >> 23) & 255u), 127 + kPcQUp); };
      auto row_at = [&](int r) {
        const int tok = r / p.nrep;
        return reinterpret_cast<const uint4*>(p.q + (long long)(t.s.first + tok) * p.q_tstride +
                                              (long long)(t.kvh * p.nrep + (r - tok * p.nrep)) * p.q_hstride);
      };
      if constexpr (NQ == 2) {
        const int r = t.row0 + rt;
        const bool real = r < t.s.rows;
        const uint4* qp = row_at(r);
        uint4 a[D / 8];
        float top = 0.f, v[8];
#pragma unroll
        for (int i = 0; i < D / 8; ++i) a[i] = real ? __ldg(qp + i) : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t u[4] = {a[i].x, a[i].y, a[i].z, a[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = half2_bits_to_float2_rt(u[k], p.f16);
            top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
          }
        }
        const int fe = scale_of(top);
        const float up = __uint_as_float((uint32_t)fe << 23);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          values(a[i], v);
          store(v, up, rt & 127, i);
        }
        mul = __uint_as_float((uint32_t)(254 - fe) << 23);
      } else {
        constexpr int LPR = D < 256 ? D / 8 : 32;   // lanes per row, 16 bytes each
        constexpr int RPI = 32 / LPR;               // rows at a time
        constexpr int C = D / 8 / LPR;              // pieces per lane
        constexpr int U = 8 / C < 16 / RPI ? 8 / C : 16 / RPI;   // row groups in flight
        const int row0 = 32 * (warp & 3) + 16 * half;            // the warp's 16 rows
        const int sub = lane / LPR, l = lane % LPR;
        pair_sync();                                // the other warp has read what `both` left in sh.row
#pragma unroll 1
        for (int g0 = 0; g0 < 16 / RPI; g0 += U) {
          uint4 a[U][C];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int r = t.row0 + row0 + (g0 + u) * RPI + sub;
            const uint4* qp = row_at(r);
#pragma unroll
            for (int c = 0; c < C; ++c) a[u][c] = r < t.s.rows ? __ldg(qp + l + 32 * c) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float v[C][8], top = 0.f;
#pragma unroll
            for (int c = 0; c < C; ++c) top = fmaxf(top, values(a[u][c], v[c]));
#pragma unroll
            for (int o = LPR / 2; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int fe = scale_of(top);
#pragma unroll
            for (int c = 0; c < C; ++c)
              store(v[c], __uint_as_float((uint32_t)fe << 23), row0 + (g0 + u) * RPI + sub, l + 32 * c);
            if (l == 0) sh.row[row0 + (g0 + u) * RPI + sub] = __uint_as_float((uint32_t)(254 - fe) << 23);
          }
        }
        pair_sync();
        mul = sh.row[rt];
        pair_sync();
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.q_full);
      return p.qscale * mul;
    };

    const PcTile* t = tile_at(0);
    float qmul_next = t != nullptr && t->n > 0 ? load_q(*t) : 0.f;
    for (int k = 0; t != nullptr; ++k) {
      const float qmul = qmul_next;
      const int n = t->n, r = t->row0 + rt;
      const bool real = r < t->s.rows;
      const int seen = real ? paged_seen(p, t->s, r) : t->keys;
      float m = -INFINITY, l = 0.f;
      int kv = 0;
      bool poison = false;
      for (int j = 0; j < n; ++j) {
        const uint32_t g = bc + j;
        const PcInfo& f = sh.info[g % kPcInfo];
        const int sb = NQ == 2 ? tq : (int)(g & 1);
        const uint32_t s_t = tmem + lanes + 128 * sb;
        wait(&sh.info_full[g % kPcInfo], g / kPcInfo);
        wait(&sh.s_full[sb], NQ == 2 ? g : g >> 1);
        tc_fence_after();
        const float mult = qmul * f.kmul;
        const int kv_new = j == 0 ? f.kv : max(kv, f.kv);
        const uint32_t flags = f.flags;
        const int left = seen - (t->j0 + j) * kPcKeys;   // keys of the block that the row sees
        const bool edge = __any_sync(0xffffffffu, left < kPcKeys);
        if (flags) {   // rare: keys on absent pages are hidden; who sees a key that is not finite becomes NaN
#pragma unroll 1
          for (int c = 4 * half; c < (NQ == 2 ? 8 : 4 * half + 4); ++c) {
            const uint32_t gone = f.gone[c >> 1] >> (16 * (c & 1)), bad = f.bad[c >> 1] >> (16 * (c & 1));
            float v[16];
            pc_ld16(s_t + 16 * c, v);
            tmem_wait_ld();
            uint32_t y[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const bool no = (gone >> i) & 1u;
              if (!no && ((bad >> i) & 1u) && 16 * c + i < left) poison = true;
              y[i] = no ? 0xff800000u : __float_as_uint(v[i]);
            }
            tmem_st16(s_t + 16 * c, y);
          }
          tmem_wait_st();
        }
        // a new reference (and unit) for the row's sums: O is rescaled with them
        auto rescale = [&](float top) {
          const float mn = fmaxf(m, top);
          const float a = mn == -INFINITY ? 1.f : pc_ex2(m - mn);
          m = mn;
          l *= a;
          if (j > 0) {
            if (NQ == 1) {   // the last block's values are in O (with two tiles the scores' barrier says so)
              wait(&sh.pv_done[(g - 1) & 1], (g - 1) >> 1);
              tc_fence_after();
            }
            const float x = a * pc_ex2((float)(kv - kv_new));
#pragma unroll 1
            for (int c = half * (DV / 16); c < (NQ == 2 ? DV / 8 : (half + 1) * (DV / 16)); ++c) pc_scale8(o_t + 8 * c, x);
          }
          kv = kv_new;
        };
        // Two tiles: the row's 128 scores do not fit the registers next to everything else: the second half is read for its
        // maximum, the first is read and kept, and the second read again as the first's registers come free. Weights lie
        // over the first half's scores.
        float u[2][32];
        auto get = [&](float (&x)[32], int c) { pc_ld32(s_t + 64 * half + 32 * c, x); };
        auto hide = [&](float (&x)[32], int c) {
          if (edge) {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (32 * c + i >= left - 64 * half) x[i] = -INFINITY;
          }
        };
        auto largest = [&](const float (&x)[32]) {
          float a = pc_max3(x[0], x[1], x[2]), b = pc_max3(x[3], x[4], x[5]);
#pragma unroll
          for (int i = 6; i < 30; i += 4) {
            a = pc_max3(a, x[i], x[i + 1]);
            b = pc_max3(b, x[i + 2], x[i + 3]);
          }
          return fmaxf(pc_max3(a, b, x[30]), x[31]);
        };
        float top = -INFINITY;
        if constexpr (NQ == 2) {
          get(u[0], 2);
          get(u[1], 3);
          tmem_wait_ld();
          hide(u[0], 2);
          hide(u[1], 3);
          top = fmaxf(largest(u[0]), largest(u[1]));
        }
        get(u[0], 0);
        get(u[1], 1);
        tmem_wait_ld();
        hide(u[0], 0);
        hide(u[1], 1);
        top = pc_max3(top, largest(u[0]), largest(u[1])) * mult;   // mult > 0
        if (j == 0) kv = kv_new;
        bool rise = __any_sync(0xffffffffu, top > m + 8.f || kv_new != kv);
        if constexpr (NQ == 1) {
          // does the other half of any row rise? Behind this both halves hold their scores in registers and weights may lie
          // over them
          tc_fence_before();
          if (lane == 0) sh.rise[g & 1][warp] = rise;
          pair_sync();
          tc_fence_after();
          rise = rise || sh.rise[g & 1][warp ^ 4] != 0;
          if (rise) top = both(top, [](float x, float y) { return fmaxf(x, y); });
        }
        if (rise) rescale(top);
        // weights times 2^7: up to 2^15, so that those far below the reference keep their bits longer, 11 of them down to
        // 2^-21 (the sum has the same factor)
        const float mm = m == -INFINITY ? 0.f : kPcWeightBits - m;
        float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        auto weigh = [&](const float (&x)[32], int c) {
          uint32_t w[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 e = __ffma2_rn(make_float2(x[2 * i], x[2 * i + 1]), make_float2(mult, mult), make_float2(mm, mm));
            const float2 y = make_float2(pc_ex2(e.x), pc_ex2(e.y));
            sum[i & 1] = __fadd2_rn(sum[i & 1], y);
            w[i] = pc_h2(y.x, y.y);
          }
          tmem_st16(s_t + 32 * half + 16 * c, w);
        };
        weigh(u[0], 0);
        if (NQ == 2) get(u[0], 2);
        weigh(u[1], 1);
        if constexpr (NQ == 2) {
          tmem_wait_ld();
          get(u[1], 3);
          hide(u[0], 2);
          weigh(u[0], 2);
          tmem_wait_ld();
          hide(u[1], 3);
          weigh(u[1], 3);
        }
        l += (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.p_full[sb]);
          mbar_arrive(&sh.info_empty[g % kPcInfo]);
        }
      }
      // the next tile's queries, while the last values are summed: every score of this tile is done
      const PcTile* next = tile_at(k + 1);
      qmul_next = next != nullptr && next->n > 0 ? load_q(*next) : 0.f;
      // ---- the row's result
      float scale = 0.f;
      if (n > 0) {
        const uint32_t g = bc + n - 1;
        if (NQ == 2) wait(&sh.pv_done[tq], tc);
        else wait(&sh.pv_done[g & 1], g >> 1);
        tc_fence_after();
        if (poison) l = __uint_as_float(0x7fc00000u);
        if (NQ == 1) l = both(l, [](float x, float y) { return x + y; });
        scale = pc_ex2((float)kv) * (t->whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f);
      }
      const bool whole = t->whole;
      const bool none = m == -INFINITY && l == l;   // the row saw no key
      const int tok = r / p.nrep;
      // (an instance of its own for calls that want it, and the approximate logarithm: in the one kernel for all calls the
      // registers cost the softmax loop 3 to 5 % of the chunk over 32768 keys)
      if constexpr (LSE) {
        if (real && whole && half == 0 && t->part == 0)
          p.lse[(long long)(t->s.first + tok) * p.H + t->kvh * p.nrep + (r - tok * p.nrep)] =
              l == 0.f ? -INFINITY : (m - kPcWeightBits + pc_lg2(l)) * 0.693147180559945309f;
      }
      const size_t slot = (size_t)(2 * cta + t->mine) * MT + rt;
      uint4* out = reinterpret_cast<uint4*>(
          p.out + ((long long)(t->s.first + tok) * p.H + t->kvh * p.nrep + (r - tok * p.nrep)) * D + t->part * DV);
      float4* po = reinterpret_cast<float4*>(p.part_o + slot * DV);
#pragma unroll 1
      for (int c = half * (DV / 64); c < (NQ == 2 ? DV / 32 : (half + 1) * (DV / 64)); ++c) {
        float v[2][16];
        if (n > 0) {
          pc_ld16(o_t + 32 * c, v[0]);
          pc_ld16(o_t + 32 * c + 16, v[1]);
          tmem_wait_ld();
        }
        float o[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) o[(i & ~7) + pc_dim<BITS>(i & 7)] = none ? 0.f : v[i >> 4][i & 15] * scale;
        if (!real) continue;
        if (whole) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t y[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = o[8 * x + 2 * i], b = o[8 * x + 2 * i + 1];
              if (p.f16) {
                y[i] = pc_h2(a, b);
              } else {
                const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
                y[i] = *reinterpret_cast<const uint32_t*>(&h);
              }
            }
            out[4 * c + x] = make_uint4(y[0], y[1], y[2], y[3]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 8; ++x) po[8 * c + x] = make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
        }
      }
      if (real && !whole && half == 0) p.part_ml[slot] = make_float2(m, l);
      tc_fence_before();
      bc += n;
      tc += n > 0;
      tile_done(k);
      t = next;
    }
  } else if (warp < W_MMA) {
    // ========================================================================= codes -> fp16 tiles in shared memory
    pc_regs<G::R_DEQ, G::R_ALL>();
    constexpr int UPR = SD / 32;               // units of 32 codes (which share a scale) per row of a slot
    constexpr int NU = 128 * UPR / (DEQ * 32);
    constexpr int UW = BITS;                   // words of codes per unit
    constexpr int ROWB = D * BITS / 8;         // bytes of codes per row
    constexpr int AHEAD = G::AHEAD;            // items whose codes are under way
    const int id = tid - W_DEQ * 32;
    const int row = id / UPR, q = id % UPR;    // this thread's units: unit q of rows row, row + threads / UPR, ...
    const int gshift = 31 - __clz(p.GS);
    const uint32_t sstride = p.NG * 2;
    // where a unit's four 16-byte pieces of operand go in a slot: rows of 64 values, pieces XORed by the row. The order of the
    // pieces differs between the halves of a row, so that eight lanes' stores meet all banks
    const int turn = UPR == 4 && q >= 2 ? 2 : 0;
    uint32_t to[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int piece = q * 4 + (u ^ turn);
      to[u] = (piece >> 3) * 16384 + row * 128 + (((piece & 7) ^ (row & 7)) << 4);
    }
    struct Item {
      uint32_t code[NU][UW];
      uint32_t s[NU], b[NU];                   // as they are in memory: nothing waits for a load before its item's turn
      uint32_t ok;                             // bit per unit: the key counts (else it is zero)
    };
    // The slots of a tile come in groups g = -1 ... n - 1 of KSL + VSL items: the keys of block g + 1, the values of block g
    // (where there are such). Items are loaded AHEAD items before they are converted.
    constexpr int P = KSL + VSL;
    static_assert(P % (AHEAD + 1) == 0, "an item's registers are known at compile time");
    Item reg[AHEAD + 1];
    for (int k = 0;; ++k) {
      const PcTile* t = tile_at(k);
      if (t == nullptr) break;
      const int n = t->n, left0 = t->keys - t->j0 * kPcKeys;
      const int vd0 = t->part * DV + 32 * q;
      const char* ksrc = reinterpret_cast<const char*>(p.kp) + 4 * BITS * q;
      const char* vsrc = reinterpret_cast<const char*>(p.vp) + vd0 * BITS / 8;
      uint32_t prk[NU], prv[NU], okk = 0, okv = 0;   // pool rows of the block whose keys were loaded last, and of the one before
#pragma unroll
      for (int i = 0; i < NU; ++i) prk[i] = prv[i] = 0;
      int kv_run = -126;
      uint32_t at = ic;                              // slots so far
      auto load = [&](auto item, int g) {
        constexpr int X = decltype(item)::value;
        constexpr bool VAL = X >= KSL;
        constexpr int SL = VAL ? X - KSL : X;
        if (VAL ? g < 0 : g + 1 >= n) return;
        Item& it = reg[X % (AHEAD + 1)];
        if constexpr (X == 0) {
          const uint32_t x = bc + g + 1;
          const PcInfo& f = sh.info[x % kPcInfo];
          wait(&sh.info_full[x % kPcInfo], x / kPcInfo);
          const int left = left0 - (g + 1) * kPcKeys;
          okv = okk;
          okk = 0;
#pragma unroll
          for (int i = 0; i < NU; ++i) {
            const int r = row + i * (DEQ * 32 / UPR);
            const uint32_t base = f.row[r >> 4];
            const bool ok = base != kPcNoRow && r < left;
            prv[i] = prk[i];
            prk[i] = ok ? base + (r & 15) : 0u;
            okk |= (uint32_t)ok << i;
          }
        } else if constexpr (X == KSL) {
          if (g + 1 >= n) {   // the last group has no keys: its values are of the block whose keys came last
            okv = okk;
#pragma unroll
            for (int i = 0; i < NU; ++i) prv[i] = prk[i];
          }
        }
        const uint32_t goff = (((VAL ? vd0 : 32 * q) + SL * SD) >> gshift) * 2;
        const char* src = (VAL ? vsrc : ksrc) + SL * SD * BITS / 8;
        const char* ss = reinterpret_cast<const char*>(VAL ? p.vs : p.ks) + goff;
        const char* bs = reinterpret_cast<const char*>(VAL ? p.vb : p.kb) + goff;
        it.ok = VAL ? okv : okk;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          const uint32_t pr = VAL ? prv[i] : prk[i];
          const uint4* c = reinterpret_cast<const uint4*>(src + (uint64_t)pr * ROWB);
#pragma unroll
          for (int u = 0; u < UW / 4; ++u) {
            const uint4 v = __ldg(c + u);
            it.code[i][4 * u] = v.x;
            it.code[i][4 * u + 1] = v.y;
            it.code[i][4 * u + 2] = v.z;
            it.code[i][4 * u + 3] = v.w;
          }
          it.s[i] = __ldg(reinterpret_cast<const uint16_t*>(ss + (uint64_t)pr * sstride));
          it.b[i] = __ldg(reinterpret_cast<const uint16_t*>(bs + (uint64_t)pr * sstride));
        }
      };
      auto convert = [&](auto item, int g) {
        constexpr int X = decltype(item)::value;
        constexpr bool VAL = X >= KSL;
        constexpr int SL = VAL ? X - KSL : X;
        if (VAL ? g < 0 : g + 1 >= n) return;
        const Item& it = reg[X % (AHEAD + 1)];
        const PcInfo& f = sh.info[(bc + g + (VAL ? 0 : 1)) % kPcInfo];
        if constexpr (VAL && SL == 0) kv_run = max(kv_run, f.kv);
        const float fac = VAL ? __uint_as_float((uint32_t)(127 - kv_run) << 23) : f.kfac;
        const bool odd = f.flags & 2u;
        const uint32_t slot = at % SLOTS;
        wait(&sh.empty[slot], at / SLOTS + 1);
        ++at;
        const uint32_t dst = smem_addr(ring) + slot * G::SLOT;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          float s, b;
          if (p.f16) {
            s = fp16_bits_to_float(it.s[i]);
            b = fp16_bits_to_float(it.b[i]);
          } else {
            s = __uint_as_float(it.s[i] << 16);
            b = __uint_as_float(it.b[i] << 16);
          }
          if (!((it.ok >> i) & 1u) || (odd && !(fmaxf(fabsf(s), fabsf(b)) < FINITE))) s = b = 0.f;
          s *= fac;
          b *= fac;
          const uint32_t s1 = pc_h2(s * 16777216.f, s * 16777216.f), s16 = pc_h2(s * 1048576.f, s * 1048576.f), b2 = pc_h2(b, b);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t y[4];
            if constexpr (BITS == 4) {
              const uint32_t w = turn ? it.code[i][u ^ 2] : it.code[i][u];
              const uint32_t w8 = w >> 8;
              y[0] = pc_fma2(w & 0x000F000Fu, s1, b2);
              y[1] = pc_fma2(w & 0x00F000F0u, s16, b2);
              y[2] = pc_fma2(w8 & 0x000F000Fu, s1, b2);
              y[3] = pc_fma2(w8 & 0x00F000F0u, s16, b2);
            } else {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint32_t w = turn ? it.code[i][2 * (u ^ 2) + h] : it.code[i][2 * u + h];
                y[2 * h] = pc_fma2(w & 0x00FF00FFu, s1, b2);
                y[2 * h + 1] = pc_fma2((w >> 8) & 0x00FF00FFu, s1, b2);
              }
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(dst + to[u] + i * (DEQ * 32 / UPR) * 128),
                         "r"(y[0]), "r"(y[1]), "r"(y[2]), "r"(y[3])
                         : "memory");
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.full[slot]);
          if (VAL && SL == VSL - 1) mbar_arrive(&sh.info_empty[(bc + g) % kPcInfo]);
        }
      };
      if (n > 0) {
        pc_each<AHEAD>([&](auto item) { load(item, -1); });
        for (int g = -1; g < n; ++g)
          pc_each<P>([&](auto item) {
            constexpr int NEXT = decltype(item)::value + AHEAD;
            load(std::integral_constant<int, NEXT % P>{}, g + NEXT / P);
            convert(item, g);
          });
      }
      bc += n;
      ic += n * P;
      tile_done(k);
    }
  } else {
   pc_regs<G::R_LAST, G::R_ALL>();
   if (warp == W_MMA) {
    // ================================================================================ one thread issues the products
    constexpr uint32_t ID_QK = (1u << 4) | ((uint32_t)(128 >> 3) << 17) | (8u << 24);               // M 128, N 128
    constexpr uint32_t ID_PV = (1u << 4) | (1u << 16) | ((uint32_t)(SD >> 3) << 17) | (8u << 24);   // M 128, N SD, B along N
    const uint32_t one = pc_elect();
    const uint32_t ring_a = smem_addr(ring), q_a = smem_addr(q_s);
    for (int k = 0;; ++k) {
      const PcTile* t = tile_at(k);
      if (t == nullptr) break;
      const int n = t->n;
      if (n > 0) {
        auto wait_slot = [&](uint32_t it) {
          wait(&sh.full[it % SLOTS], it / SLOTS);
          tc_fence_after();
        };
        // scores of tile tq from key slice sl in slot it: 32 bytes of K per product, 64 values per 128-byte row
        auto qk = [&](int tq, int sl, uint32_t it, uint32_t d) {
          const uint64_t a = pc_desc(q_a + tq * 128 * D * 2 + sl * 2 * 16384, 16);
          const uint64_t b = pc_desc(ring_a + (it % SLOTS) * G::SLOT, 16);
#pragma unroll
          for (int x = 0; x < SD / 16; ++x) {
            const uint32_t off = ((x >> 2) * 16384 + (x & 3) * 32) >> 4;
            pc_mma_ss(one, d, a + off, b + off, ID_QK, sl > 0 || x > 0);
          }
        };
        // O (+)= P V for value slice sl in slot it: 16 keys per product
        auto pv = [&](int sl, uint32_t it, uint32_t pt, uint32_t d, bool acc) {
          const uint64_t b = pc_desc(ring_a + (it % SLOTS) * G::SLOT, 16384);
#pragma unroll
          for (int x = 0; x < kPcKeys / 16; ++x)
            pc_mma_ts(one, d + sl * SD, pt + 8 * x, b + x * (2048 >> 4), ID_PV, acc || x > 0);
        };
        wait(&sh.q_full, tc);
        tc_fence_after();
        if constexpr (NQ == 2) {
          wait_slot(it_k(0));
          for (int tq = 0; tq < 2; ++tq) {
            qk(tq, 0, it_k(0), tmem + 128 * tq);
            if (tq == 1) pc_commit(one, &sh.empty[it_k(0) % SLOTS]);
            pc_commit(one, &sh.s_full[tq]);
          }
          for (int j = 0; j < n; ++j) {
#pragma unroll
            for (int tq = 0; tq < 2; ++tq) {
              if (tq == 0) wait_slot(it_v(j, n));
              wait(&sh.p_full[tq], bc + j);
              tc_fence_after();
              pv(0, it_v(j, n), tmem + 128 * tq, tmem + G::O_COL + tq * DV, j > 0);
              if (tq == 1) pc_commit(one, &sh.empty[it_v(j, n) % SLOTS]);
              if (j + 1 < n) {
                if (tq == 0) wait_slot(it_k(j + 1));
                qk(tq, 0, it_k(j + 1), tmem + 128 * tq);
                if (tq == 1) pc_commit(one, &sh.empty[it_k(j + 1) % SLOTS]);
                pc_commit(one, &sh.s_full[tq]);   // the next scores are there, and this block's values in O
              } else {
                pc_commit(one, &sh.pv_done[tq]);
              }
            }
          }
        } else {
          auto scores = [&](int j) {
            const uint32_t g = bc + j;
            for (int sl = 0; sl < KSL; ++sl) {
              wait_slot(it_k(j) + sl);
              qk(0, sl, it_k(j) + sl, tmem + 128 * (g & 1));
              pc_commit(one, &sh.empty[(it_k(j) + sl) % SLOTS]);
            }
            pc_commit(one, &sh.s_full[g & 1]);
          };
          scores(0);
          for (int j = 0; j < n; ++j) {
            const uint32_t g = bc + j;
            if (j + 1 < n) scores(j + 1);
            wait(&sh.p_full[g & 1], g >> 1);
            tc_fence_after();
            for (int sl = 0; sl < VSL; ++sl) {
              wait_slot(it_v(j, n) + sl);
              pv(sl, it_v(j, n) + sl, tmem + 128 * (g & 1), tmem + G::O_COL, j > 0);
              pc_commit(one, &sh.empty[(it_v(j, n) + sl) % SLOTS]);
            }
            pc_commit(one, &sh.pv_done[g & 1]);
          }
        }
      }
      __syncwarp();
      bc += n;
      ic += n * (KSL + VSL);
      tc += n > 0;
      tile_done(k);
    }
   } else {
    // ================================================ the piece's tiles, and pages and magnitudes of the blocks, ahead
    const int first = warp - W_MMA - 1;
    const int nvec = 16 * p.NG;   // 16-byte pieces per array
    bool more = true;             // first info warp: sh.t is a tile of this piece
    for (int k = 0;; ++k) {
      if (first == 0) {
        // the next tile with work for this CTA
        // (a role that gave up may still be at the tile before: it stays as it is, and every role ends)
        if (!wait(&sh.tile_empty[k % kPcTiles], k / kPcTiles + 1)) break;
        PcTile& e = sh.tile[k % kPcTiles];
        int n = -1;
        while (more && n < 0) {
          const PagedTile& t = sh.t;
          const int keys = paged_tile_keys(p, t, MT);
          const int nblk = (keys + kPcKeys - 1) / kPcKeys;
          const int j0 = paged_block_at(t, nblk, sh.x[0]), j1 = paged_block_at(t, nblk, sh.x[1]);
          const bool mine = sh.x[0] <= t.lo;   // the CTA that starts the tile writes it if it has no keys
          if (j1 > j0 || (nblk == 0 && mine)) {
            n = j1 - j0;
            if (lane == 0) {
              e.n = n;
              e.j0 = j0;
              e.keys = keys;
              e.whole = j0 == 0 && j1 == nblk;
              e.mine = mine;
              e.row0 = t.i * MT;
              e.kvh = t.unit / G::PARTS;
              e.part = t.unit % G::PARTS;
              e.b = t.b;
              e.s = t.s;
            }
            // the softmax warps read the tile's queries when they are done with the tile before: on their way to L2 until then
            for (int x = lane; NQ == 1 && x < MT; x += 32) {
              const int r = t.i * MT + x, tok = r / p.nrep;
              if (r >= t.s.rows) break;
              const uint16_t* row = p.q + (long long)(t.s.first + tok) * p.q_tstride +
                                    (long long)(t.unit / G::PARTS * p.nrep + (r - tok * p.nrep)) * p.q_hstride;
              for (int i = 0; i < D / 64; ++i) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + 64 * i));
            }
          }
          __syncwarp();
          if (lane == 0 && (t.lo < sh.x[0] || t.hi > sh.x[1])) paged_record(p, pieces, t, MT, nblk, j0, j1, cta);
          if (lane == 0) sh.more = sh.x[1] > sh.t.hi && paged_tile_next(p, MT, sh.t);
          __syncwarp();
          more = sh.more != 0;
          __syncwarp();
        }
        if (n < 0 && lane == 0) e.n = -1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.tile_full[k % kPcTiles]);
      }
      const PcTile* t = tile_at(k);
      if (t == nullptr) break;
      const int n = t->n, j0 = t->j0, keys = t->keys, kvh = t->kvh;
      const int* tab = p.table + (size_t)t->b * p.max_pages;
      auto page_of = [&](int j) {   // lanes 0-7: the page of 16 keys
        const int key = (j0 + j) * kPcKeys + 16 * lane;
        return lane < 8 && j < n && key < keys ? __ldg(tab + (key >> p.page_shift)) : -1;
      };
      int next = page_of(first);
      for (int j = first; j < n; j += kPcInfoWarps) {
        const uint32_t g = bc + j;
        PcInfo& f = sh.info[g % kPcInfo];
        const int key0 = (j0 + j) * kPcKeys;
        int pg = next;
        next = page_of(j + kPcInfoWarps);
#ifdef QDA_BOUNDS_CHECK
        if (cta == 0 && (int)g == p.stall_block) continue;   // testing aid: the waits for this block must run out
#endif
        const bool asked = lane < 8 && key0 + 16 * lane < keys;
        const bool gone = asked && (unsigned)pg >= (unsigned)p.num_pages;
        if (gone) pg = -1;
        const uint32_t gone8 = __ballot_sync(0xffffffffu, gone);
        if (gone8 && lane == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
        // largest 16-bit patterns of |scale| and |bias| of the block's keys and of its values: halves of a word each
        uint32_t top[4] = {0u, 0u, 0u, 0u};
        const bool cut = key0 + kPcKeys > keys;   // rows behind the sequence may hold anything
        const uint32_t limit = p.f16 ? 0x7C00u : 0x7680u;   // fp16 infinity; 2^110 in bf16
        bool odd = false;
        auto visit = [&](auto&& each) {
          for (int v0 = 0; v0 < nvec; v0 += 32) {
            const int v = v0 + lane, g16 = min(v / (2 * p.NG), 7);
            const int pv = __shfl_sync(0xffffffffu, pg, g16);
            if (v < nvec && pv >= 0) {
              const long long row = qda_pool_row(pv, kvh, (key0 + 16 * g16) & pmask, Hkv, p.page_shift);
              const int piece = v - g16 * 2 * p.NG;
              const long long at = row * p.NG / 8 + piece;
              auto piece_of = [&](const uint16_t* array) { return __ldg(reinterpret_cast<const uint4*>(array) + at); };
              const uint4 a[4] = {piece_of(p.ks), piece_of(p.kb), piece_of(p.vs), piece_of(p.vb)};
              each(a, 16 * g16, piece);
            }
          }
        };
        visit([&](const uint4 (&a)[4], int key, int piece) {
          if (cut) odd = odd || key0 + key + (piece * 8 + 7) / p.NG >= keys;
#pragma unroll
          for (int x = 0; x < 4; ++x)
            top[x] = __vmaxu2(top[x], __vmaxu2(__vmaxu2(a[x].x & 0x7fff7fffu, a[x].y & 0x7fff7fffu),
                                               __vmaxu2(a[x].z & 0x7fff7fffu, a[x].w & 0x7fff7fffu)));
        });
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          top[x] = max(top[x] & 0xffffu, top[x] >> 16);
          odd = odd || top[x] >= limit;
        }
        uint32_t bad[4] = {0u, 0u, 0u, 0u};   // this lane's keys that are not finite
        if (__any_sync(0xffffffffu, odd)) {    // one value at a time, without rows behind the sequence
          top[0] = top[1] = top[2] = top[3] = 0u;
          visit([&](const uint4 (&a)[4], int key, int piece) {
#pragma unroll 1
            for (int e = 0; e < 8; ++e) {
              const int at = key + (piece * 8 + e) / p.NG;
              if (key0 + at >= keys) continue;
              uint32_t u[4];
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const uint32_t w = (e >> 1) == 0 ? a[x].x : (e >> 1) == 1 ? a[x].y : (e >> 1) == 2 ? a[x].z : a[x].w;
                u[x] = (w >> (16 * (e & 1))) & 0x7fffu;
              }
              if (max(max(u[0], u[1]), max(u[2], u[3])) >= limit) {
#pragma unroll
                for (int x = 0; x < 4; ++x)
                  if ((at >> 5) == x) bad[x] |= 1u << (at & 31);
              } else {
#pragma unroll
                for (int x = 0; x < 4; ++x) top[x] = max(top[x], u[x]);
              }
            }
          });
        }
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          top[x] = __reduce_max_sync(0xffffffffu, top[x]);
          bad[x] = __reduce_or_sync(0xffffffffu, bad[x]);
        }
        // no key (value) of the block is larger than scale * QMAX + bias of the largest ones: to [2^T, 2^(T + 1)), where
        // a scale times 2^24 stays below 2^16
        constexpr int T = BITS == 4 ? -6 : -3;
        const uint32_t tk = __float_as_uint(fmaf(pc_half(top[0], p.f16), QMAX, pc_half(top[1], p.f16)));
        const uint32_t tv = __float_as_uint(fmaf(pc_half(top[2], p.f16), QMAX, pc_half(top[3], p.f16)));
        const int fk = max(1, min(254 + T - (int)(tk >> 23), 127 + kPcKUp)), fv = max(1, min(254 + T - (int)(tv >> 23), 253));
        wait(&sh.info_empty[g % kPcInfo], g / kPcInfo + 1);
        if (lane < 8)
          f.row[lane] = pg < 0 ? kPcNoRow : (uint32_t)qda_pool_row(pg, kvh, (key0 + 16 * lane) & pmask, Hkv, p.page_shift);
        if (lane < 4) {
          f.gone[lane] = ((gone8 >> (2 * lane)) & 1u ? 0xffffu : 0u) | ((gone8 >> (2 * lane + 1)) & 1u ? 0xffff0000u : 0u);
          f.bad[lane] = lane == 0 ? bad[0] : lane == 1 ? bad[1] : lane == 2 ? bad[2] : bad[3];
        }
        if (lane == 0) {
          f.kfac = __uint_as_float((uint32_t)fk << 23);
          f.kmul = __uint_as_float((uint32_t)(254 - fk) << 23);
          f.kv = 127 - fv;
          f.flags = (gone8 != 0) | ((bad[0] | bad[1] | bad[2] | bad[3]) ? 2u : 0u);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.info_full[g % kPcInfo]);
      }
      bc += n;
      if (first != 0) tile_done(k);
    }
   }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) {
    // no product is under way when the tensor memory goes back (after a wait that gave up some may be): a commit speaks for
    // the products of its own thread, so it is the same elected lane's
    if (pc_elect()) {
      volatile int none = 0;
      mma_commit(&sh.drain);
      mbar_wait_bounded(&sh.drain, 0, &none, p.err, 2u);
    }
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int BITS, int NQ, bool LSE>
cudaError_t pc_run(const QdaPagedParams* p, bool prepare, cudaStream_t s) {
  auto kern = qda_paged_chunk_kernel<D, BITS, NQ, LSE>;
  constexpr int smem = pc_smem<D, BITS, NQ>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  if (prepare) return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  kern<<<p->ctas, PcGeom<D, BITS, NQ>::WARPS * 32, smem, s>>>(*p);
  return cudaGetLastError();
}

template <int BITS, bool LSE>
cudaError_t pc_pick(const QdaPagedParams* p, int D, int tiles, bool prepare, cudaStream_t s) {
  switch (D) {
    case 64: return tiles == 2 ? pc_run<64, BITS, 2, LSE>(p, prepare, s) : pc_run<64, BITS, 1, LSE>(p, prepare, s);
    case 128: return tiles == 2 ? pc_run<128, BITS, 2, LSE>(p, prepare, s) : pc_run<128, BITS, 1, LSE>(p, prepare, s);
    case 256: return pc_run<256, BITS, 1, LSE>(p, prepare, s);
    case 512: return pc_run<512, BITS, 1, LSE>(p, prepare, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qda
