// Accumulated attention weight for many query rows per KV head (sm_103a), the products on tcgen05.
//
// A CTA per SM takes blocks of 128 keys under a KV head. A block's codes become operands once, and all of its query rows pass
// by in chunks of 128: S^T = K Q^T with keys in tensor memory's lanes and query rows in its columns, so that a thread owns a
// key: it reads its scores, takes exp(s - lse) and adds them up, and the sum over the rows needs no exchange at all.
//
// Masses are fp32, so scores should come near it: a key is two fp16 operands, its value to 11 bits and what those leave (22
// bits in all, 2^-24 of what a group of 4-bit codes can hold where they are put together, and 2^-39 of the most that the key
// can), each key scaled by its own power of two. A query row is fp16 under a power of two that it shares with the rows of its
// part where their largest values lie near (kPvNear: its values are then off by 2^-27 of its own largest at most), else under
// its own (2^-39). Both products go to the same fp32 accumulator.
//   key loader           a warp: a block's codes, scales and biases by asynchronous copies of 16 bytes into a ring, codes at
//                        places that eight threads' rows do not share banks at (bulk copies of sixteen keys each, one after
//                        the other, took 4200 cycles a block, more than all that follows with up to 128 rows);
//   dequantising warps   eight: two threads per key, codes -> the two operands in tensor memory (where products read them
//                        without a share of the shared memory's bandwidth; two blocks of them at D <= 128), and what undoes
//                        the key's scale;
//   row loader           one lane: a chunk's operands and scalars, laid out by the kernel ahead, by bulk copies into a ring;
//   MMA warps            two, a lane of each issues the products of every other chunk into an accumulator of its own (one
//                        lane alone took 106 cycles a product, whose arithmetic takes 64);
//   exponential warps    eight: two threads per key, half of a chunk's columns each (sixteen of 72 registers: ragged chunks
//                        216 us instead of 206).
// Every link is an mbarrier; every wait is bounded and sets the device error word, and after one that gave up every role ends.
//
// Ragged chunks (8 sequences, 1 to 1023 tokens over 1024 to 9001 keys, 2 heads per KV head, D 256, 8-bit): 204 us with the
// kernel ahead (18), 0.60 PFLOP/s of products counted once; the tensor pipe is busy 61 % of the time with twice those: at D 256
// the operands of one block fill their half of the tensor memory, so that no block is dequantised while the one before is
// multiplied. The last 64 tokens over 32768 keys (256 rows, D 128, 4-bit): 49 us (layout 6): the latency of the warps'
// instructions (some ten cycles each at five warps per scheduler), a block's hand-overs, some 4000 cycles that two chunks hide
// little of, and query rows that come from L2 again for every block. With both operands in shared memory the former took 390 us
// instead of 343 then: a product reads all of them there. With a loop over the few rows' kernel they take 3025 and 478 us.
#pragma once

#include "qda_paged_tc.cuh"
#include "qda_paged_weights.h"

namespace qda {

constexpr int kPvKeys = 128;
// Work of a block beside its query rows, in query rows. Ragged chunks at D 256 take 231 us with 64, 211 with 128, 204 with 200 and
// with 240, 206 with 300, 208 with 450; the window of 64 tokens 49 with any.
constexpr int kPvCost = 240;
constexpr int kPvExp = 8, kPvDeq = 8, kPvWarps = kPvExp + kPvDeq + 4;
constexpr int kPvParts = kPvExp / 4, kPvCols = kPvRows / kPvParts;   // threads of a key, columns of each
constexpr int kPvScalars = 3;  // chunks' scalars in flight
constexpr int kPvSlices = 10;  // operand slices in flight, at most

// A chunk's scalars. The rows of a part (those of one exponential thread) share a power of two where the largest values of all
// of them lie within 2^kPvNear (they then lose no more than that of the 39 bits' room below): what undoes it and the softmax
// scale is the part's `mul`; else that is 0 and every row has its own.
constexpr int kPvNear = 12;
struct alignas(16) PvScalars {
  float lse[kPvRows];          // minus a row's lse in log2 units; -inf: no row
  float muls[kPvRows];         // what undoes a row's own scale
  int last[kPvRows];           // last key that the row sees; -1: no row
  float mul[kPvParts];
};
static_assert(sizeof(PvScalars) % 16 == 0, "a bulk copy's size");

template <int D>
struct PvGeom {
  static constexpr int SD = 64;                          // dimensions of an operand slice
  static constexpr int SLICES = D / SD, SLICE = kPvRows * SD * 2;
  static constexpr int CHUNK = SLICES * SLICE + (int)sizeof(PvScalars);   // bytes in memory
  static constexpr int AS = D <= 128 ? 2 : 1;            // blocks in tensor memory, D columns each (two values a column, two operands)
  static constexpr int A_COL = 256;                      // they stand behind two accumulators
};

template <int BITS, int D>
struct PvKeys {
  static constexpr int RB = D * BITS / 8;                // a row of codes
  static constexpr int SC = kPvKeys * (D / 32) * 2;      // room for the scales of the smallest groups
  static constexpr int RAW = kPvKeys * RB + 2 * SC;
  static constexpr int RS = RAW > 24 * 1024 ? 2 : 3;     // blocks' codes in flight
  static constexpr int BS0 = (210 * 1024 - RS * RAW) / PvGeom<D>::SLICE;
  static constexpr int BS = BS0 > kPvSlices ? kPvSlices : BS0;   // operand slices in flight
  // (A wait tells neighbouring phases of a slot apart only. Before a chunk's slices are waited for, the exponentials of the
  // chunk two before are done, and with them all its slices: the phase before is over.)
  static_assert(BS >= 2 * PvGeom<D>::SLICES, "slots of two chunks");
};

// Chunks of a sequence under a KV head.
__device__ __forceinline__ int pv_chunks(const QdaWeightsParams& p, const PwSeq& s) {
  return s.n > 0 ? (int)(((long long)s.count * p.nrep + kPvRows - 1) / kPvRows) : 0;
}

// Sums of chunks stay at kPvTop, more than there is ever room for: starts that fall may count a row many times.
constexpr int kPvTop = 0x3fffffff;
__device__ __forceinline__ int pv_add(int a, int b) { return min(a + b, kPvTop); }

// Work of the first i blocks of a sequence under one KV head: the rows of a block's chunks, the last one as if it were full.
__device__ __forceinline__ long long pv_prefix(const QdaWeightsParams& p, const PwSeq& s, int i) {
  return pw_prefix<kPvKeys>(p, s, i, kPvCost + (long long)pv_chunks(p, s) * kPvRows, kPvCost + kPvRows);
}

// Where a CTA stands on its piece of the line: at a block of keys. Every role walks for itself, with what a sequence has in
// hand: at some twenty warps a block, what a step costs is what the block costs.
struct PvWalk {
  int b, kvh, x, blocks, flat, chunks;   // flat: blocks that all of the sequence's chunks see
  long long pos;               // the block's place
  PwSeq s;

  __device__ __forceinline__ void enter(const QdaWeightsParams& p) {
    s = pw_seq(p, b);
    blocks = pw_blocks<kPvKeys>(s);
    flat = pw_flat<kPvKeys>(s);
    chunks = pv_chunks(p, s);
  }
  __device__ __forceinline__ void start(const QdaWeightsParams& p, const long long* line, long long from) {
    b = qda_seq_of(line, p.B, from);
    enter(p);
    const long long head = pv_prefix(p, s, blocks);
    kvh = (int)((from - line[b]) / head);
    const long long at = line[b] + kvh * head;
    x = pw_block_at(blocks, from, [&](int i) { return at + pv_prefix(p, s, i); });
    pos = at + pv_prefix(p, s, x);
  }
  // The block at hand, or the next one that there is; false behind the piece.
  __device__ __forceinline__ bool here(const QdaWeightsParams& p, long long to) {
    if (pos >= to) return false;
    if (x >= blocks) {
      x = 0;
      if (++kvh >= p.Hkv) {
        kvh = 0;
        do {
          if (++b >= p.B) return false;
          enter(p);
        } while (blocks == 0);
      }
    }
    return true;
  }
  __device__ __forceinline__ void step(const QdaWeightsParams& p) {   // (as pv_prefix has it)
    if (x < flat) pos += kPvCost + (long long)chunks * kPvRows;
    else pos += kPvCost + kPvRows + (long long)p.nrep * (s.n - x * kPvKeys);
    ++x;
  }
  // The chunks whose rows see the block's first key: from this one to the sequence's last.
  __device__ __forceinline__ int first_chunk(const QdaWeightsParams& p) const {
    if (x < flat) return 0;
    const int before = max(0, x * kPvKeys - s.base - (s.len - s.count));   // counted tokens that do not
    return (int)(((long long)before * p.nrep) >> 7);
  }
};

// A slot of a ring of N and the parity of its phase, counted on.
template <int N>
struct PvSlot {
  uint32_t at = 0, phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) {
      at = 0;
      phase ^= 1u;
    }
  }
};

// As mbar_wait_bounded, for many warps that wait much: the barrier's own try suspends the warp for a while, and clock and abort
// flag are looked at every 64th time only (with both at every time, waiting took half of the instructions that the kernel
// issued).
__device__ __forceinline__ bool pv_wait(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int* err) {
  uint64_t t0 = 0;
  for (uint32_t n = 1; !mbar_try_wait(bar, parity); ++n) {
    if (n & 63u) continue;
    if (*abort) return false;
    const uint64_t t = globaltimer_ns();
    if (t0 == 0) t0 = t;
    if (t - t0 > 1000000000ull) {
      atomicOr(err, 1u);
      *abort = 1;
      return false;
    }
  }
  return true;
}

static_assert(kPvRows == 128 && kPvCols % 32 == 0, "first_chunk; columns of a load");

struct PvShared {
  PvScalars scal[kPvScalars];
  float kmul[2][kPvKeys];
  float part[2][kPvParts - 1][kPvKeys];   // sums of a key's other threads, by a block's parity
  long long at[QDA_MAX_B + 1]; // sequences on the line of work
  int chunk[QDA_MAX_B + 1];    // chunks before each sequence
  PvWalk walk;
  long long row[8][8];         // pool rows of a block's sixteens of keys (-1: none), eight blocks
  long long tot[kPvWarps];
  int ctot[kPvWarps];
  uint64_t r_full[3], r_empty[3], a_full[2], a_empty[2], b_full[kPvSlices], b_empty[kPvSlices], c_full[kPvScalars], c_empty[kPvScalars],
      d_full[2], d_empty[2], p_full[2], p_empty[2], drain;
  uint32_t tmem;
  int abort;
};

template <int BITS, int D>
constexpr int pv_smem() {
  using G = PvGeom<D>;
  return 1024 + PvKeys<BITS, D>::BS * G::SLICE + PvKeys<BITS, D>::RS * PvKeys<BITS, D>::RAW + (int)sizeof(PvShared);
}

// 2^e, and e that brings x to [2^14, 2^15) (0 for what is no positive number, or infinite).
__device__ __forceinline__ float pv_pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
__device__ __forceinline__ int pv_up(float x) {
  return x > 0.f && x < INFINITY ? max(-100, min(141 - (int)(__float_as_uint(x) >> 23), 100)) : 0;
}

template <int BITS, int D>
__global__ void __launch_bounds__(kPvWarps * 32, 1) qda_paged_weights_tc_kernel(const __grid_constant__ QdaWeightsParams p) {
  using G = PvGeom<D>;
  using K = PvKeys<BITS, D>;
  constexpr int SD = G::SD;
  extern __shared__ __align__(1024) unsigned char pv_smem_raw[];
  unsigned char* base = pv_smem_raw + ((1024u - (smem_addr(pv_smem_raw) & 1023u)) & 1023u);
  unsigned char* b_s = base;
  unsigned char* raw_s = base + K::BS * G::SLICE;
  PvShared& sh = *reinterpret_cast<PvShared*>(raw_s + K::RS * K::RAW);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int W_MMA = kPvExp + kPvDeq, W_KEYS = W_MMA + 2;   // behind the exponential and the dequantising warps
  volatile int* abort = &sh.abort;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.a_full[i], kPvDeq);
      mbar_init(&sh.a_empty[i], 2 + kPvExp);
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], kPvExp);
      mbar_init(&sh.p_full[i], kPvExp - 4);
      mbar_init(&sh.p_empty[i], 4);
    }
    for (int i = 0; i < kPvSlices; ++i) {
      mbar_init(&sh.b_full[i], 1);
      mbar_init(&sh.b_empty[i], 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(&sh.r_full[i], 33);   // the lanes' copies, and the rows' numbers
      mbar_init(&sh.r_empty[i], kPvDeq);
    }
    for (int i = 0; i < kPvScalars; ++i) {
      mbar_init(&sh.c_full[i], 1);
      mbar_init(&sh.c_empty[i], kPvExp);
    }
    mbar_init(&sh.drain, 2);
    sh.abort = 0;
    sh.at[0] = 0;
    sh.chunk[0] = 0;
    fence_barrier_init();
  }
  // ---- the line of work and the chunks: every CTA scans the lengths for itself
  long long carry = 0;
  int ccarry = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPvWarps * 32) {
    const int b = b0 + tid;
    long long v = 0;
    int c = 0;
    if (b < p.B) {
      const int start = p.q_start[b], end = p.q_start[b + 1], n = p.kv_len[b];
      const PwSeq s = pw_seq(p, start, end, n);
      v = p.Hkv * pv_prefix(p, s, pw_blocks<kPvKeys>(s));
      c = pv_chunks(p, s);
      if (blockIdx.x == 0 && pw_bad(p, start, end, n, s)) atomicOr(p.err, QDA_ERR_BIT_PAGED);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      const int z = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) {
        v += y;
        c = pv_add(c, z);
      }
    }
    if (lane == 31) {
      sh.tot[warp] = v;
      sh.ctot[warp] = c;
    }
    __syncthreads();
    long long before = carry;
    int cbefore = ccarry;
    for (int w = 0; w < kPvWarps; ++w) {
      if (w < warp) {
        before += sh.tot[w];
        cbefore = pv_add(cbefore, sh.ctot[w]);
      }
      carry += sh.tot[w];
      ccarry = pv_add(ccarry, sh.ctot[w]);
    }
    if (b < p.B) {
      sh.at[b + 1] = before + v;
      sh.chunk[b + 1] = pv_add(cbefore, c);
    }
    __syncthreads();
  }
  const long long piece = (carry + gridDim.x - 1) / gridDim.x;
  const long long from = min(carry, piece * blockIdx.x), to = min(carry, from + piece);
  if (from >= to || ccarry > p.max_chunks) {   // (more chunks than there can be: starts that fall)
    pdl_wait();
    return;
  }
  if (warp == W_MMA) tmem_alloc(&sh.tmem, 512);
  if (tid == 0) sh.walk.start(p, sh.at, from);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  auto wait = [&](uint64_t* bar, uint32_t parity) { return pv_wait(bar, parity, abort, p.err); };
  // a warp's wait, for which it ends as one
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, wait(bar, parity)) != 0; };
  PvWalk w = sh.walk;
  // where every role stands in the rings: operands and codes of blocks, chunks, their scalars, slices
  PvSlot<G::AS> as;
  PvSlot<K::RS> rs;
  PvSlot<2> ds, ps2;
  PvSlot<kPvScalars> cs;
  PvSlot<K::BS> bs;
  uint32_t bc = 0;             // blocks so far
  if (warp < kPvExp) {
    // ============================================================================ exponentials: some threads per key
    const int part = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t d_t = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kPvCols * part;
    for (; w.here(p, to); w.step(p), ++bc, as.next(), ps2.next()) {
      const int key = w.x * kPvKeys + r;
      if (!wait_all(&sh.a_full[as.at], as.phase)) break;
      const float km = sh.kmul[as.at][r];
      const long long row0 = sh.row[bc & 7][r >> 4], row = row0 + (r & 15);
      const bool there = row0 >= 0 && key < w.s.n, keep = there && key < w.s.base;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.a_empty[as.at]);
      float old = 0.f;
      if (part == 0 && keep) old = p.mass[row];
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      bool ok = true;
#pragma unroll 1
      for (int c = w.first_chunk(p); c < w.chunks; ++c, ds.next(), cs.next()) {
        const int buf = ds.at, ps = cs.at;
        ok = wait_all(&sh.c_full[ps], cs.phase) && wait_all(&sh.d_full[buf], ds.phase);
        if (!ok) break;
        tc_fence_after();
        const PvScalars& f = sh.scal[ps];
        // all of the chunk's rows see all of the block's keys: the last key against the first row's token
        const bool open = w.x + 1 < w.flat ||
                          (long long)(w.x * kPvKeys + kPvKeys - 1 - w.s.base - (w.s.len - w.s.count)) * p.nrep <= (long long)c * kPvRows;
#pragma unroll 1
        for (int q = 0; q < kPvCols / 32; ++q) {   // (a loop that stays small: the roles share the instruction cache)
          const int col = kPvCols * part + 32 * q;
          float v[32];
          pc_ld32(d_t + 128 * buf + 32 * q, v);
          tmem_wait_ld();
          if (q == kPvCols / 32 - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.d_empty[buf]);
          }
          float one = km * f.mul[part];
          if (f.mul[part] == 0.f) {   // rare: rows with scales of their own
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= f.muls[col + i];   // (exact: the same bits as with one scale for all)
            one = km * p.qscale;
          }
          if (open) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float4 m = *reinterpret_cast<const float4*>(f.lse + col + 4 * i);
              const float2 e0 = __ffma2_rn(make_float2(v[4 * i], v[4 * i + 1]), make_float2(one, one), make_float2(m.x, m.y));
              const float2 e1 = __ffma2_rn(make_float2(v[4 * i + 2], v[4 * i + 3]), make_float2(one, one), make_float2(m.z, m.w));
              sum[0] = __fadd2_rn(sum[0], make_float2(pc_ex2(e0.x), pc_ex2(e0.y)));
              sum[1] = __fadd2_rn(sum[1], make_float2(pc_ex2(e1.x), pc_ex2(e1.y)));
            }
          } else {   // what a row does not see stays out, whatever the row and its lse hold
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float y = pc_ex2(fmaf(v[i], one, f.lse[col + i]));
              sum[i & 1].x += key > f.last[col + i] ? 0.f : y;
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.c_empty[ps]);
      }
      if (!ok) break;
      float add = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (part > 0) {   // the key's first thread takes it from here
        if (!wait_all(&sh.p_empty[ps2.at], ps2.phase ^ 1u)) break;
        sh.part[ps2.at][part - 1][r] = add;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[ps2.at]);
        continue;
      }
      if (!wait_all(&sh.p_full[ps2.at], ps2.phase)) break;
#pragma unroll
      for (int i = 0; i < kPvParts - 1; ++i) add += sh.part[ps2.at][i][r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_empty[ps2.at]);
      if (keep) {
        p.mass[row] = fmaf(p.decay, old, add);
      } else if (there) {
        p.mass[row] = add;
        p.token[row] = key + (p.shift != nullptr ? p.shift[w.b] : 0);
      }
    }
  } else if (warp < W_MMA) {
    // ============================================================================ codes -> operands: two threads per key
    const int r = (tid - kPvExp * 32) & 127, half = (tid - kPvExp * 32) >> 7;
    constexpr float QMAX = (float)((1 << BITS) - 1);
    const uint32_t a_t = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + G::A_COL;
    for (; w.here(p, to); w.step(p), ++bc, as.next(), rs.next()) {
      const int st = rs.at;
      if (!wait_all(&sh.r_full[st], rs.phase)) break;
      const unsigned char* raw = raw_s + st * K::RAW;
      const bool there = sh.row[bc & 7][r >> 4] >= 0;
      // all of the key's scales and biases (pairs of 16 bits)
      uint32_t sw[4] = {0, 0, 0, 0}, bw[4] = {0, 0, 0, 0};
      if (there) {
        const unsigned char *ks = raw + kPvKeys * K::RB + r * p.NG * 2, *kb = ks + kPvKeys * p.NG * 2;
        if (p.NG == 8) {
          const uint4 x = *reinterpret_cast<const uint4*>(ks), y = *reinterpret_cast<const uint4*>(kb);
          sw[0] = x.x, sw[1] = x.y, sw[2] = x.z, sw[3] = x.w;
          bw[0] = y.x, bw[1] = y.y, bw[2] = y.z, bw[3] = y.w;
        } else if (p.NG == 4) {
          const uint2 x = *reinterpret_cast<const uint2*>(ks), y = *reinterpret_cast<const uint2*>(kb);
          sw[0] = x.x, sw[1] = x.y;
          bw[0] = y.x, bw[1] = y.y;
        } else if (p.NG == 2) {
          sw[0] = *reinterpret_cast<const uint32_t*>(ks);
          bw[0] = *reinterpret_cast<const uint32_t*>(kb);
        } else {
          sw[0] = *reinterpret_cast<const uint16_t*>(ks);
          bw[0] = *reinterpret_cast<const uint16_t*>(kb);
        }
      }
      // what the key can hold at most, to [2^14, 2^15)
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 a = half2_bits_to_float2_rt(sw[i], p.f16), z = half2_bits_to_float2_rt(bw[i], p.f16);
        top = fmaxf(top, fmaxf(fmaf(fabsf(a.x), QMAX, fabsf(z.x)), fmaf(fabsf(a.y), QMAX, fabsf(z.y))));
      }
      const int e = pv_up(top);
      const float up = pv_pow2(e);
      if (!wait_all(&sh.a_empty[as.at], as.phase ^ 1u)) break;
      tc_fence_after();
      const uint32_t hi_t = a_t + as.at * D, lo_t = hi_t + D / 2;
      if (half == 0) sh.kmul[as.at][r] = pv_pow2(-e);
#pragma unroll 1
      for (int i = 0; i < D / 64; ++i) {   // 32 values: 16 columns of either operand
        const int u = half * (D / 64) + i, g = (u * 32) >> p.gs_shift;
        uint32_t code[BITS];
#pragma unroll
        for (int k = 0; k < BITS / 4; ++k) {
          const uint4 q = *reinterpret_cast<const uint4*>(raw + pw_chunk<K::RB>(r, u * (BITS / 4) + k));
          code[4 * k] = q.x;
          code[4 * k + 1] = q.y;
          code[4 * k + 2] = q.z;
          code[4 * k + 3] = q.w;
        }
        const uint32_t s2 = g < 4 ? (g < 2 ? sw[0] : sw[1]) : (g < 6 ? sw[2] : sw[3]);
        const uint32_t z2 = g < 4 ? (g < 2 ? bw[0] : bw[1]) : (g < 6 ? bw[2] : bw[3]);
        // (a key that is not there has scale and bias 0)
        float s = half_bits_to_float_rt((s2 >> (16 * (g & 1))) & 0xffffu, p.f16) * up;
        float z = half_bits_to_float_rt((z2 >> (16 * (g & 1))) & 0xffffu, p.f16) * up;
        if constexpr (BITS == 4) {
          z = fmaf(s, -16.f, z);
          s *= 16.f;
        }
        uint32_t h[16], l[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float2 v;
          if constexpr (BITS == 4) {   // codes as 1 + c / 16: z - 16 s is rounded once, by no more than the value itself may be
            const uint32_t w0 = ((code[k >> 2] << 3) & 0x78787878u) | 0x80808080u, w1 = ((code[k >> 2] >> 1) & 0x78787878u) | 0x80808080u;
            const float2 c = make_float2(__uint_as_float(__byte_perm(w0, 0x3F000000u, 0x7044 + ((k & 3) << 8))),
                                         __uint_as_float(__byte_perm(w1, 0x3F000000u, 0x7044 + ((k & 3) << 8))));
            v = __ffma2_rn(make_float2(s, s), c, make_float2(z, z));
          } else {                     // 2^23 + c, less 2^23
            const float2 c = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(code[k >> 1], 0x4B000000u, 0x7440 + 2 * (k & 1))),
                                                    __uint_as_float(__byte_perm(code[k >> 1], 0x4B000000u, 0x7441 + 2 * (k & 1)))),
                                        make_float2(-8388608.f, -8388608.f));
            v = __ffma2_rn(make_float2(s, s), c, make_float2(z, z));
          }
          h[k] = pc_h2(v.x, v.y);
          const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
          const float2 d = __fadd2_rn(v, make_float2(-b.x, -b.y));
          l[k] = pc_h2(d.x, d.y);
        }
        tmem_st16(hi_t + 16 * u, h);
        tmem_st16(lo_t + 16 * u, l);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&sh.a_full[as.at]);
        mbar_arrive(&sh.r_empty[st]);
      }
    }
  } else if (warp < W_KEYS) {
    // ============================================================================ a lane issues the products of its chunks
    constexpr uint32_t ID = (1u << 4) | ((uint32_t)(kPvRows >> 3) << 17) | (8u << 24);   // M 128, N 128, fp16, fp32 sums
    const uint32_t one = pc_elect();
    const uint32_t b_a = smem_addr(b_s);
    bool ok = true;
    for (; ok && w.here(p, to); w.step(p), as.next()) {
      ok = wait_all(&sh.a_full[as.at], as.phase);
      for (int c = w.first_chunk(p); ok && c < w.chunks; ++c, ds.next()) {
        const int buf = ds.at;
        if (buf != warp - W_MMA) {   // the other warp's
#pragma unroll
          for (int sl = 0; sl < G::SLICES; ++sl) bs.next();
          continue;
        }
        ok = wait_all(&sh.d_empty[buf], ds.phase ^ 1u);
        for (int sl = 0; ok && sl < G::SLICES; ++sl, bs.next()) {
          ok = wait_all(&sh.b_full[bs.at], bs.phase);
          if (!ok) break;
          tc_fence_after();
          const uint64_t b = pc_desc(b_a + bs.at * G::SLICE, 16);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint32_t a = tmem + G::A_COL + as.at * D + y * (D / 2) + sl * (SD / 2);
#pragma unroll
            for (int x = 0; x < SD / 16; ++x)
              pc_mma_ts(one, tmem + 128 * buf, a + 8 * x, b + (x * 32 >> 4), ID, sl > 0 || y > 0 || x > 0);
          }
          pc_commit(one, &sh.b_empty[bs.at]);
        }
        if (ok) pc_commit(one, &sh.d_full[buf]);
      }
      if (ok) pc_commit(one, &sh.a_empty[as.at]);
      __syncwarp();
    }
  } else if (warp == W_KEYS) {
    // ============================================================================ codes, scales and biases of the blocks
    // four lanes have sixteen keys: a row's chunks of 64 bytes, row after row, then chunks of the scales and of the biases
    const int g = lane >> 2, l4 = lane & 3, ng2 = 2 * p.NG;   // 16-byte chunks of sixteen keys' scales
    const char* const codes = reinterpret_cast<const char*>(p.kp) + 16 * l4;
    constexpr int CPR = K::RB / 16;                           // 16-byte chunks of a row of codes
    for (; w.here(p, to); w.step(p), ++bc, rs.next()) {
      const int key = w.x * kPvKeys + 16 * g;
      const int pg = key < w.s.n ? __ldg(p.table + (size_t)w.b * p.max_pages + (key >> p.page_shift)) : -1;
      const bool there = (unsigned)pg < (unsigned)p.num_pages;
      if (!there && key < w.s.n) atomicOr(p.err, QDA_ERR_BIT_PAGED);
      // (pool rows are below 2^32 - 1)
      const uint32_t row = (((uint32_t)pg * (uint32_t)p.Hkv + (uint32_t)w.kvh) << p.page_shift) +
                           (uint32_t)(key & ((1 << p.page_shift) - 1));
      if (!wait_all(&sh.r_empty[rs.at], rs.phase ^ 1u)) break;
      if (l4 == 0) sh.row[bc & 7][g] = there ? (long long)row : -1;   // (the exponential warps are at most six blocks behind)
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.r_full[rs.at]);
      if (there) {
        const uint32_t raw = smem_addr(raw_s + rs.at * K::RAW), dst = raw + 16 * g * K::RB;
        const char* src = codes + (uint64_t)row * K::RB;
#pragma unroll 8
        for (int i = 0; i < 4 * CPR; ++i) {
          const int c = 4 * i + l4;
          pw_copy16(dst + pw_chunk<K::RB>(c / CPR, c % CPR), src + 64 * i);
        }
        const uint32_t to_s = raw + kPvKeys * K::RB + g * ng2 * 16, to_z = to_s + 8 * ng2 * 16;
        const char* ks = reinterpret_cast<const char*>(p.ks) + (uint64_t)row * ng2;
        const char* kb = reinterpret_cast<const char*>(p.kb) + (uint64_t)row * ng2;
        for (int c = 16 * l4; c < 16 * ng2; c += 64) {
          pw_copy16(to_s + c, ks + c);
          pw_copy16(to_z + c, kb + c);
        }
      }
      asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(&sh.r_full[rs.at])) : "memory");
    }
    pw_wait<0>();   // no copy is under way when the CTA's shared memory goes
  } else if (lane == 0) {
    // ============================================================================ operands and scalars of the chunks
    pdl_wait();   // the kernel ahead has laid them out
    asm volatile("fence.proxy.async;" ::: "memory");
    const uint64_t policy = [] {
      uint64_t x;
      asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(x));
      return x;
    }();
    bool ok = true;
    uint32_t sc = 0, cc = 0;   // slices and chunks so far
    for (; ok && w.here(p, to); w.step(p)) {
      const int c0 = sh.chunk[w.b];
      for (int c = w.first_chunk(p); ok && c < w.chunks; ++c, ++cc, cs.next()) {
        const char* src = p.chunks + ((size_t)(c0 + c) * p.Hkv + w.kvh) * G::CHUNK;
        ok = wait(&sh.c_empty[cs.at], cs.phase ^ 1u);
        if (!ok) break;
        mbar_arrive_expect_tx(&sh.c_full[cs.at], sizeof(PvScalars));
        bulk_g2s(&sh.scal[cs.at], src + G::SLICES * G::SLICE, sizeof(PvScalars), &sh.c_full[cs.at], policy);
        for (int sl = 0; sl < G::SLICES; ++sl, ++sc, bs.next()) {
          ok = wait(&sh.b_empty[bs.at], bs.phase ^ 1u);
          if (!ok) break;
#ifdef QDA_BOUNDS_CHECK
          if (blockIdx.x == 0 && (p.stall == (int)sc)) continue;   // testing aid: the waits for this slice must run out
#endif
          mbar_arrive_expect_tx(&sh.b_full[bs.at], G::SLICE);
          bulk_g2s(b_s + bs.at * G::SLICE, src + sl * G::SLICE, G::SLICE, &sh.b_full[bs.at], policy);
        }
      }
    }
    if (!ok || *abort) {
      // a wait gave up: copies under way land before the CTA's shared memory goes (a phase that a copy never began is waited
      // for in vain, until the limit)
      volatile int none = 0;
      for (uint32_t i = sc < (uint32_t)K::BS ? 0 : sc - K::BS; i < sc; ++i)
        none = 0, mbar_wait_bounded(&sh.b_full[i % K::BS], (i / K::BS) & 1u, &none, p.err, 2u);
      for (uint32_t i = cc < (uint32_t)kPvScalars ? 0 : cc - kPvScalars; i < cc; ++i)
        none = 0, mbar_wait_bounded(&sh.c_full[i % kPvScalars], (i / kPvScalars) & 1u, &none, p.err, 2u);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // no product is under way when the tensor memory goes back: an elected lane's commit speaks for its own products
  if (warp == W_MMA || warp == W_MMA + 1) {
    if (pc_elect()) mma_commit(&sh.drain);
    __syncwarp();
  }
  if (warp == W_MMA) {
    if (lane == 0) {
      volatile int none = 0;
      mbar_wait_bounded(&sh.drain, 0, &none, p.err, 2u);
    }
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

template <int BITS, int D>
cudaError_t pv_run(const QdaWeightsParams* p, bool prepare, cudaStream_t s) {
  auto kern = qda_paged_weights_tc_kernel<BITS, D>;
  constexpr int smem = pv_smem<BITS, D>();
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  if (prepare) return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)p->ctas);
  cfg.blockDim = dim3(kPvWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, *p);
}

template <int BITS>
cudaError_t pv_pick(const QdaWeightsParams* p, int D, bool prepare, cudaStream_t s) {
  switch (D) {
    case 64: return pv_run<BITS, 64>(p, prepare, s);
    case 128: return pv_run<BITS, 128>(p, prepare, s);
    case 256: return pv_run<BITS, 256>(p, prepare, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace qda
