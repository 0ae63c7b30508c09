// Accumulated attention weight for many query rows per KV head (sm_103a), the products on tcgen05.
//
// A CTA per SM takes blocks of 128 keys under a KV head. A block's codes become operands once, and all of its query rows pass
// by in chunks of 128: S^T = K Q^T with keys in tensor memory's lanes and query rows in its columns, so that a thread owns a
// key: it reads its scores, takes exp(s - lse) and adds them up, and the sum over the rows needs no exchange at all.
//
// Masses are fp32, so scores must be: a key is two fp16 operands, its value to 11 bits and what those leave (22 bits, or 2^-39
// of the key's largest possible value), each key scaled by its own power of two, and a query row is exact in fp16 scaled by
// its own (what is 2^-39 of the row's largest and less loses bits). Both products go to the same fp32 accumulator.
//   dequantising warps   eight: two threads per key, codes -> the two operands in shared memory (two blocks ahead of each
//                        other where they fit), and what undoes the key's scale;
//   producer             one lane: a chunk's operands and scalars, laid out by the kernel ahead, by bulk copies into a ring;
//   MMA warp             one lane issues every product; two accumulators of 128 columns take turns;
//   exponential warps    eight: a thread per key and half of a chunk's columns.
// Every link is an mbarrier; every wait is bounded and sets the device error word, and after one that gave up every role ends.
#pragma once

#include "qda_paged_tc.cuh"
#include "qda_paged_weights.h"

namespace qda {

constexpr int kPvKeys = 128;
constexpr int kPvCost = 48;    // work of a block beside its query rows, in query rows
constexpr int kPvExp = 8, kPvDeq = 8, kPvWarps = kPvExp + kPvDeq + 2;
constexpr int kPvScalars = 3;  // chunks' scalars in flight

// A chunk's scalars: pairs of rows side by side.
struct PvScalars {
  float4 ml[kPvRows / 2];      // what undoes a row's scale times the softmax scale, twice; minus its lse in log2 units, twice
  int2 last[kPvRows / 2];      // last key that the row sees; -1: no row
};

template <int D>
struct PvGeom {
  static constexpr int SD = D < 128 ? D : 128;           // dimensions of an operand slice
  static constexpr int SLICES = D / SD, SLICE = kPvRows * SD * 2;
  static constexpr int CHUNK = SLICES * SLICE + (int)sizeof(PvScalars);   // bytes in memory
  static constexpr int A = 2 * kPvKeys * D * 2;          // a block's two operands
  static constexpr int AS = D <= 128 ? 2 : 1;            // blocks in shared memory
  static constexpr int BS = D == 64 ? 4 : 2;             // operand slices in flight
};

struct PvShared {
  PvScalars scal[kPvScalars];
  float kmul[2][kPvKeys];
  float part[2][kPvKeys];      // the second half's sums, by a block's parity
  long long at[QDA_MAX_B + 1]; // sequences on the line of work
  int chunk[QDA_MAX_B + 1];    // chunks before each sequence
  long long tot[kPvWarps];
  int ctot[kPvWarps];
  uint64_t a_full[2], a_empty[2], b_full[4], b_empty[4], c_full[kPvScalars], c_empty[kPvScalars], d_full[2], d_empty[2],
      p_full[2], p_empty[2], drain;
  uint32_t tmem;
  int abort;
};

template <int D>
constexpr int pv_smem() {
  using G = PvGeom<D>;
  return 1024 + G::AS * G::A + G::BS * G::SLICE + (int)sizeof(PvShared);
}

// Chunks of a sequence under a KV head.
__device__ __forceinline__ int pv_chunks(const QdaWeightsParams& p, const PwSeq& s) {
  return s.n > 0 ? (int)(((long long)s.count * p.nrep + kPvRows - 1) / kPvRows) : 0;
}

// Where a CTA stands on its piece of the line.
struct PvWalk {
  int b, kvh, x, blocks;
  long long head, at;
  PwSeq s;

  __device__ __forceinline__ void enter(const QdaWeightsParams& p) {
    s = pw_seq(p, b);
    blocks = pw_blocks<kPvKeys>(s);
    head = pw_prefix<kPvKeys, kPvCost>(p, s, blocks);
  }
  __device__ __forceinline__ void start(const QdaWeightsParams& p, const long long* line, long long from) {
    b = qda_seq_of(line, p.B, from);
    enter(p);
    kvh = (int)((from - line[b]) / head);
    at = line[b] + kvh * head;
    x = pw_block_at<kPvKeys, kPvCost>(p, s, blocks, at, from);
  }
  // The block at hand, or the next one that there is; false behind the piece.
  __device__ __forceinline__ bool here(const QdaWeightsParams& p, long long to) {
    if (x >= blocks) {
      x = 0;
      at += head;
      if (++kvh >= p.Hkv) {
        kvh = 0;
        do {
          if (++b >= p.B) return false;
          enter(p);
        } while (blocks == 0);
      }
    }
    return at + pw_prefix<kPvKeys, kPvCost>(p, s, x) < to;
  }
  // The chunks whose rows see the block's first key: from this one to the sequence's last.
  __device__ __forceinline__ int first_chunk(const QdaWeightsParams& p) const {
    const int before = max(0, x * kPvKeys - s.base - (s.len - s.count));   // counted tokens that do not
    return (int)((long long)before * p.nrep / kPvRows);
  }
};

template <int BITS, int D>
__global__ void __launch_bounds__(kPvWarps * 32, 1) qda_paged_weights_tc_kernel(const __grid_constant__ QdaWeightsParams p) {
  using G = PvGeom<D>;
  constexpr int W = D * BITS / 32, SD = G::SD;
  extern __shared__ __align__(1024) unsigned char pv_smem_raw[];
  unsigned char* base = pv_smem_raw + ((1024u - (smem_addr(pv_smem_raw) & 1023u)) & 1023u);
  unsigned char* a_s = base;
  unsigned char* b_s = base + G::AS * G::A;
  PvShared& sh = *reinterpret_cast<PvShared*>(b_s + G::BS * G::SLICE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  constexpr int W_MMA = kPvExp + kPvDeq;   // behind the exponential and the dequantising warps; the producer behind it
  volatile int* abort = &sh.abort;
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.a_full[i], kPvDeq);
      mbar_init(&sh.a_empty[i], 1 + kPvExp);
      mbar_init(&sh.d_full[i], 1);
      mbar_init(&sh.d_empty[i], kPvExp);
      mbar_init(&sh.p_full[i], kPvExp / 2);
      mbar_init(&sh.p_empty[i], kPvExp / 2);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&sh.b_full[i], 1);
      mbar_init(&sh.b_empty[i], 1);
    }
    for (int i = 0; i < kPvScalars; ++i) {
      mbar_init(&sh.c_full[i], 1);
      mbar_init(&sh.c_empty[i], kPvExp);
    }
    mbar_init(&sh.drain, 1);
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
      v = p.Hkv * pw_prefix<kPvKeys, kPvCost>(p, s, pw_blocks<kPvKeys>(s));
      c = pv_chunks(p, s);
      if (blockIdx.x == 0 && pw_bad(p, start, end, n, s)) atomicOr(p.err, QDA_ERR_BIT_PAGED);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, v, o);
      const int z = __shfl_up_sync(0xffffffffu, c, o);
      if (lane >= o) {
        v += y;
        c += z;
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
        cbefore += sh.ctot[w];
      }
      carry += sh.tot[w];
      ccarry += sh.ctot[w];
    }
    if (b < p.B) {
      sh.at[b + 1] = before + v;
      sh.chunk[b + 1] = cbefore + c;
    }
    __syncthreads();
  }
  const long long piece = (carry + gridDim.x - 1) / gridDim.x;
  const long long from = min(carry, piece * blockIdx.x), to = min(carry, from + piece);
  if (from >= to || ccarry > p.max_chunks) {   // (more chunks than there can be: starts that fall)
    pdl_wait();
    return;
  }
  if (warp == W_MMA) tmem_alloc(&sh.tmem, 256);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  auto wait = [&](uint64_t* bar, uint32_t phase) { return mbar_wait_bounded(bar, phase & 1u, abort, p.err, 1u); };
  // a warp's wait, for which it ends as one
  auto wait_all = [&](uint64_t* bar, uint32_t phase) { return __all_sync(0xffffffffu, wait(bar, phase)) != 0; };
  const int pmask = (1 << p.page_shift) - 1;
  PvWalk w;
  w.start(p, sh.at, from);
  // blocks, chunks and slices so far: every role counts them for itself
  uint32_t bc = 0, cc = 0, sc = 0;
  auto key_row = [&](int key, bool* there) -> long long {
    const int pg = key < w.s.n ? __ldg(p.table + (size_t)w.b * p.max_pages + (key >> p.page_shift)) : -1;
    *there = (unsigned)pg < (unsigned)p.num_pages;
    return *there ? qda_pool_row(pg, w.kvh, key & pmask, p.Hkv, p.page_shift) : 0;
  };

  if (warp < kPvExp) {
    // ============================================================================ exponentials: two threads per key
    const int half = warp >> 2, r = 32 * (warp & 3) + lane;
    const uint32_t d_t = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + 64 * half;
    for (; w.here(p, to); ++w.x, ++bc) {
      const int key = w.x * kPvKeys + r;
      bool there;
      const long long row = key_row(key, &there);
      const bool keep = there && key < w.s.base;
      float old = 0.f;
      if (half == 0 && keep) old = p.mass[row];
      const int first_tok = w.s.len - w.s.count;
      const int chunks = sh.chunk[w.b + 1] - sh.chunk[w.b];
      if (!wait_all(&sh.a_full[bc % G::AS], bc / G::AS)) break;
      const float km = sh.kmul[bc % G::AS][r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.a_empty[bc % G::AS]);
      float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      bool ok = true;
      for (int c = w.first_chunk(p); c < chunks; ++c, ++cc) {
        const int buf = cc & 1, ps = cc % kPvScalars;
        ok = wait_all(&sh.c_full[ps], cc / kPvScalars) && wait_all(&sh.d_full[buf], cc >> 1);
        if (!ok) break;
        tc_fence_after();
        const PvScalars& f = sh.scal[ps];
        const float2 km2 = make_float2(km, km);
        // all of the chunk's rows see all of the block's keys
        const bool open = w.x * kPvKeys + kPvKeys - 1 <= w.s.base + first_tok + (int)((long long)c * kPvRows / p.nrep);
        // sixteen columns at a time, the next ones on their way
        float v[2][16];
        auto weigh = [&](const float (&u)[16], int q, bool masked) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 ml = f.ml[32 * half + 8 * q + i];
            const float2 s2 = __fmul2_rn(make_float2(u[2 * i], u[2 * i + 1]), km2);
            const float2 e = __ffma2_rn(s2, make_float2(ml.x, ml.y), make_float2(ml.z, ml.w));
            float2 y = make_float2(pc_ex2(e.x), pc_ex2(e.y));
            if (masked) {
              const int2 last = f.last[32 * half + 8 * q + i];
              y = make_float2(key <= last.x ? y.x : 0.f, key <= last.y ? y.y : 0.f);
            }
            sum[i & 1] = __fadd2_rn(sum[i & 1], y);
          }
        };
        pc_ld16(d_t + 128 * buf, v[0]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          tmem_wait_ld();
          if (q < 3) pc_ld16(d_t + 128 * buf + 16 * (q + 1), v[(q + 1) & 1]);
          if (q == 3) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.d_empty[buf]);
          }
          if (open) weigh(v[q & 1], q, false);
          else weigh(v[q & 1], q, true);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.c_empty[ps]);
      }
      if (!ok) break;
      float add = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
      if (half == 1) {   // the other half's threads take it from here
        if (!wait_all(&sh.p_empty[bc & 1], (bc >> 1) + 1)) break;
        sh.part[bc & 1][r] = add;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.p_full[bc & 1]);
        continue;
      }
      if (!wait_all(&sh.p_full[bc & 1], bc >> 1)) break;
      add += sh.part[bc & 1][r];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.p_empty[bc & 1]);
      if (there && key < w.s.n) {
        if (keep) {
          p.mass[row] = fmaf(p.decay, old, add);
        } else {
          p.mass[row] = add;
          p.token[row] = key + (p.shift != nullptr ? p.shift[w.b] : 0);
        }
      }
    }
  } else if (warp < W_MMA) {
    // ============================================================================ codes -> operands: two threads per key
    const int r = (tid - kPvExp * 32) & 127, half = (tid - kPvExp * 32) >> 7;
    constexpr float QMAX = (float)((1 << BITS) - 1);
    for (; w.here(p, to); ++w.x, ++bc) {
      const int key = w.x * kPvKeys + r;
      bool there;
      const long long row = key_row(key, &there);
      if (!there && key < w.s.n) atomicOr(p.err, QDA_ERR_BIT_PAGED);
      // what the key can hold at most, to [2^14, 2^15)
      float top = 0.f;
      if (there) {
        for (int g = 0; g < p.NG; ++g) {
          const float s = half_bits_to_float_rt(__ldg(p.ks + row * p.NG + g), p.f16), z = half_bits_to_float_rt(__ldg(p.kb + row * p.NG + g), p.f16);
          top = fmaxf(top, fmaf(fabsf(s), QMAX, fabsf(z)));
        }
      }
      const int e = top > 0.f && top < INFINITY ? max(-100, min(14 - ilogbf(top), 100)) : 0;
      const float up = exp2f((float)e);
      if (!wait_all(&sh.a_empty[bc % G::AS], bc / G::AS + 1)) break;
      unsigned char* hi = a_s + (bc % G::AS) * G::A;
      unsigned char* lo = hi + kPvKeys * D * 2;
      if (half == 0) sh.kmul[bc % G::AS][r] = exp2f((float)-e);
      // 32 values at a time: D / 64 of them for each thread
      for (int i = 0; i < D / 64; ++i) {
        const int u = half * (D / 64) + i;
        uint32_t code[BITS];
#pragma unroll
        for (int k = 0; k < BITS / 4; ++k) {
          const uint4 q = there ? __ldg(reinterpret_cast<const uint4*>(p.kp + row * W + u * BITS) + k) : make_uint4(0, 0, 0, 0);
          code[4 * k] = q.x;
          code[4 * k + 1] = q.y;
          code[4 * k + 2] = q.z;
          code[4 * k + 3] = q.w;
        }
        const int g = u * 32 / p.GS;
        const float s = there ? half_bits_to_float_rt(__ldg(p.ks + row * p.NG + g), p.f16) * up : 0.f;
        const float z = there ? half_bits_to_float_rt(__ldg(p.kb + row * p.NG + g), p.f16) * up : 0.f;
#pragma unroll
        for (int o = 0; o < 4; ++o) {   // 8 values: 16 bytes of either operand
          uint32_t h[4], l[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float v[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int at = 8 * o + 2 * k + j;
              const uint32_t c = (code[at * BITS / 32] >> (at * BITS % 32)) & ((1u << BITS) - 1);
              v[j] = fmaf(s, __uint_as_float(0x4B000000u | c) - 8388608.f, z);
            }
            h[k] = pc_h2(v[0], v[1]);
            const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
            l[k] = pc_h2(v[0] - b.x, v[1] - b.y);
          }
          const int piece = u * 4 + o;   // 16 bytes of the row; blocks of 64 values, rows of 128 bytes, swizzled
          const int to16 = (piece >> 3) * 16384 + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
          *reinterpret_cast<uint4*>(hi + to16) = make_uint4(h[0], h[1], h[2], h[3]);
          *reinterpret_cast<uint4*>(lo + to16) = make_uint4(l[0], l[1], l[2], l[3]);
        }
      }
      fence_proxy_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh.a_full[bc % G::AS]);
    }
  } else if (warp == W_MMA) {
    // ============================================================================ one lane issues the products
    constexpr uint32_t ID = (1u << 4) | ((uint32_t)(kPvRows >> 3) << 17) | (8u << 24);   // M 128, N 128, fp16, fp32 sums
    const uint32_t one = pc_elect();
    const uint32_t a_a = smem_addr(a_s), b_a = smem_addr(b_s);
    bool ok = true;
    for (; ok && w.here(p, to); ++w.x, ++bc) {
      const int chunks = sh.chunk[w.b + 1] - sh.chunk[w.b];
      ok = wait_all(&sh.a_full[bc % G::AS], bc / G::AS);
      for (int c = w.first_chunk(p); ok && c < chunks; ++c, ++cc) {
        const int buf = cc & 1;
        ok = wait_all(&sh.d_empty[buf], (cc >> 1) + 1);
        for (int sl = 0; ok && sl < G::SLICES; ++sl, ++sc) {
          ok = wait_all(&sh.b_full[sc % G::BS], sc / G::BS);
          if (!ok) break;
          tc_fence_after();
          const uint64_t b = pc_desc(b_a + (sc % G::BS) * G::SLICE, 16);
#pragma unroll
          for (int y = 0; y < 2; ++y) {
            const uint64_t a = pc_desc(a_a + (bc % G::AS) * G::A + y * kPvKeys * D * 2 + sl * (SD / 64) * 16384, 16);
#pragma unroll
            for (int x = 0; x < SD / 16; ++x) {
              const uint32_t off = ((x >> 2) * 16384 + (x & 3) * 32) >> 4;
              pc_mma_ss(one, tmem + 128 * buf, a + off, b + off, ID, sl > 0 || y > 0 || x > 0);
            }
          }
          pc_commit(one, &sh.b_empty[sc % G::BS]);
        }
        if (ok) pc_commit(one, &sh.d_full[buf]);
      }
      if (ok) pc_commit(one, &sh.a_empty[bc % G::AS]);
      __syncwarp();
    }
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
    for (; ok && w.here(p, to); ++w.x) {
      const int c0 = sh.chunk[w.b], chunks = sh.chunk[w.b + 1] - c0;
      for (int c = w.first_chunk(p); ok && c < chunks; ++c, ++cc) {
        const char* src = p.chunks + ((size_t)(c0 + c) * p.Hkv + w.kvh) * G::CHUNK;
        const int ps = cc % kPvScalars;
        ok = wait(&sh.c_empty[ps], cc / kPvScalars + 1);
        if (!ok) break;
        mbar_arrive_expect_tx(&sh.c_full[ps], sizeof(PvScalars));
        bulk_g2s(&sh.scal[ps], src + G::SLICES * G::SLICE, sizeof(PvScalars), &sh.c_full[ps], policy);
        for (int sl = 0; sl < G::SLICES; ++sl, ++sc) {
          ok = wait(&sh.b_empty[sc % G::BS], sc / G::BS + 1);
          if (!ok) break;
#ifdef QDA_BOUNDS_CHECK
          if (blockIdx.x == 0 && (p.stall == (int)sc)) continue;   // testing aid: the waits for this slice must run out
#endif
          mbar_arrive_expect_tx(&sh.b_full[sc % G::BS], G::SLICE);
          bulk_g2s(b_s + (sc % G::BS) * G::SLICE, src + sl * G::SLICE, G::SLICE, &sh.b_full[sc % G::BS], policy);
        }
      }
    }
    if (!ok || *abort) {
      // a wait gave up: copies under way land before the CTA's shared memory goes (a phase that a copy never began is waited
      // for in vain, until the limit)
      volatile int none = 0;
      for (uint32_t i = sc < (uint32_t)G::BS ? 0 : sc - G::BS; i < sc; ++i)
        none = 0, mbar_wait_bounded(&sh.b_full[i % G::BS], (i / G::BS) & 1u, &none, p.err, 2u);
      for (uint32_t i = cc < (uint32_t)kPvScalars ? 0 : cc - kPvScalars; i < cc; ++i)
        none = 0, mbar_wait_bounded(&sh.c_full[i % kPvScalars], (i / kPvScalars) & 1u, &none, p.err, 2u);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == W_MMA) {
    // no product is under way when the tensor memory goes back: the elected lane's commit speaks for its own products
    if (pc_elect()) {
      volatile int none = 0;
      mma_commit(&sh.drain);
      mbar_wait_bounded(&sh.drain, 0, &none, p.err, 2u);
    }
    __syncwarp();
    tmem_dealloc(tmem, 256);
  }
}

template <int BITS, int D>
cudaError_t pv_run(const QdaWeightsParams* p, bool prepare, cudaStream_t s) {
  auto kern = qda_paged_weights_tc_kernel<BITS, D>;
  constexpr int smem = pv_smem<D>();
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
