// Eviction from the paged cache by accumulated attention weight (sm_103a).
#include <algorithm>
#include <atomic>
#include <cstring>

#include <cooperative_groups.h>

#include "qda_paged_check.h"
#include "qda_ptx.cuh"

namespace qda {

namespace cg = cooperative_groups;

constexpr int kEvThreads = 256;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvHeld = 16384;      // keys that a CTA holds in shared memory (64 KB); those behind them are read again
constexpr int kEvBins = 2048;       // 11 bits of a rank at a time
constexpr int kEvFew = 256;         // ranks that are compared one by one
constexpr int kEvCluster = 8;

struct EvictParams {
  uint32_t *kp, *vp;
  uint16_t *ks, *kb, *vs, *vb;
  float* mass;
  int* token;
  const int* kv_len;
  int *new_len, *table, *freed, *n_freed, *shift;
  int B, Hkv, num_pages, page_shift, max_pages, max_freed, budget, limit, sinks, recent, W, NG;
  int most;                   // rows that a head can move
  int held;                   // keys of a CTA's piece in shared memory
  uint32_t *hole, *come;      // [B * Hkv, most] pool rows: the i-th of `come` goes to the i-th of `hole`
  int* moves;                 // [B * Hkv]
  unsigned int* err;
};

// A mass as an unsigned number that orders alike, zeros of either sign as one; no number ranks below all, and the highest pattern
// stays free.
__device__ __forceinline__ uint32_t ev_rank(float m) {
  const uint32_t u = __float_as_uint(m + 0.f);   // (-0 + 0 is 0; everything else stays as it is)
  return m != m ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// A row's rank: its mass, and of equal ones the lower row first. 32 bits of either.
__device__ __forceinline__ uint64_t ev_full(uint32_t key, int row) { return (uint64_t)key << 32 | (uint32_t)~row; }

struct alignas(16) EvShared {
  int hist[kEvBins];
  int coarse[kEvBins / 32];   // sums of 32 bins
  uint64_t few[kEvFew];       // this CTA's ranks that are left
  uint64_t all[kEvFew];       // the cluster's
  int warp[kEvWarps][2];
  int tot[2];                 // this CTA's counts, for the cluster
  int pick[3];                // bin, ranks above it, ranks in it
  int n_few;
  uint64_t edge;              // the budget-th rank
};

// One cluster per (sequence, KV head), a contiguous piece of its rows per CTA (ONE: clusters of one CTA). The budget-th
// largest rank is found by 11 bits at a time over histograms that the cluster adds up through distributed shared memory, and
// once no more than kEvFew ranks are left, by comparing them all. Ranks are all different (a row's number is part of its
// rank), so what stays is what is not below the edge. Then holes and rows that come are counted in order, a bit a row, and
// listed: the i-th hole meets the i-th row that comes, whatever the timing. A row's mass and token are read once. Limited by
// latency: loads two deep, then some ten barriers; reading all of the other CTAs' bins took half of the time (distributed
// shared memory is slow to read), so that sums of 32 bins come first and then the 32 that matter (32768 rows of eight heads: 43
// to 31 us, both kernels). It takes 14.6 us for 512 heads of 2049 rows in CTAs of their own, 20 us for eight of 32768 in clusters
// of eight, 23 us for 128 heads of 300 to 9001 rows in clusters of four. Comparing the last ranks instead of going on bit by bit:
// 43 to 29 us for the first.
template <bool ONE>
__global__ void __launch_bounds__(kEvThreads) qda_paged_evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_key[];   // keys, and behind them the pool row of every sixteenth row (-1: none)
  __shared__ EvShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = ONE ? 1 : cl.num_blocks(), me = ONE ? 0 : cl.block_rank();
  auto sync = [&]() {
    if constexpr (ONE) __syncthreads();
    else cl.sync();
  };
  auto of = [&](auto* x, int r) {
    if constexpr (ONE) return x;
    else return cl.map_shared_rank(x, r);
  };
  const int unit = blockIdx.x / cs, b = unit / p.Hkv, kvh = unit - b * p.Hkv;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  const int n = p.kv_len[b];
  const bool bad = n < 0 || n > (long long)p.max_pages << p.page_shift;
  if (bad || n <= p.limit) {   // (the whole cluster goes)
    if (me == 0 && tid == 0) {
      p.moves[unit] = 0;
      if (bad) atomicOr(p.err, QDA_ERR_BIT_PAGED);
    }
    return;
  }
  const int piece = (((n + cs - 1) / cs) + 31) & ~31;
  const int lo = (int)min((long long)n, (long long)piece * me), hi = (int)min((long long)n, (long long)lo + piece);
  const int pmask = (1 << p.page_shift) - 1;
  const int* tab = p.table + (size_t)b * p.max_pages;
  // the newest position that `recent` does not protect (counted down from the newest of all, which is below 2^31; the one behind
  // it need not be)
  const int old = n - 1 + (p.shift != nullptr ? p.shift[b] : 0) - p.recent;
  // (pool rows are below 2^32 - 1, which stands for a row that is not there)
  auto row_of = [&](int i) -> uint32_t {
    const int pg = __ldg(tab + (i >> p.page_shift));
    return (unsigned)pg < (unsigned)p.num_pages
               ? (((uint32_t)pg * (uint32_t)p.Hkv + (uint32_t)kvh) << p.page_shift) + (uint32_t)(i & pmask) : 0xffffffffu;
  };
  auto load_key = [&](int i) -> uint32_t {
    const uint32_t r = row_of(i);
    if (r == 0xffffffffu) {
      atomicOr(p.err, QDA_ERR_BIT_PAGED);
      return 0u;
    }
    const int t = __ldg(p.token + r);
    const uint32_t k = ev_rank(__ldg(p.mass + r));
    return t < p.sinks || t > old ? 0xffffffffu : k;
  };
  uint32_t* const s_row = s_key + p.held;
  // four rows of a page at a time (pages hold sixteens of rows, masses and tokens are aligned), four such loads on their way
  constexpr int LQ = 4;
  for (int i0 = lo + 4 * tid; i0 < min(hi, lo + p.held); i0 += LQ * 4 * kEvThreads) {
    uint32_t r[LQ];
    float4 m[LQ];
    int4 t[LQ];
#pragma unroll
    for (int u = 0; u < LQ; ++u) {
      const int i = i0 + u * 4 * kEvThreads;
      r[u] = i < min(hi, lo + p.held) ? row_of(i) : 0xfffffffeu;
    }
#pragma unroll
    for (int u = 0; u < LQ; ++u) {
      if (r[u] >= 0xfffffffeu) continue;
      m[u] = __ldg(reinterpret_cast<const float4*>(p.mass + r[u]));
      t[u] = __ldg(reinterpret_cast<const int4*>(p.token + r[u]));
    }
#pragma unroll
    for (int u = 0; u < LQ; ++u) {
      const int i = i0 + u * 4 * kEvThreads;
      if (r[u] == 0xfffffffeu) continue;
      uint4 k = make_uint4(0, 0, 0, 0);
      if (r[u] == 0xffffffffu) {
        atomicOr(p.err, QDA_ERR_BIT_PAGED);
      } else {
        auto rank = [&](float x, int y) { return y < p.sinks || y > old ? 0xffffffffu : ev_rank(x); };
        k = make_uint4(rank(m[u].x, t[u].x), rank(m[u].y, t[u].y), rank(m[u].z, t[u].z), rank(m[u].w, t[u].w));
      }
      *reinterpret_cast<uint4*>(s_key + i - lo) = k;   // (a piece's room is a multiple of 32 keys)
      if ((i & 15) == 0) s_row[(i - lo) >> 4] = r[u];
    }
  }
  auto key_at = [&](int i) { return i - lo < p.held ? s_key[i - lo] : load_key(i); };
  auto row_at = [&](int i) {
    if (i - lo >= p.held) return row_of(i);
    const uint32_t r = s_row[(i - lo) >> 4];
    return r == 0xffffffffu ? r : r + (i & 15);
  };
  // f(key, row) for the CTA's rows that have the known bits
  auto each = [&](uint64_t prefix, int known, auto&& f) {
    if (known <= 32) {
      const uint32_t want = (uint32_t)prefix;
      const int shift = 32 - known;
      for (int i = lo + tid; i < hi; i += kEvThreads) {
        const uint32_t k = key_at(i);
        if (known == 0 || (k >> shift) == want) f(k, i);
      }
    } else {
      for (int i = lo + tid; i < hi; i += kEvThreads) {
        const uint32_t k = key_at(i);
        if ((ev_full(k, i) >> (64 - known)) == prefix) f(k, i);
      }
    }
  };

  // ---- the budget-th largest rank
  uint64_t prefix = 0;        // the bits that are known, from the top
  int known = 0;
  int above = 0, left = n;    // ranks above the prefix, ranks that have it
  while (left > kEvFew) {     // (64 known bits leave one)
    const int width = min(11, 64 - known), shift = 64 - known - width;
    for (int i = tid; i < kEvBins / 4; i += kEvThreads) reinterpret_cast<int4*>(sh.hist)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    if (shift >= 32) {
      each(prefix, known, [&](uint32_t k, int) { atomicAdd(&sh.hist[(k >> (shift - 32)) & ((1u << width) - 1)], 1); });
    } else {
      each(prefix, known, [&](uint32_t k, int i) { atomicAdd(&sh.hist[(ev_full(k, i) >> shift) & ((1u << width) - 1)], 1); });
    }
    __syncthreads();
    {   // eight bins a thread, four threads a sum
      const int4 *h = reinterpret_cast<const int4*>(sh.hist + 8 * tid), u = h[0], v = h[1];
      int x = (u.x + u.y) + (u.z + u.w) + (v.x + v.y) + (v.z + v.w);
      x += __shfl_xor_sync(0xffffffffu, x, 1);
      x += __shfl_xor_sync(0xffffffffu, x, 2);
      if ((tid & 3) == 0) sh.coarse[tid >> 2] = x;
    }
    sync();
    if (warp == 0) {
      // the cluster's sums, the highest bins first: two a lane, the bin of 32 that holds the budget-th rank, then its 32
      auto gather = [&](const int* x) {
        int v[ONE ? 1 : kEvCluster], sum = 0;
#pragma unroll
        for (int r = 0; r < (ONE ? 1 : kEvCluster); ++r) v[r] = r < cs ? *of(x, r) : 0;
#pragma unroll
        for (int r = 0; r < (ONE ? 1 : kEvCluster); ++r) sum += v[r];
        return sum;
      };
      auto scan = [&](int x) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, x, o);
          if (lane >= o) x += v;
        }
        return x;
      };
      const int c0 = gather(sh.coarse + 63 - 2 * lane), c1 = gather(sh.coarse + 62 - 2 * lane);
      int before = above + scan(c0 + c1) - c0 - c1;   // ranks in higher bins
      const bool in0 = before < p.budget && before + c0 >= p.budget;
      const bool in1 = before + c0 < p.budget && before + c0 + c1 >= p.budget;
      const uint32_t who = __ballot_sync(0xffffffffu, in0 || in1);
      const int src = __ffs(who) - 1;
      const int group = __shfl_sync(0xffffffffu, in0 ? 63 - 2 * lane : 62 - 2 * lane, src);
      before = __shfl_sync(0xffffffffu, in0 ? before : before + c0, src);
      const int c = gather(sh.hist + 32 * group + 31 - lane);
      before += scan(c) - c;
      if (before < p.budget && before + c >= p.budget) {
        sh.pick[0] = 32 * group + 31 - lane;
        sh.pick[1] = before;
        sh.pick[2] = c;
      }
    }
    sync();   // every CTA has read the histograms
    prefix = prefix << width | (uint32_t)sh.pick[0];
    known += width;
    above = sh.pick[1];
    left = sh.pick[2];
  }
  // ---- the ranks that are left, all of them against each other
  if (tid == 0) sh.n_few = 0;
  __syncthreads();
  each(prefix, known, [&](uint32_t k, int i) { sh.few[atomicAdd(&sh.n_few, 1)] = ev_full(k, i); });   // (in any order; few)
  sync();
  const uint64_t* all = sh.few;
  if constexpr (!ONE) {   // every CTA takes all of them, and finds the edge for itself
    int m[kEvCluster];
    uint64_t k[kEvCluster];
#pragma unroll
    for (int r = 0; r < kEvCluster; ++r) m[r] = r < cs ? *cl.map_shared_rank(&sh.n_few, r) : 0;
#pragma unroll
    for (int r = 0; r < kEvCluster; ++r) k[r] = tid < m[r] ? cl.map_shared_rank(sh.few, r)[tid] : 0;
    int at = tid;
#pragma unroll
    for (int r = 0; r < kEvCluster; ++r) {
      if (tid < m[r]) sh.all[at] = k[r];
      at += m[r];
    }
    all = sh.all;
    __syncthreads();
  }
  if (tid < left) {
    const uint64_t k = all[tid];
    int higher = above;
#pragma unroll 8
    for (int i = 0; i < left; ++i) higher += all[i] > k;
    if (higher == p.budget - 1) sh.edge = k;
  }
  __syncthreads();
  const uint32_t edge_key = (uint32_t)(sh.edge >> 32);
  const int edge_row = (int)~(uint32_t)sh.edge;

  // ---- rows in order, 32 at a time as the bits of a word: holes and rows that come before each
  const int words = (hi - lo + 31) >> 5;
  const uint32_t below = (1u << lane) - 1;
  // rows of word w that lie before the budget
  auto inside = [&](int w) {
    const int c = p.budget - (lo + 32 * w);
    return c >= 32 ? 0xffffffffu : c <= 0 ? 0u : (1u << c) - 1;
  };
  auto real = [&](int w) {
    const int c = hi - (lo + 32 * w);
    return c >= 32 ? 0xffffffffu : (1u << c) - 1;
  };
  auto stays = [&](int w) {
    const int i = lo + 32 * w + lane;
    const uint32_t k = i < hi ? key_at(i) : 0u;
    return __ballot_sync(0xffffffffu, i < hi && (k > edge_key || (k == edge_key && i <= edge_row)));
  };
  int holes = 0, comes = 0;   // of this warp's words: contiguous, so that warps are in order
  const int part = (words + kEvWarps - 1) / kEvWarps, w_lo = min(words, part * warp), w_hi = min(words, w_lo + part);
  uint32_t kept = 0;          // lane l: the bits of the warp's word l, where it has no more than 32
#pragma unroll 2
  for (int w = w_lo; w < w_hi; ++w) {
    const uint32_t stay = stays(w);
    if (lane == ((w - w_lo) & 31)) kept = stay;
    holes += __popc(~stay & inside(w) & real(w));
    comes += __popc(stay & ~inside(w));
  }
  if (lane == 0) {
    sh.warp[warp][0] = holes;
    sh.warp[warp][1] = comes;
  }
  __syncthreads();
  int h_at = 0, c_at = 0, h_all = 0, c_all = 0;
#pragma unroll
  for (int w = 0; w < kEvWarps; ++w) {
    const int x = sh.warp[w][0], y = sh.warp[w][1];
    h_at += w < warp ? x : 0;
    c_at += w < warp ? y : 0;
    h_all += x;
    c_all += y;
  }
  if constexpr (!ONE) {
    if (tid == 0) {
      sh.tot[0] = h_all;
      sh.tot[1] = c_all;
    }
    cl.sync();
    for (int r = 0; r < me; ++r) {
      const int* t = cl.map_shared_rank(sh.tot, r);
      h_at += t[0];
      c_at += t[1];
    }
    cl.sync();   // (no CTA goes while another reads its counts)
  }
  if (me == cs - 1 && tid == kEvThreads - 32) p.moves[unit] = h_at + holes;
  uint32_t* const hole_list = p.hole + (size_t)unit * p.most;
  uint32_t* const come_list = p.come + (size_t)unit * p.most;
  for (int w = w_lo; w < w_hi; ++w) {
    const uint32_t stay = part <= 32 ? __shfl_sync(0xffffffffu, kept, (w - w_lo) & 31) : stays(w);
    const uint32_t h = ~stay & inside(w) & real(w), c = stay & ~inside(w);
    if ((h | c) == 0) continue;   // (the whole warp)
    if (((h | c) >> lane) & 1u) {
      const bool hole = (h >> lane) & 1u;
      const int j = hole ? h_at + __popc(h & below) : c_at + __popc(c & below);
      if (j < p.most) (hole ? hole_list : come_list)[j] = row_at(lo + 32 * w + lane);
    }
    h_at += __popc(h);
    c_at += __popc(c);
  }
}

// The rows that come are copied to the holes: a lane has one fixed piece of a row (16 bytes of codes, scales or biases, its
// mass, its token) and walks the rows, so that its addresses are a multiplication and an addition. Sources lie behind the
// budget and holes before it: no order among CTAs matters. CTA (0, 0) also does the lengths and the table, which the
// selection has read and this kernel's other CTAs do not. Rows are read where they lie, 512 bytes and less at a place, so that
// latency binds before HBM does: 25 us for 100 MB of rows (D 256, 8-bit; HBM at 50 %), 7 us for one row of each of 512 heads.
constexpr int kEvMoveThreads = 256;

__global__ void __launch_bounds__(kEvMoveThreads) qda_paged_evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int s_first[QDA_MAX_B + 1];
  __shared__ int s_count[kEvMoveThreads / 32];
  const int tid = threadIdx.x;
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    // table entries that go before each sequence's, the first sequences' first
    if (tid < 32) {
      int carry = 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + tid;
        int pages = 0;
        if (b < p.B) {
          const int n = p.kv_len[b];
          const bool cut = n > p.limit && n <= (long long)p.max_pages << p.page_shift;
          const int pmask = (1 << p.page_shift) - 1;
          if (cut) {
            pages = (int)(((long long)n + pmask) >> p.page_shift) - (int)(((long long)p.budget + pmask) >> p.page_shift);
            if (p.shift != nullptr) p.shift[b] += n - p.budget;
          }
          p.new_len[b] = cut ? p.budget : n;
        }
        int up = pages;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, up, o);
          if (tid >= o) up += v;
        }
        if (b < p.B) s_first[b] = carry + up - pages;
        carry += __shfl_sync(0xffffffffu, up, 31);
      }
      if (tid == 0) s_first[p.B] = carry;
    }
    __syncthreads();
    const int keep = (int)(((long long)p.budget + (1 << p.page_shift) - 1) >> p.page_shift);
    const int total = s_first[p.B];
    auto entry = [&](int i) {
      const int b = qda_seq_of(s_first, p.B, i);
      return p.table + (size_t)b * p.max_pages + keep + (i - s_first[b]);
    };
    bool absent = false;   // entries outside the pool leave the table, but are no pages that could be given back
#pragma unroll 4
    for (int i = tid; i < total; i += kEvMoveThreads) absent |= (unsigned)*entry(i) >= (unsigned)p.num_pages;
    int at = total;
    if (!__syncthreads_or(absent)) {
      for (int i = tid; i < total; i += kEvMoveThreads) {
        int* e = entry(i);
        if (i < p.max_freed) p.freed[i] = *e;
        *e = -1;
      }
    } else {
      const int lane = tid & 31, warp = tid >> 5;
      at = 0;
      for (int i0 = 0; i0 < total; i0 += kEvMoveThreads) {
        int pg = -1;
        if (i0 + tid < total) {
          int* e = entry(i0 + tid);
          pg = *e;
          *e = -1;
        }
        const bool real = (unsigned)pg < (unsigned)p.num_pages;
        const uint32_t some = __ballot_sync(0xffffffffu, real);
        if (lane == 0) s_count[warp] = __popc(some);
        __syncthreads();
        int to = at + __popc(some & ((1u << lane) - 1));
        for (int w = 0; w < kEvMoveThreads / 32; ++w) {
          to += w < warp ? s_count[w] : 0;
          at += s_count[w];
        }
        if (real && to < p.max_freed) p.freed[to] = pg;
        __syncthreads();
      }
    }
    if (tid == 0) {
      p.n_freed[0] = at;
      if (at > p.max_freed) atomicOr(p.err, QDA_ERR_BIT_PAGED);
    }
  }
  const int unit = blockIdx.y, moves = min(p.moves[unit], p.most);
  if (moves == 0) return;
  const uint32_t* hole = p.hole + (size_t)unit * p.most;
  const uint32_t* come = p.come + (size_t)unit * p.most;
  // pieces of a row: K codes, V codes (16 bytes each), scales and biases (up to 16 bytes each), mass, token. Many codes go by
  // themselves, a power of two of lanes to a row; the rest then takes 8 or 16 lanes.
  const int cq = p.W / 4, sb = p.NG * 2, sp = sb > 16 ? sb / 16 : 1;
  const int small = 4 * sp + 2, codes = 2 * cq;
  auto copy = [&](int first, int pieces, int lanes) {
    const int sub = tid / lanes, group = kEvMoveThreads / lanes, per = group * gridDim.x;
    for (int it = first + tid % lanes; it < first + pieces; it += lanes) {
      char* base;
      int stride, size, off;
      if (it < codes) {
        base = reinterpret_cast<char*>(it < cq ? p.kp : p.vp);
        stride = p.W * 4;
        size = 16;
        off = (it < cq ? it : it - cq) * 16;
      } else if (it < codes + 4 * sp) {
        const int j = it - codes, a = j / sp;
        base = reinterpret_cast<char*>(a == 0 ? p.ks : a == 1 ? p.kb : a == 2 ? p.vs : p.vb);
        stride = sb;
        size = min(sb, 16);
        off = (j - a * sp) * 16;
      } else {
        base = it == codes + small - 1 ? reinterpret_cast<char*>(p.token) : reinterpret_cast<char*>(p.mass);
        stride = size = 4;
        off = 0;
      }
      base += off;
      constexpr int U = 4;
      for (int i0 = blockIdx.x * group + sub; i0 < moves; i0 += U * per) {
        uint32_t f[U], t[U];
        uint4 v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * per;
          f[u] = i < moves ? come[i] : 0xffffffffu;
          t[u] = i < moves ? hole[i] : 0xffffffffu;
          if (t[u] == 0xffffffffu) f[u] = t[u];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (f[u] == 0xffffffffu) continue;
          const char* src = base + (uint64_t)f[u] * stride;
          if (size == 16) v[u] = *reinterpret_cast<const uint4*>(src);
          else if (size == 8) *reinterpret_cast<uint2*>(&v[u]) = *reinterpret_cast<const uint2*>(src);
          else if (size == 4) v[u].x = *reinterpret_cast<const uint32_t*>(src);
          else v[u].x = *reinterpret_cast<const uint16_t*>(src);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (f[u] == 0xffffffffu) continue;
          char* dst = base + (uint64_t)t[u] * stride;
          if (size == 16) *reinterpret_cast<uint4*>(dst) = v[u];
          else if (size == 8) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(&v[u]);
          else if (size == 4) *reinterpret_cast<uint32_t*>(dst) = v[u].x;
          else *reinterpret_cast<uint16_t*>(dst) = (uint16_t)v[u].x;
        }
      }
    }
  };
  if (codes + small <= 16) {
    copy(0, codes + small, 16);
  } else {
    copy(0, codes, min(codes, 32));
    copy(codes, small, small <= 8 ? 8 : 16);
  }
}

struct EvictPlan {
  int cluster, held, move_x;
  long long most;
  size_t list_bytes, bytes;
};

static EvictPlan evict_plan(int B, int Hkv, long long rows, int budget, int sms) {
  EvictPlan e;
  const int units = B * Hkv;
  // CTAs per head: enough to fill the SMs, none with room for less than 2048 rows. Room is the table's: lengths are not known here,
  // and a short sequence of a wide table is cut as finely as a long one. Room in shared memory goes by the table too: one row
  // each from 512 heads of 2049 takes 17.4 us with tables of 33 to 128 pages of 64, 21.5 with 256 and 22.5 with 512 and more, where
  // CTAs of 82 KB leave an SM two.
  e.cluster = kEvCluster;
  while (e.cluster > 1 && ((long long)units * e.cluster > 4LL * sms || rows < 2048LL * e.cluster)) e.cluster /= 2;
  e.held = (int)std::min<long long>(kEvHeld, ((rows + e.cluster - 1) / e.cluster + 31) & ~31LL);
  e.most = std::max(1LL, std::min((long long)budget, rows - budget));
  e.list_bytes = ((size_t)units * e.most * 4 + 255) & ~(size_t)255;
  e.bytes = 2 * e.list_bytes + (size_t)units * 4;
  e.move_x = (int)std::max(1LL, std::min((8LL * sms + units - 1) / units, (e.most + 63) / 64));
  return e;
}

}  // namespace qda

extern "C" int qdecode_paged_evict_workspace_bytes(int B, int Hkv, int page, int max_pages, int budget, size_t* bytes) {
  using namespace qda;
  if (bytes == nullptr || B < 1 || Hkv < 1 || page < 1 || max_pages < 1 || budget < 1) return QDA_ERR_INVALID;
  if (B > QDA_MAX_B || Hkv > QDA_EVICT_MAX_HEADS || !good_page(page)) return QDA_ERR_UNSUPPORTED;
  *bytes = evict_plan(B, Hkv, (long long)max_pages * page, budget, 1).bytes;
  return QDA_OK;
}

extern "C" int qdecode_paged_evict(uint32_t* k_packed, void* k_scales, void* k_biases, uint32_t* v_packed, void* v_scales,
                                   void* v_biases, float* mass, int32_t* token, const int32_t* kv_len, int32_t* new_len,
                                   int32_t* block_table, int32_t* freed, int32_t* n_freed, int32_t* shift, int B, int Hkv,
                                   int num_pages, int page, int max_pages, int max_freed, int budget, int limit, int sinks,
                                   int recent, int D, int GS, int bits, void* stream) {
  using namespace qda;
  if (!k_packed || !k_scales || !k_biases || !v_packed || !v_scales || !v_biases || !mass || !token || !kv_len || !new_len ||
      !block_table || !n_freed)
    return QDA_ERR_INVALID;
  if (B < 1 || Hkv < 1 || max_pages < 1 || max_freed < 0 || (max_freed > 0 && !freed)) return QDA_ERR_INVALID;
  if (budget < 1 || limit < budget || sinks < 0 || recent < 0 || (long long)sinks + recent > budget) return QDA_ERR_INVALID;
  int st = check_codec(D, GS, bits);
  if (st == QDA_OK) st = check_pool(num_pages, page);
  if (st != QDA_OK) return st;
  if (B > QDA_MAX_B || Hkv > QDA_EVICT_MAX_HEADS) return QDA_ERR_UNSUPPORTED;
  if ((long long)num_pages * page * Hkv >= 0xffffffffLL) return QDA_ERR_UNSUPPORTED;   // pool rows are 32-bit
  if ((long long)max_pages * page > 0x7ffffe00LL) return QDA_ERR_UNSUPPORTED;
  const void* ptrs[8] = {k_packed, k_scales, k_biases, v_packed, v_scales, v_biases, mass, token};
  for (const void* p : ptrs)
    if (off16(p)) return QDA_ERR_ALIGN;
  const void* words[6] = {kv_len, new_len, block_table, freed, n_freed, shift};
  for (const void* p : words)
    if (off4(p)) return QDA_ERR_ALIGN;
  // lengths are read, and new ones and shifts written, a warp of sequences after the other
  auto apart = [&](const int32_t* x, const int32_t* y) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(x), b = reinterpret_cast<uintptr_t>(y);
    return x == nullptr || y == nullptr || (a < b ? b - a : a - b) >= 4 * (uintptr_t)B;
  };
  if (!apart(kv_len, new_len) || !apart(kv_len, shift) || !apart(new_len, shift)) return QDA_ERR_INVALID;
  EvictParams p;
  std::memset(&p, 0, sizeof(p));
  int sms;
  st = qda_device(&sms, &p.err);
  if (st != QDA_OK) return st;
  const EvictPlan e = evict_plan(B, Hkv, (long long)max_pages * page, budget, sms);
  void* ws = nullptr;
  st = qda_workspace(e.bytes, &ws);
  if (st != QDA_OK) return st;
  p.kp = k_packed;
  p.vp = v_packed;
  p.ks = static_cast<uint16_t*>(k_scales);
  p.kb = static_cast<uint16_t*>(k_biases);
  p.vs = static_cast<uint16_t*>(v_scales);
  p.vb = static_cast<uint16_t*>(v_biases);
  p.mass = mass;
  p.token = token;
  p.kv_len = kv_len;
  p.new_len = new_len;
  p.table = block_table;
  p.freed = freed;
  p.n_freed = n_freed;
  p.shift = shift;
  p.B = B;
  p.Hkv = Hkv;
  p.num_pages = num_pages;
  p.page_shift = page_shift_of(page);
  p.max_pages = max_pages;
  p.max_freed = max_freed;
  p.budget = budget;
  p.limit = limit;
  p.sinks = sinks;
  p.recent = recent;
  p.W = D * bits / 32;
  p.NG = D / GS;
  p.most = (int)e.most;
  p.held = e.held;
  p.hole = static_cast<uint32_t*>(ws);
  p.come = reinterpret_cast<uint32_t*>(static_cast<char*>(ws) + e.list_bytes);
  p.moves = reinterpret_cast<int*>(static_cast<char*>(ws) + 2 * e.list_bytes);
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  int dev = 0;
  cudaError_t ce = cudaGetDevice(&dev);
  if (ce != cudaSuccess || dev < 0 || dev >= 64) return qda_cuda_fail(ce == cudaSuccess ? cudaErrorInvalidDevice : ce);
  static std::atomic<bool> ready[64] = {};
  if (!ready[dev].load()) {
    constexpr int most = kEvHeld * 4 + kEvHeld / 4;
    ce = cudaFuncSetAttribute(qda_paged_evict_select_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (ce == cudaSuccess)
      ce = cudaFuncSetAttribute(qda_paged_evict_select_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (ce != cudaSuccess) return qda_cuda_fail(ce);
    ready[dev].store(true);
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * Hkv * e.cluster));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = (size_t)e.held * 4 + e.held / 4;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)e.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ce = e.cluster == 1 ? cudaLaunchKernelEx(&cfg, qda_paged_evict_select_kernel<true>, p)
                      : cudaLaunchKernelEx(&cfg, qda_paged_evict_select_kernel<false>, p);
  if (ce != cudaSuccess) return qda_cuda_fail(ce);
  cfg.gridDim = dim3((unsigned)e.move_x, (unsigned)(B * Hkv));
  cfg.blockDim = dim3(kEvMoveThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  ce = cudaLaunchKernelEx(&cfg, qda_paged_evict_move_kernel, p);
  return ce == cudaSuccess ? QDA_OK : qda_cuda_fail(ce);
}
