// Eviction from the paged cache by accumulated attention weight (sm_103a).
#include <algorithm>
#include <atomic>
#include <cstring>

#include <cooperative_groups.h>

#include "qda_paged_check.h"
#include "qda_ptx.cuh"

namespace qda {

namespace cg = cooperative_groups;

constexpr int kEvThreads = 512;
constexpr int kEvWarps = kEvThreads / 32;
constexpr int kEvHeld = 16384;      // keys that a CTA holds in shared memory (64 KB); those behind them are read again
constexpr int kEvBins = 2048;       // 11 bits of a key at a time
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

// A mass as an unsigned number that orders alike; no number ranks below all, and the highest pattern stays free.
__device__ __forceinline__ uint32_t ev_rank(float m) {
  const uint32_t u = __float_as_uint(m);
  return m != m ? 0u : (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

struct alignas(16) EvShared {
  int hist[kEvBins];
  int warp[kEvWarps][2];
  int tot[2];                 // this CTA's counts, for the cluster
  int pick[2];                // bin, keys above it
};

// One cluster per (sequence, KV head), a contiguous piece of its rows per CTA. The rank of the budget-th key is found by 11
// bits at a time over histograms that the cluster adds up through distributed shared memory; then rows are counted in order
// (ballots in a warp, warps and CTAs through prefix sums), so that ties fall to the lowest rows and the i-th hole meets the
// i-th row that comes, whatever the timing. A row's mass and token are read once.
__global__ void __launch_bounds__(kEvThreads) qda_paged_evict_select_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ uint32_t s_key[];
  __shared__ EvShared sh;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = cl.num_blocks(), me = cl.block_rank();
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
  const int seen = n + (p.shift != nullptr ? p.shift[b] : 0);
  const int young = seen - p.recent;
  auto row_of = [&](int i) -> long long {
    const int pg = tab[i >> p.page_shift];
    return (unsigned)pg < (unsigned)p.num_pages ? qda_pool_row(pg, kvh, i & pmask, p.Hkv, p.page_shift) : -1;
  };
  auto load_key = [&](int i) -> uint32_t {
    const long long r = row_of(i);
    if (r < 0) {
      atomicOr(p.err, QDA_ERR_BIT_PAGED);
      return 0u;
    }
    const int t = p.token[r];
    const uint32_t k = ev_rank(p.mass[r]);
    return t < p.sinks || t >= young ? 0xffffffffu : k;
  };
  for (int i = lo + tid; i < min(hi, lo + p.held); i += kEvThreads) s_key[i - lo] = load_key(i);
  auto key_at = [&](int i) { return i - lo < p.held ? s_key[i - lo] : load_key(i); };

  // ---- the budget-th largest key
  uint32_t prefix = 0;
  int above = 0;              // keys above the prefix
  int equal = 0;
  constexpr int SHIFT[3] = {21, 10, 0}, WIDTH[3] = {11, 11, 10};
#pragma unroll
  for (int pass = 0; pass < 3; ++pass) {
    for (int i = tid; i < kEvBins; i += kEvThreads) sh.hist[i] = 0;
    __syncthreads();
    const int up = SHIFT[pass] + WIDTH[pass];
    for (int i = lo + tid; i < hi; i += kEvThreads) {
      const uint32_t k = key_at(i);
      if (pass == 0 || (k >> (up & 31)) == prefix) atomicAdd(&sh.hist[(k >> SHIFT[pass]) & ((1 << WIDTH[pass]) - 1)], 1);
    }
    cl.sync();
    // the cluster's counts of four bins a thread, highest bins first
    int c[4] = {0, 0, 0, 0};
    const int bin0 = kEvBins - 4 - 4 * tid;
    for (int r = 0; r < cs; ++r) {
      const int4 v = *reinterpret_cast<const int4*>(cl.map_shared_rank(sh.hist, r) + bin0);
      c[0] += v.w;
      c[1] += v.z;
      c[2] += v.y;
      c[3] += v.x;
    }
    const int mine = c[0] + c[1] + c[2] + c[3];
    int up_to = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, up_to, o);
      if (lane >= o) up_to += v;
    }
    if (lane == 31) sh.warp[warp][0] = up_to;
    __syncthreads();
    for (int w = 0; w < warp; ++w) up_to += sh.warp[w][0];
    int before = above + up_to - mine;   // keys in higher bins
    if (before < p.budget && before + mine >= p.budget) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (before < p.budget && before + c[j] >= p.budget) {
          sh.pick[0] = bin0 + 3 - j;
          sh.pick[1] = before;
          sh.tot[0] = c[j];
        }
        before += c[j];
      }
    }
    __syncthreads();
    prefix = pass == 0 ? (uint32_t)sh.pick[0] : (prefix << WIDTH[pass]) | (uint32_t)sh.pick[0];
    above = sh.pick[1];
    equal = sh.tot[0];
    cl.sync();   // every CTA has read the histograms
  }
  const uint32_t edge = prefix;
  const int ties = p.budget - above;   // rows of that rank that stay, lowest first

  // ---- rows in order: a warp takes a contiguous part of the CTA's piece, 32 rows at a time
  const int part = ((hi - lo + kEvWarps - 1) / kEvWarps + 31) & ~31;
  const int w_lo = min(hi, lo + part * warp), w_hi = min(hi, w_lo + part);
  // sums over the warps and CTAs before this one, of two counts of each warp
  auto before_of = [&](int x, int y) {
    if (lane == 0) {
      sh.warp[warp][0] = x;
      sh.warp[warp][1] = y;
    }
    __syncthreads();
    int2 mine = make_int2(0, 0), all = make_int2(0, 0);
    for (int w = 0; w < kEvWarps; ++w) {
      const int2 v = make_int2(sh.warp[w][0], sh.warp[w][1]);
      if (w < warp) {
        mine.x += v.x;
        mine.y += v.y;
      }
      all.x += v.x;
      all.y += v.y;
    }
    if (tid == 0) {
      sh.tot[0] = all.x;
      sh.tot[1] = all.y;
    }
    cl.sync();
    for (int r = 0; r < me; ++r) {
      const int* t = cl.map_shared_rank(sh.tot, r);
      mine.x += t[0];
      mine.y += t[1];
    }
    cl.sync();
    return mine;
  };
  int tied = 0;   // rows of the edge's rank before this warp's part
  if (ties < equal) {
    int c = 0;
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      const int i = i0 + lane;
      c += __popc(__ballot_sync(0xffffffffu, i < w_hi && key_at(i) == edge));
    }
    tied = before_of(c, 0).x;
  }
  const uint32_t below = (1u << lane) - 1;
  // f(row, stays) for the rows of a 32-wide step
  auto walk = [&](auto&& f) {
    int t = tied;
    for (int i0 = w_lo; i0 < w_hi; i0 += 32) {
      const int i = i0 + lane;
      const bool in = i < w_hi;
      const uint32_t k = in ? key_at(i) : 0u;
      bool stays = in && k > edge;
      const uint32_t eq = __ballot_sync(0xffffffffu, in && k == edge);
      if (in && k == edge) stays = ties >= equal || t + __popc(eq & below) < ties;
      t += __popc(eq);
      f(i, in && !stays && i < p.budget, stays && i >= p.budget);
    }
  };
  int holes = 0, comes = 0;
  walk([&](int, bool hole, bool come) {
    holes += __popc(__ballot_sync(0xffffffffu, hole));
    comes += __popc(__ballot_sync(0xffffffffu, come));
  });
  int2 at = before_of(holes, comes);
  if (me == cs - 1 && warp == kEvWarps - 1 && lane == 0) p.moves[unit] = at.x + holes;
  uint32_t* const hole_list = p.hole + (size_t)unit * p.most;
  uint32_t* const come_list = p.come + (size_t)unit * p.most;
  walk([&](int i, bool hole, bool come) {
    const uint32_t h = __ballot_sync(0xffffffffu, hole), c = __ballot_sync(0xffffffffu, come);
    if (hole || come) {
      const uint32_t r = (uint32_t)row_of(i);   // (-1: no such row; pool rows are below 2^32 - 1)
      const int j = hole ? at.x + __popc(h & below) : at.y + __popc(c & below);
      if (j < p.most) (hole ? hole_list : come_list)[j] = r;
    }
    at.x += __popc(h);
    at.y += __popc(c);
  });
}

// The rows that come are copied to the holes: a lane has one fixed piece of a row (16 bytes of codes, scales or biases, its
// mass, its token) and walks the rows, so that its addresses are a multiplication and an addition. Sources lie behind the
// budget and holes before it: no order among CTAs matters. CTA (0, 0) also does the lengths and the table, which the
// selection has read and this kernel's other CTAs do not.
constexpr int kEvMoveThreads = 256;

__global__ void __launch_bounds__(kEvMoveThreads) qda_paged_evict_move_kernel(const __grid_constant__ EvictParams p) {
  __shared__ int s_first[QDA_MAX_B + 1];
  const int tid = threadIdx.x;
  pdl_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0) {
    // freed pages before each sequence, the first sequences' first
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
      if (tid == 0) {
        s_first[p.B] = carry;
        p.n_freed[0] = carry;
        if (carry > p.max_freed) atomicOr(p.err, QDA_ERR_BIT_PAGED);
      }
    }
    __syncthreads();
    const int keep = (int)(((long long)p.budget + (1 << p.page_shift) - 1) >> p.page_shift);
    for (int i = tid; i < s_first[p.B]; i += kEvMoveThreads) {
      const int b = qda_seq_of(s_first, p.B, i);
      int* e = p.table + (size_t)b * p.max_pages + keep + (i - s_first[b]);
      if (i < p.max_freed) p.freed[i] = *e;
      *e = -1;
    }
  }
  const int unit = blockIdx.y, moves = min(p.moves[unit], p.most);
  if (moves == 0) return;
  const uint32_t* hole = p.hole + (size_t)unit * p.most;
  const uint32_t* come = p.come + (size_t)unit * p.most;
  // pieces of a row: K codes, V codes (16 bytes each), scales and biases (up to 16 bytes each), mass, token
  const int cq = p.W / 4, sb = p.NG * 2, sp = sb > 16 ? sb / 16 : 1;
  const int pieces = 2 * cq + 4 * sp + 2;
  const int lanes = pieces <= 8 ? 8 : pieces <= 16 ? 16 : 32;
  const int sub = tid / lanes, per = kEvMoveThreads / lanes * gridDim.x;
  for (int it = tid % lanes; it < pieces; it += lanes) {
    char* base;
    int stride, size, off;
    if (it < 2 * cq) {
      base = reinterpret_cast<char*>(it < cq ? p.kp : p.vp);
      stride = p.W * 4;
      size = 16;
      off = (it < cq ? it : it - cq) * 16;
    } else if (it < 2 * cq + 4 * sp) {
      const int j = it - 2 * cq, a = j / sp;
      base = reinterpret_cast<char*>(a == 0 ? p.ks : a == 1 ? p.kb : a == 2 ? p.vs : p.vb);
      stride = sb;
      size = min(sb, 16);
      off = (j - a * sp) * 16;
    } else {
      base = it == pieces - 1 ? reinterpret_cast<char*>(p.token) : reinterpret_cast<char*>(p.mass);
      stride = size = 4;
      off = 0;
    }
    constexpr int U = 4;
    for (int i0 = blockIdx.x * (kEvMoveThreads / lanes) + sub; i0 < moves; i0 += U * per) {
      const char* src[U];
      char* dst[U];
      uint4 v[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * per;
        const uint32_t f = i < moves ? come[i] : 0xffffffffu, t = i < moves ? hole[i] : 0xffffffffu;
        src[u] = f == 0xffffffffu || t == 0xffffffffu ? nullptr : base + (uint64_t)f * stride + off;
        dst[u] = base + (uint64_t)t * stride + off;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (src[u] == nullptr) continue;
        if (size == 16) v[u] = *reinterpret_cast<const uint4*>(src[u]);
        else if (size == 8) *reinterpret_cast<uint2*>(&v[u]) = *reinterpret_cast<const uint2*>(src[u]);
        else if (size == 4) v[u].x = *reinterpret_cast<const uint32_t*>(src[u]);
        else v[u].x = *reinterpret_cast<const uint16_t*>(src[u]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (src[u] == nullptr) continue;
        if (size == 16) *reinterpret_cast<uint4*>(dst[u]) = v[u];
        else if (size == 8) *reinterpret_cast<uint2*>(dst[u]) = *reinterpret_cast<uint2*>(&v[u]);
        else if (size == 4) *reinterpret_cast<uint32_t*>(dst[u]) = v[u].x;
        else *reinterpret_cast<uint16_t*>(dst[u]) = (uint16_t)v[u].x;
      }
    }
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
  // CTAs per head: enough to fill the SMs, none with less than 2048 rows
  e.cluster = kEvCluster;
  while (e.cluster > 1 && ((long long)units * e.cluster > 2LL * sms || rows < 2048LL * e.cluster)) e.cluster /= 2;
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
  if (B < 1 || Hkv < 1 || max_pages < 1 || max_freed < 0 || (max_freed > 0 && !freed) || new_len == kv_len) return QDA_ERR_INVALID;
  if (budget < 1 || limit < budget || sinks < 0 || recent < 0 || (long long)sinks + recent > budget) return QDA_ERR_INVALID;
  int st = check_codec(D, GS, bits);
  if (st == QDA_OK) st = check_pool(num_pages, page);
  if (st != QDA_OK) return st;
  if (B > QDA_MAX_B || Hkv > QDA_EVICT_MAX_HEADS) return QDA_ERR_UNSUPPORTED;
  if ((long long)num_pages * page * Hkv >= 0xffffffffLL) return QDA_ERR_UNSUPPORTED;   // pool rows are 32-bit
  if ((long long)max_pages * page > 0x7ffffe00LL) return QDA_ERR_UNSUPPORTED;
  const void* ptrs[6] = {k_packed, k_scales, k_biases, v_packed, v_scales, v_biases};
  for (const void* p : ptrs)
    if (off16(p)) return QDA_ERR_ALIGN;
  const void* words[8] = {mass, token, kv_len, new_len, block_table, freed, n_freed, shift};
  for (const void* p : words)
    if (off4(p)) return QDA_ERR_ALIGN;
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
    ce = cudaFuncSetAttribute(qda_paged_evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kEvHeld * 4);
    if (ce != cudaSuccess) return qda_cuda_fail(ce);
    ready[dev].store(true);
  }
  cudaLaunchAttribute attr[1];
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * Hkv * e.cluster));
  cfg.blockDim = dim3(kEvThreads);
  cfg.dynamicSmemBytes = (size_t)e.held * 4;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)e.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  ce = cudaLaunchKernelEx(&cfg, qda_paged_evict_select_kernel, p);
  if (ce != cudaSuccess) return qda_cuda_fail(ce);
  cfg.gridDim = dim3((unsigned)e.move_x, (unsigned)(B * Hkv));
  cfg.blockDim = dim3(kEvMoveThreads);
  cfg.dynamicSmemBytes = 0;
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  ce = cudaLaunchKernelEx(&cfg, qda_paged_evict_move_kernel, p);
  return ce == cudaSuccess ? QDA_OK : qda_cuda_fail(ce);
}
