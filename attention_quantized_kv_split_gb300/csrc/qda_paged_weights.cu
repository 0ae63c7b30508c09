// Accumulated attention weight over the paged cache (sm_103a): the layout of query rows for the kernel for many, host side.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "qda_paged_check.h"
#include "qda_paged_weights_tc.cuh"

namespace qda {

constexpr int kPlThreads = 512;

// A CTA lays out a part of a chunk of counted query rows of a sequence under a KV head in the swizzled form that the products
// read, and its scalars: the rows in fp16 times a power of two that brings the largest value of all of them to [2^14, 2^15),
// or of each of them where they differ too much; rows behind the sequence's last are zeros that weigh nothing. Bound by the
// latency of its loads and exchanges: 18 us for 3500 tokens of 16 heads at D 256 (28.8 MB read, kept in L2 for the products), 6 us
// for 64 tokens of 32 heads at D 128.
template <int D>
__global__ void __launch_bounds__(kPlThreads, 3) qda_paged_weights_lay_kernel(const __grid_constant__ QdaWeightsParams p) {
  using G = PvGeom<D>;
  __shared__ int s_chunk[QDA_MAX_B + 1];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_launch_dependents();
  if (warp == 0) {   // chunks before each sequence
    int c0 = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int c = b < p.B ? pv_chunks(p, pw_seq(p, b)) : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int z = __shfl_up_sync(0xffffffffu, c, o);
        if (lane >= o) c = pv_add(c, z);
      }
      if (b < p.B) s_chunk[b + 1] = pv_add(c0, c);
      c0 = pv_add(c0, __shfl_sync(0xffffffffu, c, 31));
    }
    if (lane == 0) s_chunk[0] = 0;
  }
  __syncthreads();
  const int carry = s_chunk[p.B];
  if (carry > p.max_chunks) {
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid == 0) atomicOr(p.err, QDA_ERR_BIT_PAGED);
    return;
  }
  const int kvh = blockIdx.y;
  __shared__ int s_top[2];   // largest and smallest exponent of a row's largest value
  constexpr int LPR = D / 8 < 32 ? D / 8 : 32, RPW = 32 / LPR;   // a row takes D / 8 lanes of 8 values
  constexpr int RPC = kPlThreads / 32 * RPW;                     // rows of the CTA at a time
  constexpr int N = kPvCols / RPC < 1 ? 1 : kPvCols / RPC;       // rows of a thread
  for (long long x = blockIdx.x; x < (long long)carry * kPvParts; x += gridDim.x) {
    const int ci = (int)(x / kPvParts), part = (int)(x % kPvParts);
    const int b = qda_seq_of(s_chunk, p.B, ci);
    const PwSeq s = pw_seq(p, b);
    const int row0 = (s.len - s.count) * p.nrep + (ci - s_chunk[b]) * kPvRows, row_end = s.len * p.nrep;
    char* dst = p.chunks + ((size_t)ci * p.Hkv + kvh) * G::CHUNK;
    PvScalars* scal = reinterpret_cast<PvScalars*>(dst + G::SLICES * G::SLICE);
    if (tid == 0) {
      s_top[0] = -1000;
      s_top[1] = 1000;
    }
    __syncthreads();
    const int piece = lane % LPR;
    uint4 a[N];
    float top[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int in = j * RPC + warp * RPW + lane / LPR, row = row0 + part * kPvCols + in, tok = row / p.nrep;
      const int h = kvh * p.nrep + row - tok * p.nrep;
      a[j] = make_uint4(0, 0, 0, 0);
      if (in < kPvCols && row < row_end)
        a[j] = __ldg(reinterpret_cast<const uint4*>(p.q + (long long)(s.first + tok) * p.q_tstride + (long long)h * p.q_hstride) + piece);
    }
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t u[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
      top[j] = 0.f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = half2_bits_to_float2_rt(u[k], p.f16);
        top[j] = fmaxf(top[j], fmaxf(fabsf(f.x), fabsf(f.y)));
      }
#pragma unroll
      for (int o = LPR / 2; o >= 1; o >>= 1) top[j] = fmaxf(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
      if (piece == 0 && top[j] > 0.f) {   // (zeros take any scale)
        const int e = (int)(__float_as_uint(top[j]) >> 23);
        atomicMax(&s_top[0], e);
        atomicMin(&s_top[1], e);
      }
    }
    __syncthreads();
    // (an infinite value has the exponent 255: its row alone)
    const bool near = s_top[0] < 255 && s_top[0] - s_top[1] <= kPvNear;
    const int shared_up = near ? pv_up(__uint_as_float((uint32_t)max(s_top[0], 0) << 23)) : 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int i = part * kPvCols + j * RPC + warp * RPW + lane / LPR, row = row0 + i, tok = row / p.nrep;
      if (i >= (part + 1) * kPvCols) continue;
      const int h = kvh * p.nrep + row - tok * p.nrep;
      const bool real = row < row_end;
      const int e = near ? shared_up : pv_up(top[j]);
      const float up = pv_pow2(e);
      const uint32_t u[4] = {a[j].x, a[j].y, a[j].z, a[j].w};
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = half2_bits_to_float2_rt(u[k], p.f16);
        w[k] = pc_h2(f.x * up, f.y * up);
      }
      // slices of SD dimensions; in them blocks of 64, rows of 128 bytes, 16-byte pieces swizzled
      const int sl = piece / (G::SD / 8), at = piece % (G::SD / 8);
      *reinterpret_cast<uint4*>(dst + sl * G::SLICE + (at >> 3) * 16384 + i * 128 + (((at & 7) ^ (i & 7)) << 4)) =
          make_uint4(w[0], w[1], w[2], w[3]);
      if (piece == 0) {
        scal->lse[i] = real ? p.lse[(long long)(s.first + tok) * p.H + h] * -1.4426950408889634f : -INFINITY;
        scal->muls[i] = pv_pow2(-e);
        scal->last[i] = real ? s.base + tok : -1;
        if (i == part * kPvCols) scal->mul[part] = near ? p.qscale * pv_pow2(-e) : 0.f;
      }
    }
    __syncthreads();   // s_top is read
  }
}

// Rows (counted new tokens times query heads of a KV head) up to which the kernel on matrix instructions takes a call, in the
// instance for 8, 16 or 32 of them. Against the kernel for many (a max_q that is not the true one chooses either), 4 sequences of
// 8192 keys, 8 KV heads, 32 query heads, D 128, 4-bit, one call after the other: 8 rows 15 / 43 us, 16 rows 18 / 43, 32 rows 25 / 43,
// 64 rows 68 / 43 (D 256, 8-bit: 32 rows 33 / 63, 64 rows 99 / 64; D 64, 4-bit: 32 rows 24 / 35, 64 rows 59 / 35). D 512 has no
// kernel for many: both operands of a whole key would fill the tensor memory. (256 dimensions of them at a time would fit; it is
// not built.) Its time goes with the rows: 4-bit 64 rows 125 us, 128 rows 239, 256 rows 462.
constexpr int kPwMostRows = 32;

struct WeightsPlan {
  bool tc;
  int rows, chunks;   // rows: in eights
  size_t bytes;
};

static WeightsPlan weights_plan(int B, int nrep, int Hkv, int total_q, int max_q, int window, int D) {
  WeightsPlan w;
  const long long count = window > 0 ? std::min(window, max_q) : max_q;
  const long long rows = count * nrep;
  w.tc = rows > kPwMostRows && D <= 256;
  w.rows = rows <= 8 ? 1 : rows <= 16 || rows > kPwMostRows ? 2 : 4;
  w.chunks = 0;
  w.bytes = 0;
  if (w.tc) {
    long long tokens = total_q;
    if (window > 0) tokens = std::min(tokens, (long long)window * B);
    w.chunks = (int)std::min(tokens * nrep / kPvRows + std::min((long long)B, tokens), 0x7fffffffLL);
    const size_t chunk = D == 64 ? PvGeom<64>::CHUNK : D == 128 ? PvGeom<128>::CHUNK : PvGeom<256>::CHUNK;
    w.bytes = (size_t)w.chunks * Hkv * chunk;
  }
  return w;
}

}  // namespace qda

cudaError_t qda_paged_weights_lay(const QdaWeightsParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)std::min((long long)p.max_chunks * qda::kPvParts, 1LL << 20), (unsigned)p.Hkv);
  switch (p.D) {
    case 64: qda::qda_paged_weights_lay_kernel<64><<<grid, qda::kPlThreads, 0, s>>>(p); break;
    case 128: qda::qda_paged_weights_lay_kernel<128><<<grid, qda::kPlThreads, 0, s>>>(p); break;
    default: qda::qda_paged_weights_lay_kernel<256><<<grid, qda::kPlThreads, 0, s>>>(p); break;
  }
  return cudaGetLastError();
}

extern "C" int qdecode_paged_weights_workspace_bytes(int B, int H, int Hkv, int total_q, int max_q, int window, int D,
                                                     size_t* bytes) {
  using namespace qda;
  if (bytes == nullptr || B < 1 || H < 1 || Hkv < 1 || total_q < 0 || max_q < 1 || window < 0 || H % Hkv != 0) return QDA_ERR_INVALID;
  if (D != 64 && D != 128 && D != 256 && D != 512) return QDA_ERR_UNSUPPORTED;
  if (B > QDA_MAX_B || H / Hkv > QDA_MAX_NREP || (long long)total_q * (H / Hkv) > 0x7fffff00LL) return QDA_ERR_UNSUPPORTED;
  *bytes = weights_plan(B, H / Hkv, Hkv, total_q, max_q, window, D).bytes;
  return QDA_OK;
}

extern "C" int qdecode_paged_weights(const void* q, long long q_tstride, long long q_hstride, const uint32_t* k_packed,
                                     const void* k_scales, const void* k_biases, const float* lse, float* mass,
                                     int32_t* token, const int32_t* q_start, const int32_t* kv_len,
                                     const int32_t* block_table, const int32_t* shift, int total_q, int max_q, int window,
                                     int B, int H, int Hkv, int num_pages, int page, int max_pages, int D, int GS, int bits,
                                     int dtype, double decay, void* stream) {
  using namespace qda;
  if (!k_packed || !k_scales || !k_biases || !mass || !token || !q_start || !kv_len || !block_table) return QDA_ERR_INVALID;
  if (total_q < 0 || max_q < 1 || window < 0 || B < 1 || H < 1 || Hkv < 1 || max_pages < 1 || H % Hkv != 0) return QDA_ERR_INVALID;
  if (total_q > 0 && (!q || !lse)) return QDA_ERR_INVALID;
  if ((dtype != QDA_BF16 && dtype != QDA_FP16) || !std::isfinite((float)decay)) return QDA_ERR_INVALID;
  int st = check_codec(D, GS, bits);
  if (st == QDA_OK) st = check_pool(num_pages, page);
  if (st != QDA_OK) return st;
  const int nrep = H / Hkv;
  if (B > QDA_MAX_B || nrep > QDA_MAX_NREP || Hkv > 65535) return QDA_ERR_UNSUPPORTED;
  if ((long long)num_pages * page * Hkv >= 0xffffffffLL) return QDA_ERR_UNSUPPORTED;
  if ((long long)total_q * nrep > 0x7fffff00LL) return QDA_ERR_UNSUPPORTED;
  const void* ptrs[5] = {q, k_packed, k_scales, k_biases, mass};
  for (const void* p : ptrs)
    if (off16(p)) return QDA_ERR_ALIGN;
  const void* words[6] = {lse, token, q_start, kv_len, block_table, shift};
  for (const void* p : words)
    if (off4(p)) return QDA_ERR_ALIGN;
  if (q_tstride % 8 || q_hstride % 8) return QDA_ERR_ALIGN;
  if (total_q == 0) return QDA_OK;
  QdaWeightsParams p;
  std::memset(&p, 0, sizeof(p));
  int sms;
  st = qda_device(&sms, &p.err);
  if (st != QDA_OK) return st;
  p.q = static_cast<const uint16_t*>(q);
  p.kp = k_packed;
  p.ks = static_cast<const uint16_t*>(k_scales);
  p.kb = static_cast<const uint16_t*>(k_biases);
  p.lse = lse;
  p.mass = mass;
  p.token = token;
  p.q_start = q_start;
  p.kv_len = kv_len;
  p.table = block_table;
  p.shift = shift;
  p.q_tstride = q_tstride;
  p.q_hstride = q_hstride;
  p.total_q = total_q;
  p.window = window;
  p.B = B;
  p.H = H;
  p.Hkv = Hkv;
  p.nrep = nrep;
  p.num_pages = num_pages;
  p.page_shift = page_shift_of(page);
  p.max_pages = max_pages;
  p.f16 = dtype == QDA_FP16;
  p.qscale = 1.4426950408889634f / sqrtf((float)D);
  p.decay = (float)decay;
  p.D = D;
  p.gs_shift = GS == 32 ? 5 : GS == 64 ? 6 : 7;
  p.NG = D / GS;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  const WeightsPlan plan = weights_plan(B, nrep, Hkv, total_q, max_q, window, D);
  const int rows = plan.rows;
  int dev = 0;
  const cudaError_t de = cudaGetDevice(&dev);
  if (de != cudaSuccess || dev < 0 || dev >= 64) return qda_cuda_fail(de == cudaSuccess ? cudaErrorInvalidDevice : de);
  if (plan.tc) {
    const auto run = bits == 4 ? qda_paged_weights_tc_b4 : qda_paged_weights_tc_b8;
    static std::atomic<bool> ready[64][2][3] = {};
    std::atomic<bool>& r = ready[dev][bits == 8][D / 128];
    if (!r.load()) {
      const cudaError_t e = run(nullptr, D, true, nullptr);
      if (e != cudaSuccess) return qda_cuda_fail(e);
      r.store(true);
    }
    void* ws = nullptr;
    st = qda_workspace(plan.bytes, &ws);
    if (st != QDA_OK) return st;
    p.chunks = static_cast<char*>(ws);
    p.max_chunks = plan.chunks;
    p.ctas = sms;
#ifdef QDA_BOUNDS_CHECK
    p.stall = qda_stall_chunk();
#endif
    cudaError_t e = qda_paged_weights_lay(p, s);
    if (e == cudaSuccess) e = run(&p, D, false, s);
    return e == cudaSuccess ? QDA_OK : qda_cuda_fail(e);
  }
  const int di = D == 64 ? 0 : D == 128 ? 1 : D == 256 ? 2 : 3, gi = GS == 32 ? 0 : GS == 64 ? 1 : 2;
  static std::atomic<int> cache[64][2][2][4][3][3] = {};
  std::atomic<int>& slot = cache[dev][bits == 8][p.f16][di][gi][rows / 2];
  const auto launch = bits == 4 ? (p.f16 ? qda_paged_weights_b4_f1 : qda_paged_weights_b4_f0)
                                : (p.f16 ? qda_paged_weights_b8_f1 : qda_paged_weights_b8_f0);
  int occ = slot.load();
  if (occ == 0) {
    const cudaError_t e = launch(nullptr, D, GS, rows, &occ, nullptr);
    if (e != cudaSuccess) return qda_cuda_fail(e);
    occ = std::max(occ, 1);
    slot.store(occ);
  }
  p.ctas = sms * occ;
  const cudaError_t e = launch(&p, D, GS, rows, nullptr, s);
  return e == cudaSuccess ? QDA_OK : qda_cuda_fail(e);
}
