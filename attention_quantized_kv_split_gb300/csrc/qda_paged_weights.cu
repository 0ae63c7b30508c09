// Accumulated attention weight over the paged cache: host side.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstring>

#include "qda_paged_check.h"
#include "qda_paged_weights.h"

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
  if ((dtype != QDA_BF16 && dtype != QDA_FP16) || !std::isfinite(decay)) return QDA_ERR_INVALID;
  int st = check_codec(D, GS, bits);
  if (st == QDA_OK) st = check_pool(num_pages, page);
  if (st != QDA_OK) return st;
  const int nrep = H / Hkv;
  if (B > QDA_MAX_B || nrep > QDA_MAX_NREP) return QDA_ERR_UNSUPPORTED;
  if ((long long)num_pages * page * Hkv >= 0xffffffffLL) return QDA_ERR_UNSUPPORTED;
  if ((long long)total_q * nrep > 0x7fffff00LL) return QDA_ERR_UNSUPPORTED;
  const void* ptrs[4] = {q, k_packed, k_scales, k_biases};
  for (const void* p : ptrs)
    if (off16(p)) return QDA_ERR_ALIGN;
  const void* words[7] = {lse, mass, token, q_start, kv_len, block_table, shift};
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
  // the instance, and its resident CTAs per SM (0: not asked yet)
  const long long count = window > 0 ? std::min(window, max_q) : max_q;
  const int rows = (int)std::min(count * nrep, 1LL << 20);
  int dev = 0;
  const cudaError_t de = cudaGetDevice(&dev);
  if (de != cudaSuccess || dev < 0 || dev >= 64) return qda_cuda_fail(de == cudaSuccess ? cudaErrorInvalidDevice : de);
  const int di = D == 64 ? 0 : D == 128 ? 1 : D == 256 ? 2 : 3, gi = GS == 32 ? 0 : GS == 64 ? 1 : 2;
  static std::atomic<int> cache[64][2][4][3][2] = {};
  std::atomic<int>& slot = cache[dev][bits == 8][di][gi][rows > 8];
  const auto launch = bits == 4 ? qda_paged_weights_b4 : qda_paged_weights_b8;
  int occ = slot.load();
  if (occ == 0) {
    const cudaError_t e = launch(nullptr, D, GS, rows, &occ, nullptr);
    if (e != cudaSuccess) return qda_cuda_fail(e);
    occ = std::max(occ, 1);
    slot.store(occ);
  }
  p.ctas = sms * occ;
  const cudaError_t e = launch(&p, D, GS, rows, nullptr, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? QDA_OK : qda_cuda_fail(e);
}
