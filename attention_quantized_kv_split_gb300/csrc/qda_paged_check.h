// Host-side checks that the paged calls share.
#pragma once

#include <cstdint>

#include "qda_paged.h"

namespace qda {

inline bool good_page(int page) { return page >= QDA_PAGE_MIN && page <= QDA_PAGE_MAX && (page & (page - 1)) == 0; }

inline int page_shift_of(int page) {
  int s = 0;
  while ((1 << s) < page) ++s;
  return s;
}

// bits, GS and D of every paged call: the quantizer's
inline int check_codec(int D, int GS, int bits) {
  if (D < 1 || GS < 1) return QDA_ERR_INVALID;
  if (bits != 4 && bits != 8) return QDA_ERR_UNSUPPORTED;
  if (GS != 32 && GS != 64 && GS != 128) return QDA_ERR_UNSUPPORTED;
  if (D != 64 && D != 128 && D != 256 && D != 512) return QDA_ERR_UNSUPPORTED;
  if (D % GS != 0) return QDA_ERR_UNSUPPORTED;
  return QDA_OK;
}

inline int check_pool(int num_pages, int page) {
  if (num_pages < 1 || page < 1) return QDA_ERR_INVALID;
  if (!good_page(page) || (long long)num_pages * page > 0x7fffffffLL) return QDA_ERR_UNSUPPORTED;
  return QDA_OK;
}

inline bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
inline bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace qda
