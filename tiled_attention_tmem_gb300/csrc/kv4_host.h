// Host-side helpers of the serving operators (not part of the ABI).
#pragma once
#include "fa_paged.h"
#include "host.h"

namespace fa {

// log2 of a page size the kernels take, -1 for any other.
inline int page_log2_of(int page) {
  return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1;
}

// Shape, gains, pointers and alignment of a cache (paged.cu).
fa_status kv4_cache_checks(const fa_kv4_cache* c);

}  // namespace fa
