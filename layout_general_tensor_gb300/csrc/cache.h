// The paged 8-bit cache (include/attn_cache.h), shared by its kernels.
#pragma once
#include "attn_cache.h"

namespace lgt {

// The geometry and the pointers' presence (not their alignment).
bool cache_ok(const attn_cache_t& c);

}  // namespace lgt
