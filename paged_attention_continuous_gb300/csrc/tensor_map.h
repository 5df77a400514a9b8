// TMA tensor maps of the paged K/V caches, shared by the decode and prefill
// kernels.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "../../include/cb.h"

namespace cb {

// The 2-D view of a cache as rows; rows past the end read as zeros.
enum class CacheMap {
  kBf16,    // [num_blocks][Hkv][16][head_dim]; box 16 rows x 64 dims, 128-byte swizzle
  kCodes8,  // the same of bytes; box 16 rows x head_dim, swizzled over the row (128 or 64 bytes)
  kCodes4,  // [num_blocks][Hkv][17][head_dim / 2] bytes; box 17 rows x head_dim / 2, over the row (64 or 32)
};

// head_dim is 64 or 128.  Maps depend only on the arguments, so the last few
// are kept and reused.
cb_status cached_cache_map(CUtensorMap* m, const void* base, int64_t rows, int head_dim,
                           CacheMap kind = CacheMap::kBf16);

}  // namespace cb
