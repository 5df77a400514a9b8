// TMA tensor maps of the paged K/V caches, shared by the decode and prefill
// kernels.
#pragma once

#include <cuda.h>

#include <cstdint>

#include "../../include/cb.h"

namespace cb {

// The 2-D view [rows][head_dim] of a cache laid out as
// [num_blocks][Hkv][16][head_dim] (rows = num_blocks * Hkv * 16); rows past
// the end read as zeros.  elem_bytes 2 (bf16): box 16 rows x 64 dims with the
// 128-byte swizzle; 1 (8-bit codes): box 16 rows x head_dim, swizzled over
// the row (128 or 64 bytes).  head_dim is 64 or 128.  Maps depend only on
// the arguments, so the last few are kept and reused.
cb_status cached_cache_map(CUtensorMap* m, const void* base, int64_t rows, int head_dim,
                           int elem_bytes = 2);

}  // namespace cb
