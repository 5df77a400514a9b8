// Blocks of a row's tokens, and whether its block table holds them: shared by
// the attention kernels and the host's checks.  Lengths come from device
// memory and may be anything, so nothing here adds to one before it is
// checked: (len + block - 1) / block passes 2^31 for the last lengths below
// it, turns negative and then fits every table.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define CB_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define CB_HOST_DEVICE inline
#endif

namespace cb {

// Blocks of `block` tokens that hold `len` tokens; 0 for len <= 0.
CB_HOST_DEVICE constexpr int32_t blocks_of(int32_t len, int32_t block) {
  return len > 0 ? (int32_t)(((uint32_t)len + (uint32_t)block - 1u) / (uint32_t)block) : 0;
}

// A row of at least one token whose table of max_blocks entries holds it.
CB_HOST_DEVICE constexpr bool row_length_fits(int32_t len, int32_t block, int32_t max_blocks) {
  return len >= 1 && blocks_of(len, block) <= max_blocks;
}

// Query tokens [q0, q0 + q_len) lie within [0, num_tokens).
CB_HOST_DEVICE constexpr bool row_tokens_fit(int32_t q0, int32_t q_len, int32_t num_tokens) {
  return q0 >= 0 && q_len >= 0 && q_len <= num_tokens - q0;
}

}  // namespace cb
