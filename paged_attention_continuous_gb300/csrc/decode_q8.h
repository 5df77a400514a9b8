// Launch of the split-KV decode kernel over the 8-bit cache.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "../../include/cb.h"
#include "decode_launch.h"

namespace cb {
namespace decode_q8 {

// Runs the decode rows [0, a.num_decodes) of `a`, in launches of at most
// decode::kPlanMax rows.  Returns CB_ERR_UNSUPPORTED (without a message) for
// head counts that need more than 64 items for each (row, split).
cb_status dispatch(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                   int64_t scale_stride, const decode::Scratch& s, uint32_t* error_word,
                   cudaStream_t stream, decode::After after);

}  // namespace decode_q8
}  // namespace cb
