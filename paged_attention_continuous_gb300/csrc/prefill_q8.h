// Launch of the prefill-chunk kernel over the 8-bit cache.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/cb.h"

namespace cb {
namespace prefill_q8 {

// CTAs of the prefill rows of `a` (an upper bound; 0 without prefill rows or
// where this kernel does not take them).
int64_t ctas(const cb_attention_args& a);

// Splits of each CTA's keys, 1 for none: as many as idle SMs take when the
// CTAs fill less than half of them.  slots: places for parts, of which a call
// with splits uses splits for each of its tokens.
int splits(const cb_attention_args& a, int64_t slots);

// Where the splits leave their parts: ml [slots][Hq][2], acc [slots][Hq][D].
struct Parts {
  int32_t splits;
  float* ml;
  float* acc;
};

// Rows [num_decodes, num_reqs) of `a`.  Returns CB_ERR_UNSUPPORTED (without a
// message) for more than 128 query heads to a KV head.  The grid allows a
// kernel launched behind it with programmatic stream serialization to start
// when its last CTAs have started.
cb_status launch(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                 int64_t scale_stride, const Parts& parts, uint32_t* error_word, cudaStream_t stream);

// Joins the parts of a launch with splits, once it has completed.
cb_status join(const cb_attention_args& a, const Parts& parts, cudaStream_t stream);

}  // namespace prefill_q8
}  // namespace cb
