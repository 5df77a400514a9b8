// Host checks of a rotary plan, shared by cb_rope and cb_kv_append_q8.
#pragma once

#include "../../include/cb.h"

namespace cb {
// The plan's fields are in range; head_dim is its head_dim when given (> 0).
cb_status check_rope_plan(const cb_rope_plan* plan, int head_dim, const char* what);
}  // namespace cb
