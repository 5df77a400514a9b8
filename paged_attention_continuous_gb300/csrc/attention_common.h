// Workspace layout and argument checks shared by cb_paged_attention,
// cb_paged_attention_q8 and cb_paged_attention_q4.
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/cb.h"
#include "decode_launch.h"
#include "prefill_dispatch.h"

namespace cb {

constexpr size_t kAlign = 256;
inline size_t align_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }

struct WsLayout {
  size_t header = 0, counters = 0, prefill = 0, part_ml = 0, part_acc = 0, total = 0;
  int64_t slots = 0;  // decode partial slots
};

// Workspace regions.  The header, the decode split tickets and the prefill
// region hold state that must read zero at the start of every call (each
// call leaves them zero), so they sit at FIXED offsets that do not depend on
// the call's sizes.  The split partials are scratch rewritten by every call,
// sized by the call's decode rows.
//   header words: [0] device error bits, [1] decode item counter
//   counters: done[kPlanMax * kMaxKvHeads] (one ticket counter per
//             (decode row, KV head) of a launch)
constexpr int64_t kMaxKvHeads = 64;
constexpr int kPlanMax = decode::kPlanMax;
constexpr size_t kCounterWords = (size_t)kPlanMax * kMaxKvHeads;

inline WsLayout ws_layout(int64_t num_reqs, int64_t Hq, int64_t Hkv, int64_t D) {
  WsLayout w;
  const int64_t rows = num_reqs < kPlanMax ? num_reqs : kPlanMax;
  w.header = 0;
  w.counters = kAlign;
  w.prefill = w.counters + align_up(kCounterWords * 4);
  w.part_ml = w.prefill + align_up(prefill_workspace_bytes(Hq, Hkv, D));
  const size_t slots = (size_t)decode::partial_slots(rows, Hkv);
  w.part_acc = w.part_ml + align_up(slots * Hq * 2 * 4);
  w.total = w.part_acc + align_up(slots * Hq * D * 4);
  w.slots = (int64_t)slots;
  return w;
}

inline decode::Scratch decode_scratch(const cb_attention_args& a, const WsLayout& L) {
  uint8_t* ws = static_cast<uint8_t*>(a.workspace);
  decode::Scratch s{};
  s.work_counter = reinterpret_cast<uint32_t*>(ws + L.header) + 1;
  s.done = reinterpret_cast<uint32_t*>(ws + L.counters);
  s.part_ml = reinterpret_cast<float*>(ws + L.part_ml);
  s.part_acc = reinterpret_cast<float*>(ws + L.part_acc);
  s.slots = L.slots;
  return s;
}

// Checks of an attention call's arguments, before anything is launched.
cb_status check_attention(const cb_attention_args& a);

}  // namespace cb
