// Split-KV decode attention over the 4-bit cache (one query token per row).
//
// The definition is the decode kernel's ("Chunked Prefill", How chunked
// prefill works: the query at position seq_len - 1 attends every cached key
// of its request) with keys and values (n - 8) s, one scale s for each group
// of 32 dims of a token.  The cache is read once, 17 / 32 of the 8-bit one's
// bytes, so that at HBM's rate nearly twice as many elements a second pass
// through each SM, and what a warp does for a page decides.  That asks for
// another shape than the 8-bit kernel's:
//
//   * Work items, plan, dealing and the merge of splits are the decode kernels'
//     (split_plan.cuh, decode_merge.cuh): runs of pages of one (row, KV head),
//     drawn by independent warps, each with a ring of two stages of four pages.
//     But mostly twelve warps of 168 registers,
//     three to a scheduler, where the 8-bit kernel has eight of 255: expanding
//     codes is arithmetic, and eight warps waited for its results in half of
//     the cycles (128 requests of up to 32k tokens, 32 + 8 heads of 128: 467 us
//     with twelve, 489 with eight; sixteen and steps of two pages took 7% longer
//     than twelve).  So what a warp
//     needs once an item (the plan, the item drawn next) lies in shared memory,
//     a window of pages' places in the cache in its lanes, and what happens
//     between steps is looked at only when some of it is due.
//   * Pages are copied by 16-byte asynchronous copies of all lanes, 17 of them
//     for four pages of K and V: a page is 1088 bytes, and issuing a TMA box for
//     each took a warp a quarter of its step (when these copies took its place the
//     long decodes below went from 563 us to 489).
//     They need no barrier: a lane waits for its own group, and nothing can
//     keep it from landing.
//   * Codes become halves, with their scales, by one logic operation and one
//     fused multiply-add for two (q4.cuh), exactly; both products of a page
//     run as m16n8k16 matrix instructions with float32 accumulation.  K codes
//     are loaded as 16-byte vectors: the contraction over the dims has no
//     order, so lane qd of a row takes its quarter qd, a group (or half of
//     one), and Q^T is loaded in the same order.  V codes come through
//     transposing loads of 16 bits, four codes (every other of eight dims) of two
//     tokens to a lane; two lanes exchange their even and odd dims when a row is
//     written.
//   * Queries are scaled by a power of two to the halves' range for each
//     head, so that bfloat16 queries are halves exactly (elements under
//     2^-29 of the head's largest lose bits); float32 queries are split into
//     two halves (22 bits), and their weights too (and to 2^-24, the least
//     half, where the largest is 2^-0.5 at least).  With those, score
//     exponents are rounded at their size next to the reference: scale *
//     log2(e) is a pair of floats, the reference a whole number.
//   * Weights are 2^(x - m), x the score times log2(e), m a reference that
//     moves when passed by more than a lag: 2^7 at the reference, 2^15 at
//     most, rounded to multiples of 2^-24 at least.  Lanes first ask whether
//     any of their scores passes it, and look for the largest only then.
//   * A masked token's weights are 0 by its score and its values 0 by its
//     scale, which is replaced: what lies there may be anything.
//
// What bounds it: the warps' instructions (305 for a page of K and V and a
// KV head's 8 query heads, of which K's expansion and product are 85 and V's
// 120; 55 to 60% of the issue slots), not far from memory: 128 requests of up
// to 32k tokens (64 + 8 heads of 128) 420 us, 5.1 TB/s, 75% of the measured copy
// rate (without the arithmetic 365: pages of 1 KB lie scattered).  64 requests of up
// to 4k tokens (32 + 8 heads) 49 us: 9 until the first pages have landed,
// everybody's at once, the rest the one wave of items and their merges; 8 of up to
// 512 tokens 12 us, of latency.  The 8-bit cache takes 636, 63 and 12 us for the
// same.  (These and the figures below: passes over three states in turn, in a
// replayed graph; requests have 32 + 8 heads of 128 dims where nothing is said.)
#pragma once

#include <cstdint>
#include <type_traits>

#include "decode_launch.h"
#include "decode_merge.cuh"
#include "device_utils.cuh"
#include "mma_utils.cuh"
#include "q4.cuh"
#include "q8.cuh"
#include "split_plan.cuh"

namespace cb {
namespace decode_q4 {

using namespace decode;

// How rows are cut: the 8-bit kernel's rules, but where the pages do not go in
// one wave, one item to a warp (and its share of the last phase) up to kFewPages
// pages of it (measured without such waves: 64 requests of up to 4k tokens, 37
// pages to a warp, 52 us, 57 with two; up to 8k 84 and 90; with them 128 of up to 8k,
// 148 pages: 150 and 142; of up to 32k 518 and 468).
constexpr int kFewPages = 96;
constexpr int kItemsEven = 2;
// One wave of items, where a warp's share of the pages is small (beside a prefill
// grid, whose SMs come free one by one, smaller still): 64 requests of up to 4k
// tokens 49.4 us, 52.1 in two phases; 16 of those 23.7 and 30; 8 of up to 8k 24 and
// 34; 64 of up to 8k 77 and 84; 2 of 8k beside 512 prompt tokens 31 and 51; 96 of up
// to 8k beside 512 behind 4k 154, 192 in one wave.
constexpr int kSinglePages = 128, kSingleBeside = 32;
constexpr int kSingleLeast = 4;
constexpr int kMaxSplits = 64;
// weight exponent at the reference, which moves when passed by more than the
// lag (float32: exponents near 0 are the most exact)
template <typename T> constexpr float kTop = 7.f;
template <> constexpr float kTop<float> = 0.f;
template <typename T> constexpr float kLag = 8.f;
template <> constexpr float kLag<float> = 2.f;

struct Params {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const void* q;
  void* out;
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens;
  const int32_t* block_tables;
  int32_t row_begin, num_rows, num_tokens;
  int32_t num_blocks, max_blocks_per_seq;
  int32_t num_q_heads, num_kv_heads;
  int32_t group;           // query heads of a KV head
  int32_t parts;           // items that serve a KV head
  int32_t part_heads;      // query heads of an item (the last part may have fewer)
  float scale_log2;
  float scale_log2_low;    // what float32 leaves of it, as a share of it
  int32_t window;
  uint32_t* error_word;
  uint32_t* work_counter;  // zero between launches
  uint32_t* done;          // [num_rows * Hkv * parts] split tickets; zero between launches
  int32_t max_slots;
  float* part_ml;          // [slots][Hq][2]
  float* part_acc;         // [slots][Hq][D]
  int32_t pdl_mode;
};

struct alignas(16) ItemDesc {
  int32_t r, u, nsplit, slot;          // row, unit (part of a KV head), splits of the row, partial slot
  int32_t page0, page1, seq_len, token;
  int32_t h0, heads, g, pad;           // first query head, query heads, KV head
};

// Shared memory: every warp's page ring first, then each warp's small state,
// then the plan.
template <int D, int kStages, int kPages, int kWarps>
struct Layout {
  static constexpr int kSlot = q4::page_bytes(D);              // of a page
  static constexpr int kStageBytes = 2 * kPages * kSlot;       // K pages | V pages
  static constexpr int kRingBytes = kStages * kStageBytes;     // of a warp
  // items that the ring can hold pages of at once, and the one dealt ahead
  static constexpr int kItems = kStages + 2;
  struct State {
    ItemDesc items[kItems];
    ItemDesc pend[2];            // the items of the last two partials
  };
  // what dealing wants of the plan
  struct Deal {
    int32_t spa, spb, num_a;
    uint32_t n_static, items_dyn, workers;
  };
  static constexpr int kStateBytes = ((int)sizeof(State) + 15) / 16 * 16;
  static constexpr size_t total = (size_t)kWarps * (kRingBytes + kStateBytes) + kPlanSmemBytes;
};

// Byte offset of 16-byte chunk c of row t of a page in its slot: rows of 64
// bytes have their chunks XOR row / 2 mod 4, of 32 bytes XOR row / 4 mod 2, so
// that neither the loads of K nor the transposing ones of V meet in a bank.
// (Row 16, the scales, lies as it is.)
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int t, int c) {
  if constexpr (D == 128) return (uint32_t)(t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
  return (uint32_t)(t * 32 + ((c ^ ((t >> 2) & 1)) << 4));
}
// Quarter qd of the codes of row t: 32 dims, or 16.
template <int D>
__device__ __forceinline__ void load_words(uint32_t page, int t, int qd, uint32_t (&w)[D / 32]) {
  if constexpr (D == 128) lds128(page + chunk_off<D>(t, qd), w);
  else lds64(page + chunk_off<D>(t, qd >> 1) + (qd & 1) * 8, w);
}
// kNT: eights of query heads of an item; kStages stages of kPages pages each.
template <typename T, int D, int kNT, int kWarps, int kStages, int kPages>
__global__ void __launch_bounds__(kWarps * 32, 1) decode_kernel(const __grid_constant__ Params p) {
  // pieces of a query element and of a weight: one half, or two for float32
  constexpr int kP = std::is_same<T, float>::value ? 2 : 1;
  constexpr int kJ = D / 64;        // 16-element parts of a lane's query dims
  constexpr int kMT = D / 16;       // 16-dim tiles of the output
  constexpr int kGroups = D / q4::kGroup;
  using Lay = Layout<D, kStages, kPages, kWarps>;
  using State = typename Lay::State;
  constexpr int kSlot = Lay::kSlot;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ typename Lay::Deal deal;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int Hkv = p.num_kv_heads, Hq = p.num_q_heads;
  const int units = Hkv * p.parts;
  const int win = p.window;
  uint8_t* ring = smem + warp * Lay::kRingBytes;
  State& ws = *reinterpret_cast<State*>(smem + kWarps * Lay::kRingBytes + warp * Lay::kStateBytes);
  int32_t* plan_a = reinterpret_cast<int32_t*>(smem + kWarps * (Lay::kRingBytes + Lay::kStateBytes));
  int32_t* plan_b = plan_a + (kPlanMax + 1);
  int32_t* row_len = plan_b + (kPlanMax + 1);
  int32_t* row_tok = row_len + kPlanMax;
  {
    const SplitPlan plan = plan_splits<kWarps>(
        PlanRows{p.seq_lens, p.cu_seqlens_q, p.row_begin, p.num_rows, p.num_tokens, p.max_blocks_per_seq, units, win,
                 p.max_slots, kItemsEven, p.error_word, kPages, kPages, kMaxSplits,
                 p.pdl_mode == 2 ? kSingleBeside : kSinglePages, kSingleLeast, kFewPages, true},
        kWarps, plan_a, plan_b, row_len, row_tok);
    if (threadIdx.x == 0) {
      const int num_a = plan_a[p.num_rows], num_b = plan_b[p.num_rows];
      const uint32_t workers = gridDim.x * kWarps;
      deal.spa = plan.spa;
      deal.spb = plan.spb;
      deal.num_a = num_a;
      deal.workers = workers;
      deal.n_static = plan.ok && p.pdl_mode != 2 ? (uint32_t)min((int64_t)num_a * units, (int64_t)workers) : 0u;
      deal.items_dyn = plan.ok ? (uint32_t)((num_a + num_b) * units) - deal.n_static : 0u;
    }
  }
  __syncthreads();

  // ---- dealing: the first item is dealt statically (item w of W warps),
  // later ones are drawn from the counter.  Two steps before the producer
  // reaches the end of its item it draws the next one, and one step before,
  // it describes that item and requests its first block ids: early enough that
  // neither is waited for, and no earlier, since an item drawn is one that no
  // idle warp can take.  Beside a prefill grid every item is drawn.
  enum { kNone, kDrawn, kKnown, kEnd };  // the item after the producer's
  int nx = kNone;
  uint32_t draw = 0;           // lane 0: the counter's value
  int nx_page = -1;            // of the item described ahead: as `win`
  bool first_static = true;
  int prod_items = 0;
  // the producer's next page and its item's end; lane i: which of the cache's
  // pages is page win_base (+ 32) + i (-1: unreadable)
  int prod_page = 0, prod_end = 0, win_base = 0, places_now = -1, places_next = -1;
  int ahead = 0;               // stages issued and not consumed

  const volatile typename Lay::Deal& dl = deal;
  // where pages pg .. of an item lie: lane i page pg + i
  auto places = [&](const ItemDesc& d, int pg) -> int {
    int y = -1;
    if (pg + lane < d.page1) {
      const int b = __ldg(p.block_tables + (int64_t)(p.row_begin + d.r) * p.max_blocks_per_seq + pg + lane);
      if (b >= 0 && b < p.num_blocks) y = b * Hkv + d.g;
      else set_error(p.error_word, CB_DEVERR_BLOCK_RANGE);
    }
    return y;
  };
  auto draw_next = [&]() {
    nx = kDrawn;
    const bool is_first = first_static && warp * gridDim.x + blockIdx.x < dl.n_static;
    if (!is_first && dl.items_dyn > 0) lane0_fetch_add1(p.work_counter, draw, lane);
  };
  auto find_row = [&](const int32_t* pre, int x) -> int {  // the last row with pre[row] <= x
    const int step = (p.num_rows + 31) >> 5;
    const int i1 = lane * step;
    const bool le1 = i1 < p.num_rows && pre[i1] <= x;
    const int base = (__popc(__ballot_sync(0xffffffffu, le1)) - 1) * step;
    const int i2 = base + lane;
    const bool le2 = lane < step && i2 < p.num_rows && pre[i2] <= x;
    return base + __popc(__ballot_sync(0xffffffffu, le2)) - 1;
  };
  auto fetch_ahead = [&]() {
    nx = kEnd;
    // warp w of every CTA before warp w + 1 of any: when there are fewer large
    // items than warps, every SM gets its share of them
    const uint32_t worker = warp * gridDim.x + blockIdx.x, n_static = dl.n_static, dyn = dl.items_dyn;
    uint32_t idx = worker;
    const bool is_first = first_static && worker < n_static;
    first_static = false;
    if (!is_first) {
      if (dyn == 0) return;
      const uint32_t b = __shfl_sync(0xffffffffu, draw, 0);
      // every warp draws once past the end; the last of them resets
      if (b >= dyn) {
        if (b == dyn + dl.workers - 1 && lane == 0) atomicExch(p.work_counter, 0u);
        return;
      }
      idx = n_static + b;
    }
    nx = kKnown;
    const uint32_t x = idx / (uint32_t)units;
    const int u = (int)(idx - x * (uint32_t)units);
    const int num_a = dl.num_a;
    const bool phase_a = (int)x < num_a;
    const int i = phase_a ? find_row(plan_a, (int)x) : find_row(plan_b, (int)x - num_a);
    const int a0 = plan_a[i], na = plan_a[i + 1] - a0, b0 = plan_b[i], nb = plan_b[i + 1] - b0;
    const int split = phase_a ? (int)x - a0 : (int)x - num_a - b0;
    const int L = row_len[i];
    const int fp = first_page(L, win), end = blocks_of(L, kPageTokens), spb = dl.spb;
    const RowSplit rs = row_split(end - fp, dl.spa, spb, kPages);
    ItemDesc& d = ws.items[prod_items % Lay::kItems];
    if (lane == 0) {
      const int g = u / p.parts, part = u - g * p.parts;
      d.r = i;
      d.u = u;
      d.nsplit = na + nb;
      d.slot = a0 + b0 + (phase_a ? split : na + split);
      d.page0 = fp + (phase_a ? split * rs.size : rs.bp + split * spb);
      d.page1 = min(end, d.page0 + (phase_a ? rs.size : spb));
      d.seq_len = L;
      d.token = row_tok[i];
      d.g = g;
      d.h0 = g * p.group + part * p.part_heads;
      d.heads = min(p.part_heads, p.group - part * p.part_heads);
    }
    __syncwarp();
    nx_page = places(d, d.page0);
  };
  auto next_item = [&]() -> bool {
    if (nx == kNone) draw_next();
    if (nx == kDrawn) fetch_ahead();
    if (nx == kEnd) return false;
    nx = kNone;
    const ItemDesc& d = ws.items[prod_items % Lay::kItems];
    ++prod_items;
    prod_page = win_base = d.page0;
    prod_end = d.page1;
    places_now = nx_page;
    return true;
  };
  draw_next();
  fetch_ahead();

  // Refill one stage with the producer's next pages (whole warp), 16 bytes to a
  // lane at a time; a lane's chunks keep their places.  Without more pages the
  // group of copies is empty, so that groups and stages go together.
  constexpr int kChunks = q4::row_bytes(D) / 16;   // of a row
  constexpr int kCodes = q4::kPage * kChunks / 32; // copies of a lane for a page's codes
  const uint32_t code_at = smem_addr(ring) + chunk_off<D>(lane / kChunks, lane % kChunks);
  const uint8_t* const k_lane = p.k_cache + lane * 16;
  const uint8_t* const v_lane = p.v_cache + lane * 16;
  // the scales of all of a stage's pages are one copy more: of page scale_page,
  // K or V
  static_assert(2 * kPages * kChunks <= 32, "one copy of the scales");
  const int scale_page = lane / (2 * kChunks), scale_chunk = lane % kChunks, scale_v = lane / kChunks & 1;
  const uint8_t* const scale_lane = (scale_v ? p.v_cache : p.k_cache) + q4::scales_at(D, 0) + scale_chunk * 16;
  const uint32_t scale_at = smem_addr(ring) + (scale_v * kPages + scale_page) * kSlot + q4::scales_at(D, 0) + scale_chunk * 16;
  // What happens between two steps of an item (the next window of places, the
  // next item) is looked at every `quiet` steps, when some of it is due.
  int quiet = 0;
  auto produce = [&](int st) {
    if (quiet > 0) {
      --quiet;
    } else {
      if (prod_page >= prod_end && !next_item()) {
        asm volatile("cp.async.commit_group;" ::: "memory");
        return;
      }
      if (prod_page - win_base == 16 && win_base + 32 < prod_end)
        places_next = places(ws.items[(prod_items - 1) % Lay::kItems], win_base + 32);
      if (prod_page - win_base >= 32) {
        win_base += 32;
        places_now = places_next;
      }
      if (nx == kNone && prod_end - prod_page <= 3 * kPages) draw_next();
      else if (nx == kDrawn && prod_end - prod_page <= 2 * kPages) fetch_ahead();
      const int window = win_base + (prod_page - win_base < 16 ? 16 : 32);
      const int due = min(window, prod_end - 3 * kPages);
      quiet = max((due - prod_page + kPages - 1) / kPages - 1, 0);
    }
    const uint32_t stage_at = st * Lay::kStageBytes;
    const int off = prod_page - win_base;
    // (the window holds all of the stage's pages; zeros where there is none, or
    // none that can be read)
#pragma unroll
    for (int k = 0; k < kPages; ++k) {
      const int y = __shfl_sync(0xffffffffu, places_now, (off + k) & 31);
      const bool ok = prod_page + k < prod_end && y >= 0;
      const uint32_t at = ok ? (uint32_t)y : 0u, bytes = ok ? 16u : 0u;
      const uint8_t* ks = k_lane + (uint64_t)at * kSlot;
      const uint8_t* vs = v_lane + (uint64_t)at * kSlot;
      const uint32_t kd = code_at + stage_at + k * kSlot, vd = kd + kPages * kSlot;
#pragma unroll
      for (int i = 0; i < kCodes; ++i) {
        // (32 chunks are 8 rows or 16, after which the swizzle repeats)
        cp_async16(kd + i * 512, ks + i * 512, bytes);
        cp_async16(vd + i * 512, vs + i * 512, bytes);
      }
    }
    {
      const int y = __shfl_sync(0xffffffffu, places_now, (off + scale_page) & 31);
      const bool ok = prod_page + scale_page < prod_end && y >= 0;
      if (lane < 2 * kPages * kChunks)
        cp_async16(scale_at + stage_at, scale_lane + (uint64_t)(ok ? (uint32_t)y : 0u) * kSlot, ok ? 16u : 0u);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    prod_page += kPages;
    ++ahead;
  };

  // ---- split tickets: one for each item of a split row; a partial is
  // counted when the warp writes its next one (or finishes), by when its
  // stores are long complete and the release rarely waits.
  auto count = [&](const ItemDesc& d) { return count_split(p.done + (int64_t)d.r * units + d.u, d.nsplit, lane); };
  auto merge = [&](const ItemDesc& d) {
    merge_splits<T, D, 4, 4, true>(p.part_ml, p.part_acc, p.out, Hq, d.h0, d.heads, plan_a[d.r] + plan_b[d.r],
                                   d.nsplit, d.token);
  };
  bool pending = false;     // ws.pend[pend_at]: the item of the partial not counted yet
  int pend_at = 0;

  // the cache and the queries are read from here on: behind this step's append
  // when the launch overlaps it (a prefill grid beside has begun behind it)
  if (p.pdl_mode != 2) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) produce(s);

  // the oldest stage's copies of every lane have landed
  auto wait_full = [&]() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
    __syncwarp();
  };
  // fragment roles: rows grp and grp + 8, columns 2 qd and 2 qd + 1
  const int grp = lane >> 2, qd = lane & 3;
  const int v_tok = (lane & 7) + (lane & 8), v_chunk = lane >> 4;

  uint32_t qb[kP][kNT][kJ * 4][2];   // Q^T fragments
  float hs[kNT][2];                  // score factor of this lane's two heads
  float acc[kNT][kMT][4];
  float m_run[kNT][2], l_run[kNT][2];
  const q4::Exponents exps;
  int item = 0, st = 0;              // items begun, stage of the next step
  while (ahead > 0) {
    const ItemDesc& d = ws.items[item % Lay::kItems];
    // its queries are loaded while its first pages land
    uint4 qx[kNT][kJ][sizeof(T)];      // 16 elements each
    {
      const T* q0 = static_cast<const T*>(p.q) + ((int64_t)d.token * Hq + d.h0) * D + D / 4 * qd;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < (int)sizeof(T); ++i)
            qx[nt][j][i] = reinterpret_cast<const uint4*>(q0 + min(nt * 8 + grp, d.heads - 1) * D + 16 * j)[i];
    }
    wait_full();
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
      const bool live = nt * 8 + grp < d.heads;
      float x[kJ][16];
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        load16(reinterpret_cast<const T*>(qx[nt][j]), x[j]);
#pragma unroll
        for (int e = 0; e < 16; ++e) amax = fmaxf(amax, fabsf(x[j][e]));
      }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      // largest magnitude to [2^14, 2^15); a head of zeros, or one that
      // is not finite (whose scores are not either), keeps factor 1
      const int k = amax > 0.f && amax <= 3.402823466e38f ? max((int)(__float_as_uint(amax) >> 23) - 127, -110) : 14;
      // (the scale's sign goes with the query; the factor is never 0, so that a
      // masked score stays -inf under it)
      const float up = copysignf(q8::exp2i(14 - k), p.scale_log2);
      const float down = fmaxf(fabsf(p.scale_log2) * q8::exp2i(k - 14), 1.17549435e-38f);
      hs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * qd);
      hs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * qd + 4);
#pragma unroll
      for (int j = 0; j < kJ; ++j)
#pragma unroll
        for (int s = 0; s < 4; ++s)
#pragma unroll
          for (int hlf = 0; hlf < 2; ++hlf) {
            const int e = 4 * s + 2 * hlf;
            const float a = live ? x[j][e] * up : 0.f, b = live ? x[j][e + 1] * up : 0.f;
            const __half2 h = __floats2half2_rn(a, b);
            qb[0][nt][j * 4 + s][hlf] = as_u32(h);
            if constexpr (kP == 2) {
              const float2 f = __half22float2(h);
              qb[kP - 1][nt][j * 4 + s][hlf] = as_u32(__floats2half2_rn(a - f.x, b - f.y));
            }
          }
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_run[nt][0] = l_run[nt][1] = 0.f;
    }
    // pages [c_lo, c_hi) are read whole
    const int c_end = d.page1;
    const int c_lo = blocks_of(first_key(d.seq_len, win), kPageTokens);
    const int c_hi = min(c_end, d.seq_len / kPageTokens);
#pragma unroll 1
    for (int c_page = d.page0; c_page < c_end; c_page += kPages) {
      if (c_page != d.page0) wait_full();
      --ahead;
      const bool whole = c_page >= c_lo && c_page + kPages <= c_hi;
      // otherwise keys [lo[k], hi[k]) of page k are read (hi <= 0: none)
      int lo[kPages], hi[kPages];
      if (!whole) {
#pragma unroll
        for (int k = 0; k < kPages; ++k) {
          const int pg = c_page + k;
          hi[k] = pg < c_end ? min(kPageTokens, d.seq_len - pg * kPageTokens) : 0;
          lo[k] = first_key(d.seq_len, win) - pg * kPageTokens;
        }
      }
      const uint8_t* stage = ring + st * Lay::kStageBytes;
      const uint32_t kp = smem_addr(stage);
      const uint32_t vp = kp + kPages * kSlot;

      // ---- S^T = K Q^T: an accumulator chain for each page
      float s[kPages][kNT][4];
      {
        // a lane's quarter of a row is 32 dims (or 16), of one group
        constexpr int kWords = D / 32;
        uint32_t w0[kPages][kWords], w1[kPages][kWords];
        q4::Scale s0[kPages], s1[kPages];
#pragma unroll
        for (int k = 0; k < kPages; ++k) {
          load_words<D>(kp + k * kSlot, grp, qd, w0[k]);
          load_words<D>(kp + k * kSlot, grp + 8, qd, w1[k]);
          const uint8_t* sc = stage + k * kSlot + qd * D / 128;
          s0[k] = q4::scale_twice(sc[q4::scales_at(D, grp)]);
          s1[k] = q4::scale_twice(sc[q4::scales_at(D, grp + 8)]);
        }
#pragma unroll
        for (int e = 0; e < kWords; ++e)
#pragma unroll
          for (int k = 0; k < kPages; ++k) {
            uint32_t h0[4], h1[4];
            q4::halves8(w0[k][e], s0[k], exps, h0);
            q4::halves8(w1[k][e], s1[k], exps, h1);
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              const uint32_t a[4] = {h0[2 * m], h1[2 * m], h0[2 * m + 1], h1[2 * m + 1]};
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt) {
                if (e == 0 && m == 0) mma_f16_first(s[k][nt], a, qb[0][nt][0][0], qb[0][nt][0][1]);
                else mma_f16(s[k][nt], a, qb[0][nt][2 * e + m][0], qb[0][nt][2 * e + m][1]);
                if constexpr (kP == 2)
                  mma_f16(s[k][nt], a, qb[kP - 1][nt][2 * e + m][0], qb[kP - 1][nt][2 * e + m][1]);
              }
            }
          }
      }
      // ---- online softmax (base 2) per head ------------------------------------
      uint32_t pb[kP][kPages][kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        if (!whole) {
#pragma unroll
          for (int k = 0; k < kPages; ++k) {
            if (!(grp < hi[k] && grp >= lo[k])) s[k][nt][0] = s[k][nt][1] = -INFINITY;
            if (!(grp + 8 < hi[k] && grp + 8 >= lo[k])) s[k][nt][2] = s[k][nt][3] = -INFINITY;
          }
        }
        float pm[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          pm[c] = fmaxf(s[0][nt][c], s[0][nt][c + 2]);
#pragma unroll
          for (int k = 1; k < kPages; ++k) pm[c] = fmaxf(pm[c], fmaxf(s[k][nt][c], s[k][nt][c + 2]));
          pm[c] = fmaf(pm[c], hs[nt][c], -kTop<T>);
        }
        // The reference moves only when a step passes it by more than the lag,
        // so the lanes first ask whether any of theirs does (most steps: none)
        // and look for a head's largest then.
        const bool over = pm[0] - m_run[nt][0] > kLag<T> || pm[1] - m_run[nt][1] > kLag<T>;
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) {
            pm[0] = fmaxf(pm[0], __shfl_xor_sync(0xffffffffu, pm[0], o));
            pm[1] = fmaxf(pm[1], __shfl_xor_sync(0xffffffffu, pm[1], o));
          }
          float alpha[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float top = kP == 2 ? rintf(pm[c]) : pm[c];
            const bool up = top > m_run[nt][c];
            alpha[c] = up ? ex2_approx(m_run[nt][c] - top) : 1.f;
            m_run[nt][c] = up ? top : m_run[nt][c];
            l_run[nt][c] *= alpha[c];
          }
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            acc[nt][mt][0] *= alpha[0];
            acc[nt][mt][1] *= alpha[1];
            acc[nt][mt][2] *= alpha[0];
            acc[nt][mt][3] *= alpha[1];
          }
        }
        float sum[2] = {l_run[nt][0], l_run[nt][1]};
#pragma unroll
        for (int k = 0; k < kPages; ++k) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = s[k][nt][e], f = hs[nt][e & 1];
            float x = fmaf(y, f, -m_run[nt][e & 1]);
            if constexpr (kP == 2) x = y == -INFINITY ? y : fmaf(y, f * p.scale_log2_low, x);
            w[e] = ex2_approx(x);
          }
          sum[0] += w[0] + w[2];
          sum[1] += w[1] + w[3];
          // weights rounded to halves (the matrix operand), transposed to
          // (token pair, head)
          const __half2 p0 = __floats2half2_rn(w[0], w[1]), p1 = __floats2half2_rn(w[2], w[3]);
          pb[0][k][nt][0] = movmatrix_trans(as_u32(p0));
          pb[0][k][nt][1] = movmatrix_trans(as_u32(p1));
          if constexpr (kP == 2) {
            const float2 g0 = __half22float2(p0), g1 = __half22float2(p1);
            pb[kP - 1][k][nt][0] = movmatrix_trans(as_u32(__floats2half2_rn(w[0] - g0.x, w[1] - g0.y)));
            pb[kP - 1][k][nt][1] = movmatrix_trans(as_u32(__floats2half2_rn(w[2] - g1.x, w[3] - g1.y)));
          }
        }
        l_run[nt][0] = sum[0];
        l_run[nt][1] = sum[1];
      }
      // ---- O^T += V^T P^T ----------------------------------------------------------
      // Lane (grp, qd) holds the codes of sixteen grp of a group of 32 dims (of
      // eight of them, from 8 (grp / 2) on, the even dims or the odd ones), of
      // tokens 2 qd and 2 qd + 1 of either half page; row grp of tile 2 c + u
      // stands for its code 2 u, row grp + 8 for its code 2 u + 1.
      uint32_t sc[kPages][2][2];   // a token's scale bytes; masked tokens: 0
#pragma unroll
      for (int k = 0; k < kPages; ++k)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = 8 * h + 2 * qd;
          const uint8_t* b = stage + (kPages + k) * kSlot + q4::scales_at(D, t);
          if constexpr (kGroups == 4) {
            const uint2 w = *reinterpret_cast<const uint2*>(b);
            sc[k][h][0] = w.x;
            sc[k][h][1] = w.y;
          } else {
            const uint32_t w = *reinterpret_cast<const uint32_t*>(b);
            sc[k][h][0] = w & 0xffffu;
            sc[k][h][1] = w >> 16;
          }
          if (!whole) {
            if (!(t < hi[k] && t >= lo[k])) sc[k][h][0] = 0u;
            if (!(t + 1 < hi[k] && t + 1 >= lo[k])) sc[k][h][1] = 0u;
          }
        }
#pragma unroll
      for (int c = 0; c < kGroups; c += 2) {
        uint32_t r[kPages][4];
#pragma unroll
        for (int k = 0; k < kPages; ++k) ldsm_x4_trans(vp + k * kSlot + chunk_off<D>(v_tok, c + v_chunk), r[k]);
        // Float32: the tensor core drops bits wherever it adds to a large
        // accumulator, so a step's products start from zero and are added here
        // (errors of 30k keys against 64 bits: 6.1 and 9.4e-7 of the norm at 64
        // and 128 dims, 16 and 17e-7 with one accumulator, 7.7 and 9.1e-7 a plain
        // float32 form; 64 requests of up to 4k tokens 41.1 us either way at 64
        // dims, 64.9 and 61.5 at 128).
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float sum[kP == 2 ? kNT : 1][2][4];
#pragma unroll
          for (int k = 0; k < kPages; ++k) {
            // groups c and c + 1 of the two tokens, side by side
            const uint32_t two0 = __byte_perm(sc[k][0][0], sc[k][0][1], c ? 0x7632 : 0x5410);
            const uint32_t two1 = __byte_perm(sc[k][1][0], sc[k][1][1], c ? 0x7632 : 0x5410);
            uint32_t h0[4], h1[4];
            q4::halves8(r[k][2 * i], q4::scale_pair(two0, i), exps, h0);
            q4::halves8(r[k][2 * i + 1], q4::scale_pair(two1, i), exps, h1);
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t a[4] = {h0[2 * u], h0[2 * u + 1], h1[2 * u], h1[2 * u + 1]};
#pragma unroll
              for (int nt = 0; nt < kNT; ++nt) {
                if constexpr (kP == 2) {
                  if (k == 0) mma_f16_first(sum[nt][u], a, pb[kP - 1][k][nt][0], pb[kP - 1][k][nt][1]);
                  else mma_f16(sum[nt][u], a, pb[kP - 1][k][nt][0], pb[kP - 1][k][nt][1]);
                  mma_f16(sum[nt][u], a, pb[0][k][nt][0], pb[0][k][nt][1]);
                } else {
                  mma_f16(acc[nt][2 * (c + i) + u], a, pb[0][k][nt][0], pb[0][k][nt][1]);
                }
              }
            }
          }
          if constexpr (kP == 2) {
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
              for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][2 * (c + i) + u][e] += sum[nt][u][e];
          }
        }
      }
      __syncwarp();
      produce(st);
      st = st + 1 == kStages ? 0 : st + 1;
    }
    // ---- item end ----------------------------------------------------------------
    const bool split = d.nsplit > 1;
    bool last = false;  // the partial before this one completed its row
    if (split && pending) last = count(ws.pend[pend_at]);
    {
      // this lane's elements of a head: of each group of 32 dims the even or the
      // odd ones of eight, in tiles 2 x and 2 x + 1.  A part's lie side by side
      // (the merge puts them in order), in places 32 x + 4 grp and the next three;
      // in a row of the output those are the dims that it has after an exchange
      // with the lane that has the eight's others.
      const int64_t base = split ? (int64_t)d.slot * Hq + d.h0 : (int64_t)d.token * Hq + d.h0;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float l = l_run[nt][c];
#pragma unroll
          for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
          const int h = nt * 8 + 2 * qd + c;
          if (!split) {
#pragma unroll
            for (int x = 0; x < kGroups; ++x) {
              const float4 o = exchange_odd(make_float4(acc[nt][2 * x][c], acc[nt][2 * x][c + 2], acc[nt][2 * x + 1][c],
                                                        acc[nt][2 * x + 1][c + 2]), grp & 1, 4);
              acc[nt][2 * x][c] = o.x;
              acc[nt][2 * x][c + 2] = o.y;
              acc[nt][2 * x + 1][c] = o.z;
              acc[nt][2 * x + 1][c + 2] = o.w;
            }
          }
          if (h < d.heads) {
            const float inv = split ? 1.f : 1.f / l;
#pragma unroll
            for (int x = 0; x < kGroups; ++x) {
              const float o[4] = {acc[nt][2 * x][c] * inv, acc[nt][2 * x][c + 2] * inv,
                                  acc[nt][2 * x + 1][c] * inv, acc[nt][2 * x + 1][c + 2] * inv};
              const int64_t e = (base + h) * D + 32 * x + 4 * grp;
              if (split || kP == 2)
                *reinterpret_cast<float4*>((split ? p.part_acc : static_cast<float*>(p.out)) + e) =
                    make_float4(o[0], o[1], o[2], o[3]);
              else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + e) =
                    make_uint2(float2_to_bf16x2(o[0], o[1]), float2_to_bf16x2(o[2], o[3]));
            }
            if (split && grp == 0) *reinterpret_cast<float2*>(p.part_ml + (base + h) * 2) = make_float2(m_run[nt][c], l);
          }
        }
    }
    if (last) merge(ws.pend[pend_at]);
    if (split) {
      pend_at ^= 1;
      if (lane == 0) ws.pend[pend_at] = d;
      pending = true;
      __syncwarp();
    }
    ++item;
  }
  if (pending && count(ws.pend[pend_at])) merge(ws.pend[pend_at]);
  // beside the prefill grid before it: this grid completes only after it
  if (p.pdl_mode == 2 && blockIdx.x == 0 && threadIdx.x == 0)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace decode_q4
}  // namespace cb
