// How a launch of decode rows is cut into work items, computed in the kernel
// from the rows' lengths: shared by the decode kernels over the 16/32-bit
// and the 8-bit caches.
#pragma once

#include <cstdint>

#include "decode_launch.h"
#include "device_utils.cuh"
#include "row_checks.h"

namespace cb {
namespace decode {

constexpr int kPageTokens = 16;
constexpr int kTailDiv = 8;         // the last 1/kTailDiv of each row's pages: phase B
constexpr int kMinSplitPages = 8;   // phase-A split size floor
// shared memory of the plan: split-count prefixes of both phases, and each
// row's sequence length (0 for a row that is skipped) and query token
constexpr int kPlanSmemBytes = (2 * (kPlanMax + 1) + 2 * kPlanMax) * (int)sizeof(int32_t);

// How a row of `pages` pages is cut, given the launch-wide split sizes spa
// (phase A) and spb (phase B): phase A covers pages [0, bp) in na full
// splits of spa pages, na = floor(leading (1 - 1/kTailDiv) of the row / spa);
// phase B covers the rest, [bp, pages), in nb splits of spb pages (the last
// one shorter).
struct RowSplit {
  int na, size, bp, nb;
};

// First key and first page a decode row of length L reads (window W, 0 = all).
__device__ __forceinline__ int first_key(int L, int W) { return W > 0 && L > W ? L - W : 0; }
__device__ __forceinline__ int first_page(int L, int W) { return first_key(L, W) / kPageTokens; }

// With `even` > 0 the leading part is cut into equal splits instead, whole
// multiples of `even` pages and as near to spa as that comes, so that less is
// left for phase B (the last of them may end the row, and be shorter).
__device__ __forceinline__ RowSplit row_split(int pages, int spa, int spb, int even = 0) {
  RowSplit s;
  const int big = pages - pages / kTailDiv;
  s.size = spa;
  s.na = big / spa;
  if (even > 0 && spa < (1 << 20) && big > 0) {
    const int n = max(1, (big + spa / 2) / spa);
    s.size = ((big + n - 1) / n + even - 1) / even * even;
    s.na = (big + s.size - 1) / s.size;
  }
  s.bp = min(s.na * s.size, pages);
  s.nb = (pages - s.bp + spb - 1) / spb;
  return s;
}

struct PlanRows {
  const int32_t* seq_lens;
  const int32_t* cu_seqlens_q;
  int32_t row_begin, num_rows, num_tokens;
  int32_t max_blocks;   // block-table columns
  int32_t units;        // items a (row, split) has: KV heads, or parts of them
  int32_t window;
  int32_t max_slots;    // partial slots available (>= 2 * num_rows)
  int32_t items_a;      // phase-A items per warp (target)
  uint32_t* error_word;
  // Splits are whole multiples of `step` pages (even: see row_split).
  // max_splits > 0: the longest row has about that many phase-A splits at
  // most, and half as many in phase B; and with at most single_pages pages to
  // a warp there is one phase, of one item to a warp (and that limit).
  int32_t step = 1;
  int32_t even = 0;
  int32_t max_splits = 0;
  int32_t single_pages = 0;
  int32_t single_least = 0;  // pages of an item of that one phase, at least
};

// ceil(a / b); the 64-bit division takes several times the 32-bit one's time
__device__ __forceinline__ int64_t ceil_div(int64_t a, int64_t b) {
  const uint64_t x = (uint64_t)(a + b - 1);
  return ((x | (uint64_t)b) >> 32) == 0 ? (int64_t)((uint32_t)x / (uint32_t)b) : (int64_t)(x / (uint64_t)b);
}

struct SplitPlan {
  int spa, spb;  // split sizes of the two phases, in pages
  bool ok;
};

// Every CTA computes the same plan, in shared memory: plan_a, plan_b
// [num_rows + 1] are the prefixes of the rows' split counts in each phase,
// row_len [num_rows] their lengths (0: skipped), row_tok their query tokens.
template <int kMaxWarps>
__device__ __forceinline__ SplitPlan plan_splits(const PlanRows& in, int nwarps, int32_t* plan_a,
                                                 int32_t* plan_b, int32_t* row_len,
                                                 int32_t* row_tok) {
  __shared__ int32_t s_red[2][kMaxWarps];
  __shared__ int32_t s_spa, s_spb;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nthreads = nwarps * 32;
  // Rows are checked once here and kept in shared memory; a row that fails a
  // check gets length 0 (no items) and its error bit.
  int64_t my_pages = 0;
  int32_t my_longest = 0;
  for (int i = threadIdx.x; i < in.num_rows; i += nthreads) {
    const int r = in.row_begin + i;
    int L = in.seq_lens[r];
    const int q0 = in.cu_seqlens_q[r];
    const int q1 = in.cu_seqlens_q[r + 1];
    if (L == 0 && q1 == q0) {
      // a padding row (no query, no context): nothing to do
    } else {
      if (!row_length_fits(L, kPageTokens, in.max_blocks)) {
        L = 0;
        if (blockIdx.x == 0) set_error(in.error_word, CB_DEVERR_SEQ_RANGE);
      }
      if (q1 - q0 != 1 || q0 < 0 || q0 >= in.num_tokens) {
        L = 0;
        if (blockIdx.x == 0) set_error(in.error_word, CB_DEVERR_DECODE_QLEN);
      }
    }
    const int pages = blocks_of(L, kPageTokens) - first_page(L, in.window);
    row_len[i] = L;
    row_tok[i] = q0;
    my_pages += pages;
    my_longest = max(my_longest, pages);
  }
  my_longest = __reduce_max_sync(0xffffffffu, my_longest);
  for (int o = 16; o > 0; o >>= 1) my_pages += __shfl_xor_sync(0xffffffffu, my_pages, o);
  if (lane == 0) {
    s_red[0][warp] = (int32_t)(my_pages < 0x3fffffff ? my_pages : 0x3fffffff);
    s_red[1][warp] = my_longest;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int64_t tot = 0;
    int32_t longest = 0;
    for (int w = 0; w < nwarps; ++w) {
      tot += s_red[0][w];
      longest = max(longest, s_red[1][w]);
    }
    const int64_t units = tot * in.units;
    const int64_t units_b = units / kTailDiv;
    const int64_t workers = (int64_t)gridDim.x * nwarps;
    const int64_t items_a = in.items_a;
    int64_t spa = ceil_div(units - units_b, workers * items_a);
    int64_t spb = ceil_div(units_b, workers * kItemsB);
    if (spa < kMinSplitPages) spa = kMinSplitPages;
    if (spb < 1) spb = 1;
    if (in.max_splits > 0) {
      const int64_t least = ceil_div(longest, in.max_splits);
      if (units <= workers * in.single_pages) {
        spb = ceil_div(units, workers);
        if (spb < in.single_least) spb = in.single_least;
        if (spb < least) spb = least;
        spa = 1 << 20;
      } else {
        if (spa < least) spa = least;
        const int64_t tail = (longest / kTailDiv + spa) * 2 / in.max_splits;
        if (spb < tail) spb = tail;
      }
    }
    spa = (spa + in.step - 1) / in.step * in.step;
    spb = (spb + in.step - 1) / in.step * in.step;
    s_spa = (int32_t)(spa < (1 << 20) ? spa : (1 << 20));
    s_spb = (int32_t)(spb < (1 << 20) ? spb : (1 << 20));
  }
  __syncthreads();
  int spa0 = s_spa, spb0 = s_spb;
  // per row split counts of both phases and their prefixes (serial segments
  // per thread + a block scan of the segment sums); if the splits exceed the
  // partial slots, double both split sizes and plan again
  for (int attempt = 0;; ++attempt) {
    const int seg = (in.num_rows + nthreads - 1) / nthreads;
    const int b = threadIdx.x * seg;
    const int e = min(b + seg, in.num_rows);
    int sum_a = 0, sum_b = 0;
    for (int i = b; i < e; ++i) {
      const int Li = row_len[i];
      const RowSplit rs =
          row_split(blocks_of(Li, kPageTokens) - first_page(Li, in.window), spa0, spb0, in.even);
      const int na = rs.na, nb = rs.nb;
      plan_a[i + 1] = na;
      plan_b[i + 1] = nb;
      sum_a += na;
      sum_b += nb;
    }
    int inc_a = sum_a, inc_b = sum_b;
    for (int o = 1; o < 32; o <<= 1) {
      const int va = __shfl_up_sync(0xffffffffu, inc_a, o);
      const int vb = __shfl_up_sync(0xffffffffu, inc_b, o);
      if (lane >= o) {
        inc_a += va;
        inc_b += vb;
      }
    }
    if (lane == 31) {
      s_red[0][warp] = inc_a;
      s_red[1][warp] = inc_b;
    }
    __syncthreads();
    int off_a = 0, off_b = 0;
    for (int w = 0; w < warp; ++w) {
      off_a += s_red[0][w];
      off_b += s_red[1][w];
    }
    int run_a = off_a + inc_a - sum_a, run_b = off_b + inc_b - sum_b;
    if (threadIdx.x == 0) {
      plan_a[0] = 0;
      plan_b[0] = 0;
    }
    for (int i = b; i < e; ++i) {
      run_a += plan_a[i + 1];
      run_b += plan_b[i + 1];
      plan_a[i + 1] = run_a;
      plan_b[i + 1] = run_b;
    }
    __syncthreads();
    if (plan_a[in.num_rows] + plan_b[in.num_rows] <= in.max_slots || attempt >= 40) break;
    if (spa0 < (1 << 29)) spa0 *= 2;
    if (spb0 < (1 << 29)) spb0 *= 2;
    __syncthreads();  // everyone has read the totals before they are rewritten
  }
  // unreachable with max_slots >= 2 * num_rows; refuse rather than overrun
  const bool plan_ok = plan_a[in.num_rows] + plan_b[in.num_rows] <= in.max_slots &&
                       (int64_t)(plan_a[in.num_rows] + plan_b[in.num_rows]) * in.units < (1 << 26);
  if (!plan_ok && blockIdx.x == 0 && threadIdx.x == 0) set_error(in.error_word, CB_DEVERR_PLAN);
  return SplitPlan{spa0, spb0, plan_ok};
}

}  // namespace decode
}  // namespace cb
