// Split-KV decode attention over the 8-bit cache (one query token per row).
//
// The definition is the decode kernel's ("Chunked Prefill", How chunked
// prefill works: the query at position seq_len - 1 attends every cached key
// of its request) with keys code * 2^ek and values code * 2^ev, one exponent
// for each (block, KV head).  The cache is read once, half the bytes of the
// 16-bit one, so HBM bounds it and at the same rate twice as many elements a
// second pass through each SM.  What that asks for:
//
//   * Work items, plan, dealing and the merge of splits are the decode
//     kernel's (split_plan.cuh): runs of pages of one (row, KV head), drawn
//     by independent warps; the warp whose ticket completes a row merges it.
//     A KV head with more than 16 query heads is served in parts.
//   * Each warp keeps a ring of kStages stages of two pages (K page, V page,
//     two scale bytes): a page is one TMA box (16 rows of D bytes, swizzled
//     over the row's width); the scales come by 4-byte asynchronous copies
//     that arrive on the same barrier.  Two pages to a step: their chains of
//     loads, conversions and matrix instructions are independent, and one
//     softmax step (reference, shuffles, rescaling) serves 32 tokens.
//   * Codes become halves (every e4m3 number is one exactly) by one
//     conversion for two elements, and both products of a page run as
//     m16n8k16 matrix instructions with float32 accumulation.  K codes are
//     loaded as 16-byte vectors: the contraction over the dims has no order,
//     so lane qd of a row takes dims 16 qd .. 16 qd + 15 of each 64 and Q^T is
//     loaded in the same order.  V codes come through transposing loads of
//     pairs of dims; a byte permute turns (token, token + 1) x (dim, dim + 1)
//     into the two pairs that the conversion wants, and the output rows are
//     the dims in that order.  Rows of the fragments stand for tokens in an
//     order that keeps both kinds of loads free of bank conflicts.
//   * Queries are scaled by a power of two to the halves' range for each
//     head, so that bfloat16 queries are halves exactly (elements under
//     2^-29 of the head's largest lose bits); float32 queries are split into
//     two halves (22 bits), and their weights too (and to 2^-24, the least
//     half, where the largest is 2^-0.5 at least).  With those, score
//     exponents are rounded at their size next to the reference: scale *
//     log2(e) is a pair of floats, the reference a whole number.
//   * Scales never touch the codes.  With x = score * log2(e), the weight
//     that multiplies a value code is 2^(x + ev - m): the running reference m
//     is over x + ev, so a block of large values and a block of small ones
//     share it, weights stay in a half's range (2^7 at the reference, 2^15
//     at most, rounded to multiples of 2^-24 at least), and the sum of weights adds 2^(x - m) = 2^(x
//     + ev - m) * 2^-ev in float32.  Exponents lie in [-40, 40], so that no
//     page's part of the sum can leave float32's range.
//
// What bounds it: at long contexts HBM (128 requests of up to 32k tokens, 64
// + 8 heads of 128: 635 us, 6.3 TB/s, 95% of the measured copy rate; without
// the arithmetic 605 us); at short ones what an item costs beside its pages
// and the end of the kernel (64 requests of up to 4k tokens 63.4 us, 4.6 TB/s:
// of that 4 us until the first page lands and 10 us from the median warp's
// last item to the last merge; 8 of up to 512 tokens 12.2 us, of which the
// plan takes 2, the first page 2.5, the item 3 and ticket and merge 3).
// e4m3 matrix instructions (warp-level m16n8k32, queries and weights split
// into e5m2 pieces) were exact enough but 1.5 times slower: they took two tensor
// instructions each and more conversions than the halves do.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <type_traits>

#include "decode_launch.h"
#include "device_utils.cuh"
#include "mma_utils.cuh"
#include "q8.cuh"
#include "split_plan.cuh"

namespace cb {
namespace decode_q8 {

using namespace decode;

// Warps of a CTA: the fragments take up to 255 registers a thread (12 warps
// of 168 registers measured the same rate at long contexts and less at short
// ones).
constexpr int kWarps = 8;
constexpr int kMaxHeads = 16;  // query heads of an item
constexpr int kPair = 2;       // pages of a stage
// An item costs about two microseconds beside its pages (its queries, its
// place in the plan, its partial and ticket), and joining a row's splits about
// one for 8 of them.  So a row is cut into equal splits, of a size that gives
// each warp kItemsEven of them (64 requests of up to 4k tokens: 64.1 us; 68.4
// with one, 69.9 with three; 67.5 with whole multiples of one size, whose
// remainders all went to the last phase).  A step with few pages to a warp is
// cut into one item each, of at least kSingleLeast pages (8 requests of up to
// 512 tokens: 12.4 us, 13.4 without the least, 19 with two phases), and a long
// row into at most kMaxSplits and the last phase's (one request of 32k tokens:
// 41 us; without the limit half as long again).
constexpr int kItemsEven = 2;
constexpr int kSinglePages = 8;
constexpr int kSingleLeast = 4;
constexpr int kMaxSplits = 64;
// weight exponent at the reference, which moves when passed by more than the
// lag (float32: exponents near 0 are the most exact)
template <typename T> constexpr float kTop = 7.f;
template <> constexpr float kTop<float> = 0.f;
template <typename T> constexpr float kLag = 8.f;
template <> constexpr float kLag<float> = 2.f;

struct Params {
  CUtensorMap tmap_k;  // [num_blocks * Hkv * 16 rows][D] bytes, box 16 rows x D
  CUtensorMap tmap_v;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  int64_t scale_stride;
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
  uint64_t wait_ns;
  int32_t pdl_mode;
  int32_t withhold_item;
};

struct alignas(16) ItemDesc {
  int32_t r, u, nsplit, slot;          // row, unit (part of a KV head), splits of the row, partial slot
  int32_t page0, page1, seq_len, token;
  int32_t g, h0, heads, pad;           // KV head, first query head, query heads
};

// Shared memory: every warp's page ring first (1024-byte aligned for the
// swizzle), then each warp's small state, then the plan.
template <int D, int kStages>
struct Layout {
  static constexpr int kPageBytes = kPageTokens * D;
  static constexpr int kStageBytes = 2 * kPair * kPageBytes;   // K pages | V pages
  static constexpr int kRingBytes = kStages * kStageBytes;     // of a warp
  // items the ring can hold pages of at once, and the one dealt ahead
  static constexpr int kItemSlots = kStages + 2;
  struct State {
    uint64_t full[kStages];
    uint32_t scales[kStages][kPair][2];       // the words around the K and the V scale
    int32_t scale_shift[kStages][kPair];      // bit offsets of the bytes: K | V << 8
    ItemDesc items[kItemSlots];
    ItemDesc pend[2];                         // the items of the last two partials
  };
  static_assert(kRingBytes % 1024 == 0, "ring alignment");
  static constexpr int kStateBytes = ((int)sizeof(State) + 15) / 16 * 16;
  static constexpr size_t total(int warps) {
    return (size_t)warps * (kRingBytes + kStateBytes) + kPlanSmemBytes + 1024;
  }
};

// Byte offset of 16-byte chunk c of page row t under the TMA swizzle (128
// bytes: chunk XOR row mod 8; 64 bytes: chunk XOR row / 2 mod 4).
template <int D>
__device__ __forceinline__ uint32_t chunk_off(int t, int c) {
  if constexpr (D == 128) return (uint32_t)(t * 128 + ((c ^ (t & 7)) << 4));
  return (uint32_t)(t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
}
// Token of fragment row r (0..7): two neighbouring rows' K vectors must lie
// in different halves of the banks.
template <int D>
__device__ __forceinline__ int row_token(int r) {
  return D == 128 ? (r >> 1) | ((r & 1) << 2) : r;
}

// Merge the n >= 2 split partials of one item group (row, heads h0 .. h0 +
// heads), whose slots start at s0, into the rows of query token q0: per head
// o = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s, in split order.
// Not inlined: it is rare.  Its caller keeps nothing alive across the call.
template <typename T, int D>
__device__ __noinline__ void merge_splits(const float* part_ml, const float* part_acc, void* out, int Hq,
                                            int h0, int heads, int s0, int n, int q0) {
  const int lane = threadIdx.x & 31;
  constexpr int kV = D / 4;      // lanes that own 4 elements each
  constexpr int kH = 4;          // heads at once
  constexpr int kB = 4;          // splits in flight: more takes registers that the caller would spill
  for (int hb = 0; hb < heads; hb += kH) {
    float M[kH], Ls[kH];
    float4 o[kH];
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      M[h] = -INFINITY;
      Ls[h] = 0.f;
      o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int b0 = 0; b0 < n; b0 += 32) {
      const int cnt = min(32, n - b0);
      float4 a[kB][kH];
      auto load = [&](int k0) {
#pragma unroll
        for (int k = 0; k < kB; ++k)
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const int head = h0 + min(hb + h, heads - 1);
            a[k][h] = k0 + k < cnt && lane < kV
                          ? __ldcg(reinterpret_cast<const float4*>(part_acc) +
                                   ((int64_t)(s0 + b0 + k0 + k) * Hq + head) * kV + lane)
                          : make_float4(0.f, 0.f, 0.f, 0.f);
          }
      };
      load(0);  // beside the sums and references
      float wl[kH];
#pragma unroll
      for (int h = 0; h < kH; ++h) {
        const int head = h0 + min(hb + h, heads - 1);
        const float2 v = lane < cnt ? __ldcg(reinterpret_cast<const float2*>(part_ml) +
                                             (int64_t)(s0 + b0 + lane) * Hq + head)
                                    : make_float2(-INFINITY, 0.f);
        float bm = v.x;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) bm = fmaxf(bm, __shfl_xor_sync(0xffffffffu, bm, k));
        const float Mn = fmaxf(M[h], bm);
        wl[h] = lane < cnt ? exp2f(v.x - Mn) : 0.f;
        float lsum = wl[h] * v.y;
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) lsum += __shfl_xor_sync(0xffffffffu, lsum, k);
        const float a_old = exp2f(M[h] - Mn);
        Ls[h] = Ls[h] * a_old + lsum;
        o[h].x *= a_old; o[h].y *= a_old; o[h].z *= a_old; o[h].w *= a_old;
        M[h] = Mn;
      }
#pragma unroll 1
      for (int k0 = 0; k0 < cnt; k0 += kB) {
#pragma unroll
        for (int k = 0; k < kB; ++k)
#pragma unroll
          for (int h = 0; h < kH; ++h) {
            const float w = __shfl_sync(0xffffffffu, wl[h], (k0 + k) & 31);
            if (k0 + k < cnt) {
              o[h].x += w * a[k][h].x; o[h].y += w * a[k][h].y; o[h].z += w * a[k][h].z; o[h].w += w * a[k][h].w;
            }
          }
        if (k0 + kB < cnt) load(k0 + kB);
      }
    }
#pragma unroll
    for (int h = 0; h < kH; ++h) {
      if (hb + h < heads && lane < kV) {
        const float inv = 1.f / Ls[h];
        T* row = static_cast<T*>(out) + ((int64_t)q0 * Hq + h0 + hb + h) * D + 4 * lane;
        if constexpr (sizeof(T) == 2) {
          *reinterpret_cast<uint2*>(row) = make_uint2(float2_to_bf16x2(o[h].x * inv, o[h].y * inv),
                                                      float2_to_bf16x2(o[h].z * inv, o[h].w * inv));
        } else {
          *reinterpret_cast<float4*>(row) = make_float4(o[h].x * inv, o[h].y * inv, o[h].z * inv, o[h].w * inv);
        }
      }
    }
  }
}

// Count one split of an item group done; true for the warp whose ticket
// completes the count of n: it merges the splits and leaves the counter zero.
// Lane 0 releases what the warp wrote before and acquires what the others
// did (64 requests: 63.5 us, 64.1 with a fence of all lanes on either side).
__device__ __forceinline__ bool count_split(uint32_t* cnt, int n, int lane) {
  __syncwarp();
  uint32_t old = 0;
  if (lane == 0) {
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(cnt) : "memory");
    if (old == (uint32_t)n - 1) *cnt = 0u;
  }
  old = __shfl_sync(0xffffffffu, old, 0);
  __syncwarp();
  return old == (uint32_t)n - 1;
}

template <typename T, int D, int kNT, int kStages>
__global__ void __launch_bounds__(kWarps * 32, 1) decode_kernel(const __grid_constant__ Params p) {
  // pieces of a query element and of a weight: one half, or two for float32
  constexpr int kP = std::is_same<T, float>::value ? 2 : 1;
  constexpr int kJ = D / 64;        // 16-byte K vectors of a lane and row
  constexpr int kMT = D / 16;       // 16-dim tiles of the output
  using Lay = Layout<D, kStages>;
  using State = typename Lay::State;
  constexpr int kRing = Lay::kItemSlots;
  constexpr int kPageBytes = Lay::kPageBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int nwarps = (int)(blockDim.x >> 5);
  const int Hkv = p.num_kv_heads, Hq = p.num_q_heads;
  const int units = Hkv * p.parts;
  const int W = p.max_blocks_per_seq;
  const int win = p.window;
  uint8_t* ring = smem + warp * Lay::kRingBytes;
  State& ws = *reinterpret_cast<State*>(smem + nwarps * Lay::kRingBytes + warp * Lay::kStateBytes);
  int32_t* plan_a = reinterpret_cast<int32_t*>(smem + nwarps * (Lay::kRingBytes + Lay::kStateBytes));
  int32_t* plan_b = plan_a + (kPlanMax + 1);
  int32_t* row_len = plan_b + (kPlanMax + 1);
  int32_t* row_tok = row_len + kPlanMax;

  const SplitPlan plan = plan_splits<kWarps>(
      PlanRows{p.seq_lens, p.cu_seqlens_q, p.row_begin, p.num_rows, p.num_tokens, W, units, win,
               p.max_slots, kItemsEven, p.error_word, kPair, kPair, kMaxSplits, kSinglePages, kSingleLeast},
      nwarps, plan_a, plan_b, row_len, row_tok);
  const int spa0 = plan.spa, spb0 = plan.spb;
  const int num_a = plan_a[p.num_rows];
  const int num_b = plan_b[p.num_rows];
  const int total_items = plan.ok ? (num_a + num_b) * units : 0;
  const uint32_t total_workers = gridDim.x * nwarps;

  if (lane == 0) {
    // a stage is full after each page's bytes and its scales' copies
    for (int s = 0; s < kStages; ++s) mbar_init(&ws.full[s], 2 * kPair);
    fence_barrier_init();
  }
  __syncwarp();
  const uint64_t pol = l2_policy_evict_first();

  // ---- dealing: the first item is dealt statically (item w of W warps),
  // later ones are drawn from the counter.  Two steps before the producer
  // reaches the end of its item it draws the next one, and one step before,
  // it decodes that item and requests its first block ids: early enough that
  // neither is waited for, and no earlier, since an item drawn is one that no
  // idle warp can take (drawn with the item before, two ahead, most of the
  // small items were dealt when the call began).  Beside a prefill grid every
  // item is drawn.
  const int items_a = num_a * units;
  // warp w of every CTA before warp w + 1 of any: when there are fewer large
  // items than warps, every SM gets its share of them
  const uint32_t worker = warp * gridDim.x + blockIdx.x;
  const uint32_t n_static =
      p.pdl_mode == 2 ? 0u : (uint32_t)min((int64_t)items_a, (int64_t)total_workers);
  bool first_static = worker < n_static;
  const uint32_t items_dyn = (uint32_t)total_items - n_static;
  uint32_t draw = 0;           // lane 0: the counter's value, drawn for the next item
  enum { kNone, kDrawn, kKnown };
  int nx = kNone;              // the item after the producer's
  const uint64_t units_magic = (0x100000000ull + units - 1) / units;  // exact: items < 2^26, units <= 64
  // the item dealt ahead is described in the ring already; lane i holds the
  // block id of its page i
  bool nx_ok = false;
  int nx_blk = -1;
  // the producer's item and the next page to copy
  int prod_page = 0, prod_end = 0, prod_row = 0, prod_g = 0;
  int prod_items = 0, cons_items = 0;
  bool prod_withheld = false, withhold_next = false;  // test hook
  int win_base = 0, blk_win = -1, blk_win2 = -1;  // lane i: block id of page win_base (+ 32) + i
  bool exhausted = false, aborted = false;
  uint32_t phases = 0;
  int ahead = 0;                                  // stages issued and not consumed

  const int fr_step = (p.num_rows + 31) >> 5;
  auto find_row = [&](const int32_t* pre, int x) -> int {
    const int i1 = lane * fr_step;
    const bool le1 = i1 < p.num_rows && pre[i1] <= x;
    const int base = (__popc(__ballot_sync(0xffffffffu, le1)) - 1) * fr_step;
    const int i2 = base + lane;
    const bool le2 = lane < fr_step && i2 < p.num_rows && pre[i2] <= x;
    return base + __popc(__ballot_sync(0xffffffffu, le2)) - 1;
  };

  auto draw_next = [&]() {
    nx = kDrawn;
    if (!first_static && items_dyn > 0) lane0_fetch_add1(p.work_counter, draw, lane);
  };
  auto fetch_ahead = [&]() {
    nx = kKnown;
    nx_ok = false;
    uint32_t idx;
    if (first_static) {
      idx = worker;
      first_static = false;
    } else {
      if (items_dyn == 0) return;
      const uint32_t b = __shfl_sync(0xffffffffu, draw, 0);
      if (b >= items_dyn) {
        // every warp draws once past the end; the last of them resets
        if (b == items_dyn + total_workers - 1 && lane == 0) atomicExch(p.work_counter, 0u);
        return;
      }
      idx = n_static + b;
    }
    const uint32_t x = (uint32_t)(((uint64_t)idx * units_magic) >> 32);
    const bool phase_a = (int)x < num_a;
    const int i = phase_a ? find_row(plan_a, (int)x) : find_row(plan_b, (int)x - num_a);
    const int a0 = plan_a[i], na = plan_a[i + 1] - a0, b0 = plan_b[i], nb = plan_b[i + 1] - b0;
    const int split = phase_a ? (int)x - a0 : (int)x - num_a - b0;
    const int L = row_len[i];
    const int fp = first_page(L, win), end = blocks_of(L, kPageTokens);
    const RowSplit rs = row_split(end - fp, spa0, spb0, kPair);
    nx_ok = true;
    const int u = (int)(idx - x * (uint32_t)units);
    int page0, page1;
    if (phase_a) {
      page0 = fp + split * rs.size;
      page1 = min(end, page0 + rs.size);
    } else {
      page0 = fp + rs.bp + split * spb0;
      page1 = min(end, page0 + spb0);
    }
    if (lane == 0) {
      ItemDesc& d = ws.items[prod_items % kRing];
      const int g = u / p.parts, part = u - g * p.parts;
      d.r = i;
      d.u = u;
      d.nsplit = na + nb;
      d.slot = a0 + b0 + (phase_a ? split : na + split);
      d.page0 = page0;
      d.page1 = page1;
      d.seq_len = L;
      d.token = row_tok[i];
      d.g = g;
      d.h0 = g * p.group + part * p.part_heads;
      d.heads = min(p.part_heads, p.group - part * p.part_heads);
    }
    withhold_next = (int)idx == p.withhold_item;
    const int pg = page0 + lane;
    nx_blk = pg < page1 ? __ldg(p.block_tables + (int64_t)(p.row_begin + i) * W + pg) : -1;
  };

  auto next_item = [&]() -> bool {
    if (nx == kNone) draw_next();
    if (nx == kDrawn) fetch_ahead();
    if (!nx_ok) return false;
    nx = kNone;
    __syncwarp();
    const ItemDesc d = ws.items[prod_items % kRing];
    ++prod_items;
    prod_row = p.row_begin + d.r;
    prod_g = d.g;
    prod_page = win_base = d.page0;
    prod_end = d.page1;
    prod_withheld = withhold_next;
    blk_win = nx_blk;
    return true;
  };
  draw_next();
  fetch_ahead();

  // refill one stage with the producer's next pages: two of one item, or its
  // last one (whole warp)
  auto produce = [&](int st) {
    if (exhausted || aborted) return;
    bool first = false;
    if (prod_page >= prod_end) {
      if (!next_item()) { exhausted = true; return; }
      first = true;
    }
    if (prod_page - win_base == 16 && win_base + 32 < prod_end) {
      const int pg = win_base + 32 + lane;
      blk_win2 = pg < prod_end ? __ldg(p.block_tables + (int64_t)prod_row * W + pg) : -1;
    }
    if (prod_page - win_base >= 32) {
      win_base += 32;
      blk_win = blk_win2;
    }
    // lane k copies page prod_page + k (the window holds both: steps are even)
    const int blk = __shfl_sync(0xffffffffu, blk_win, (prod_page - win_base + lane) & 31);
    if (lane < kPair) {
      uint64_t* full = &ws.full[st];
      uint8_t* dst = ring + st * Lay::kStageBytes + lane * kPageBytes;
      if (prod_page + lane >= prod_end) {
        // no such page: its tokens are masked
        mbar_arrive(full);
        mbar_arrive(full);
      } else if (blk >= 0 && blk < p.num_blocks) {
        // the stage's previous contents were read (generic proxy) before the
        // __syncwarp that precedes this call; the copies only write it
        mbar_arrive_expect_tx(full, 2u * kPageBytes);
        // the scale bytes: the aligned words that hold them (each lies in its
        // byte's own 4 bytes, so nothing outside the allocation is touched)
        const int64_t at = (int64_t)blk * p.scale_stride + prod_g;
        const uintptr_t ks = reinterpret_cast<uintptr_t>(p.k_scales + at);
        const uintptr_t vs = reinterpret_cast<uintptr_t>(p.v_scales + at);
        cp_async4(smem_addr(&ws.scales[st][lane][0]), reinterpret_cast<const void*>(ks & ~uintptr_t(3)));
        cp_async4(smem_addr(&ws.scales[st][lane][1]), reinterpret_cast<const void*>(vs & ~uintptr_t(3)));
        ws.scale_shift[st][lane] = (int)((ks & 3) * 8 + (vs & 3) * 2048);
        cp_async_mbar_arrive(full);
        // test hook: the withheld item's first pages are announced but never
        // copied, so the consumer's bounded wait on them runs out
        if (!(first && prod_withheld)) {
          const int row = (blk * Hkv + prod_g) * kPageTokens;
          tma_load_2d_hint(dst, &p.tmap_k, 0, row, full, pol);
          tma_load_2d_hint(dst + kPair * kPageBytes, &p.tmap_v, 0, row, full, pol);
        }
      } else {
        set_error(p.error_word, CB_DEVERR_BLOCK_RANGE);
        // unreadable page: zero it so the math stays finite
        ws.scales[st][lane][0] = ws.scales[st][lane][1] = 0x7f7f7f7fu;
        ws.scale_shift[st][lane] = 0;
        uint4* z = reinterpret_cast<uint4*>(dst);
        for (int k = 0; k < kPageBytes / 16; ++k)
          z[k] = z[k + kPair * kPageBytes / 16] = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();  // before a later page's copy into this stage
        mbar_arrive(full);
        mbar_arrive(full);
      }
    }
    prod_page += kPair;
    if (nx == kNone && prod_end - prod_page <= 2 * kPair) draw_next();
    else if (nx == kDrawn && prod_end - prod_page <= kPair) fetch_ahead();
    ++ahead;
    __syncwarp();
  };

  // ---- split tickets: one for each item of a split row; a partial is
  // counted when the warp writes its next one (or finishes), by when its
  // stores are long complete and the fence rarely waits.  A warp that aborted
  // still counts its splits, so that the counters return to zero, but merges
  // nothing.
  auto count = [&](const ItemDesc& d) {
    return count_split(p.done + (int64_t)d.r * units + d.u, d.nsplit, lane) && !aborted;
  };
  auto merge = [&](const ItemDesc& d) {
    merge_splits<T, D>(p.part_ml, p.part_acc, p.out, Hq, d.h0, d.heads, plan_a[d.r] + plan_b[d.r], d.nsplit, d.token);
  };
  bool pending = false;     // ws.pend[pend_at]: the item of the partial not counted yet
  int pend_at = 0;

  // the cache is read from here on: behind this step's append when the
  // launch overlaps it (a prefill grid beside has begun behind the append)
  if (p.pdl_mode != 2) asm volatile("griddepcontrol.wait;" ::: "memory");
#pragma unroll 1
  for (int s = 0; s < kStages; ++s) produce(s);

  // fragment roles: rows grp and grp + 8, columns 2 qd and 2 qd + 1
  const int grp = lane >> 2, qd = lane & 3;
  const int mi = lane >> 3, rr = lane & 7;
  const int tok0 = row_token<D>(grp);               // K: token of row grp (+ 8: of row grp + 8)
  const int v_tok = row_token<D>(rr) + ((mi & 1) << 3), v_chunk = mi >> 1;

  uint32_t qb[kP][kNT][kJ * 4][2];   // Q^T fragments
  float hs[kNT][2];                  // score factor of this lane's two heads
  float acc[kNT][kMT][4];
  float m_run[kNT][2], l_run[kNT][2];
  // the consumer's item: its next page and its end; pages [c_lo, c_hi) of it
  // are read whole
  int c_page = 0, c_end = 0, c_lo = 0, c_hi = 0;
  auto reset = [&]() {
#pragma unroll
    for (int nt = 0; nt < kNT; ++nt) {
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[nt][mt][e] = 0.f;
#pragma unroll
      for (int i = 0; i < kP; ++i)
#pragma unroll
        for (int k = 0; k < kJ * 4; ++k) qb[i][nt][k][0] = qb[i][nt][k][1] = 0u;
      m_run[nt][0] = m_run[nt][1] = -INFINITY;
      l_run[nt][0] = l_run[nt][1] = hs[nt][0] = hs[nt][1] = 0.f;
    }
  };
  reset();
  int st = 0;
  while (ahead > 0) {
    const bool new_item = c_page >= c_end;
    uint4 qx[kNT][kJ][sizeof(T)];      // 16 elements each
    if (new_item) {
      // the next item: its queries are loaded while its first pages land
      const ItemDesc& d = ws.items[cons_items % kRing];
      c_page = d.page0;
      c_end = d.page1;
      c_lo = blocks_of(first_key(d.seq_len, win), kPageTokens);
      c_hi = min(c_end, d.seq_len / kPageTokens);
      const T* q0 = static_cast<const T*>(p.q) + ((int64_t)d.token * Hq + d.h0) * D + 16 * qd;
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int i = 0; i < (int)sizeof(T); ++i)
            qx[nt][j][i] = reinterpret_cast<const uint4*>(q0 + min(nt * 8 + grp, d.heads - 1) * D + 64 * j)[i];
    }
    {
      // always wait (bounded) so no copy is still landing when the CTA exits
      const bool ok = mbar_wait(&ws.full[st], (phases >> st) & 1u, p.wait_ns);
      if (!__all_sync(0xffffffffu, ok)) {
        if (!aborted && lane == 0) set_error(p.error_word, CB_DEVERR_TIMEOUT);
        aborted = true;
      }
    }
    phases ^= 1u << st;
    --ahead;
    if (new_item && !aborted) {
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        const bool live = nt * 8 + grp < ws.items[cons_items % kRing].heads;
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
        const float up = q8::exp2i(14 - k);
        const float down = p.scale_log2 * q8::exp2i(k - 14);
        hs[nt][0] = __shfl_sync(0xffffffffu, down, 8 * qd);
        hs[nt][1] = __shfl_sync(0xffffffffu, down, 8 * qd + 4);
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int s = 0; s < 4; ++s)
#pragma unroll
            for (int hlf = 0; hlf < 2; ++hlf) {
              const float a = live ? x[j][4 * s + 2 * hlf] * up : 0.f;
              const float b = live ? x[j][4 * s + 2 * hlf + 1] * up : 0.f;
              const __half2 h = __floats2half2_rn(a, b);
              qb[0][nt][j * 4 + s][hlf] = as_u32(h);
              if constexpr (kP == 2) {
                const float2 f = __half22float2(h);
                qb[kP - 1][nt][j * 4 + s][hlf] = as_u32(__floats2half2_rn(a - f.x, b - f.y));
              }
            }
      }
    }
    if (!aborted) {
      // lane 2 k + v unpacks the scale of page k's K (v = 0) or V
      float ks[kPair], ev[kPair], inv_vs[kPair];
      {
        const int k = (lane >> 1) & (kPair - 1);
        const uint32_t word = ws.scales[st][k][lane & 1];
        const int e = q8::exp_of((word >> (ws.scale_shift[st][k] >> (8 * (lane & 1)) & 31)) & 255u);
#pragma unroll
        for (int i = 0; i < kPair; ++i) {
          ks[i] = q8::exp2i(__shfl_sync(0xffffffffu, e, 2 * i));
          const int v = __shfl_sync(0xffffffffu, e, 2 * i + 1);
          ev[i] = (float)v;
          inv_vs[i] = q8::exp2i(-v);
        }
      }
      const bool whole = c_page >= c_lo && c_page + kPair <= c_hi;
      // otherwise keys [lo[k], hi[k]) of page k are read (hi <= 0: none)
      int lo[kPair], hi[kPair];
      if (!whole) {
        const int len = ws.items[cons_items % kRing].seq_len;
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          const int pg = c_page + k;
          hi[k] = pg < c_end ? min(kPageTokens, len - pg * kPageTokens) : 0;
          lo[k] = first_key(len, win) - pg * kPageTokens;
        }
      }
      const uint32_t kp = smem_addr(ring + st * Lay::kStageBytes);
      const uint32_t vp = kp + kPair * kPageBytes;

      // ---- S^T = K Q^T: an accumulator chain for each page and half of the dims
      float s[kPair][kNT][2][4];
#pragma unroll
      for (int k = 0; k < kPair; ++k)
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[k][nt][0][e] = s[k][nt][1][e] = 0.f;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        uint32_t w0[kPair][4], w1[kPair][4];
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          lds128(kp + k * kPageBytes + chunk_off<D>(tok0, qd + 4 * j), w0[k]);
          lds128(kp + k * kPageBytes + chunk_off<D>(tok0 + 8, qd + 4 * j), w1[k]);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int k = 0; k < kPair; ++k) {
            uint32_t a[4];
            q8::halves4(w0[k][e], a[0], a[2]);
            q8::halves4(w1[k][e], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              mma_f16(s[k][nt][e & 1], a, qb[0][nt][j * 4 + e][0], qb[0][nt][j * 4 + e][1]);
              if constexpr (kP == 2)
                mma_f16(s[k][nt][e & 1], a, qb[kP - 1][nt][j * 4 + e][0], qb[kP - 1][nt][j * 4 + e][1]);
            }
          }
      }
      // ---- online softmax (base 2) per head --------------------------------------
      uint32_t pb[kP][kPair][kNT][2];
      bool resc = false;
      float alpha[kNT][2];
#pragma unroll
      for (int nt = 0; nt < kNT; ++nt) {
        float z[kPair][4];
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          const float f[2] = {hs[nt][0] * ks[k], hs[nt][1] * ks[k]};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s[k][nt][0][e] += s[k][nt][1][e];
            z[k][e] = fmaf(s[k][nt][0][e], f[e & 1], ev[k]);
          }
        }
        if (!whole) {
#pragma unroll
          for (int k = 0; k < kPair; ++k) {
            if (!(tok0 < hi[k] && tok0 >= lo[k])) z[k][0] = z[k][1] = -INFINITY;
            if (!(tok0 + 8 < hi[k] && tok0 + 8 >= lo[k])) z[k][2] = z[k][3] = -INFINITY;
          }
        }
        float pm[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          pm[c] = fmaxf(z[0][c], z[0][c + 2]);
#pragma unroll
          for (int k = 1; k < kPair; ++k) pm[c] = fmaxf(pm[c], fmaxf(z[k][c], z[k][c + 2]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          pm[0] = fmaxf(pm[0], __shfl_xor_sync(0xffffffffu, pm[0], o));
          pm[1] = fmaxf(pm[1], __shfl_xor_sync(0xffffffffu, pm[1], o));
        }
        // the reference moves only when a step passes it by more than the lag
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float top = kP == 2 ? rintf(pm[c] - kTop<T>) : pm[c] - kTop<T>;
          const bool up = top - m_run[nt][c] > kLag<T>;
          alpha[nt][c] = up ? ex2_approx(m_run[nt][c] - top) : 1.f;
          m_run[nt][c] = up ? top : m_run[nt][c];
          resc |= up;
        }
        float sum[2] = {l_run[nt][0] * alpha[nt][0], l_run[nt][1] * alpha[nt][1]};
#pragma unroll
        for (int k = 0; k < kPair; ++k) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = z[k][e] - m_run[nt][e & 1];
            if constexpr (kP == 2) {
              // not through z, whose rounding is that of a large exponent
              const float f = hs[nt][e & 1] * ks[k], y = s[k][nt][0][e];
              const float fine = fmaf(y, f * p.scale_log2_low, fmaf(y, f, ev[k] - m_run[nt][e & 1]));
              x = z[k][e] == -INFINITY ? -INFINITY : fine;
            }
            w[e] = ex2_approx(x);
          }
          sum[0] = fmaf(w[0] + w[2], inv_vs[k], sum[0]);
          sum[1] = fmaf(w[1] + w[3], inv_vs[k], sum[1]);
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
      if (__any_sync(0xffffffffu, resc)) {
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int mt = 0; mt < kMT; ++mt) {
            acc[nt][mt][0] *= alpha[nt][0];
            acc[nt][mt][1] *= alpha[nt][1];
            acc[nt][mt][2] *= alpha[nt][0];
            acc[nt][mt][3] *= alpha[nt][1];
          }
      }
      // ---- O^T += V^T P^T ------------------------------------------------------------
      if (!whole) {
        // codes of masked tokens may be NaN: zero their rows of V
#pragma unroll 1
        for (int i = lane; i < kPair * kPageBytes / 16; i += 32) {
          const int k = i / (kPageBytes / 16), t = i % (kPageBytes / 16) / (D / 16);
          if (t >= hi[k] || t < lo[k])
            *reinterpret_cast<uint4*>(ring + st * Lay::kStageBytes + kPair * kPageBytes + i * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();  // before a later page's copy into this stage
        __syncwarp();
      }
#pragma unroll
      for (int c = 0; c < kMT; c += 2) {
        uint32_t r[kPair][4];
#pragma unroll
        for (int k = 0; k < kPair; ++k)
          ldsm_x4_trans(vp + k * kPageBytes + chunk_off<D>(v_tok, c + v_chunk), r[k]);
#pragma unroll
        for (int k = 0; k < kPair; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a[4];
            // bytes (t0 d0, t0 d1, t1 d0, t1 d1) -> (t0 d0, t1 d0 | t0 d1, t1 d1)
            q8::halves4(__byte_perm(r[k][2 * i], 0u, 0x3120), a[0], a[1]);
            q8::halves4(__byte_perm(r[k][2 * i + 1], 0u, 0x3120), a[2], a[3]);
#pragma unroll
            for (int nt = 0; nt < kNT; ++nt) {
              mma_f16(acc[nt][c + i], a, pb[0][k][nt][0], pb[0][k][nt][1]);
              if constexpr (kP == 2) mma_f16(acc[nt][c + i], a, pb[kP - 1][k][nt][0], pb[kP - 1][k][nt][1]);
            }
          }
      }
    }
    // ---- item end ------------------------------------------------------------------
    c_page += kPair;
    if (c_page >= c_end) {
      const ItemDesc& d = ws.items[cons_items % kRing];
      const bool split = d.nsplit > 1;
      bool last = false;  // the partial before this one completed its row
      if (split && pending) last = count(ws.pend[pend_at]);
      if (!aborted) {
        // this lane's elements of a head: dims 16 mt + 2 grp and the next
        const int64_t base = split ? (int64_t)d.slot * Hq + d.h0 : (int64_t)d.token * Hq + d.h0;
#pragma unroll
        for (int nt = 0; nt < kNT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float l = l_run[nt][c];
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            const int h = nt * 8 + 2 * qd + c;
            if (h < d.heads) {
              if (!split) {
                const float inv = 1.f / l;
                T* row = static_cast<T*>(p.out) + (base + h) * D + 2 * grp;
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) store2(row + 16 * mt, acc[nt][mt][c] * inv, acc[nt][mt][c + 2] * inv);
              } else {
                float* row = p.part_acc + (base + h) * D + 2 * grp;
#pragma unroll
                for (int mt = 0; mt < kMT; ++mt) store2(row + 16 * mt, acc[nt][mt][c], acc[nt][mt][c + 2]);
                if (grp == 0) *reinterpret_cast<float2*>(p.part_ml + (base + h) * 2) = make_float2(m_run[nt][c], l);
              }
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
      ++cons_items;
      reset();  // nothing of the item outlives the call above
    }
    __syncwarp();
    produce(st);
    st = (st + 1 == kStages) ? 0 : st + 1;
  }

  // count the last partial; after an abort also every split this warp started
  // but did not finish and every one still dealt to it
  if (pending && count(ws.pend[pend_at])) merge(ws.pend[pend_at]);
  if (aborted) {
    for (int k = cons_items; k < prod_items; ++k) {
      const ItemDesc& d = ws.items[k % kRing];
      if (d.nsplit > 1) count(d);
    }
    while (next_item()) {
      const ItemDesc d = ws.items[(prod_items - 1) % kRing];
      if (d.nsplit > 1) count(d);
      __syncwarp();  // before a later item takes its place
    }
  }
  // beside the prefill grid before it: this grid completes only after it
  if (p.pdl_mode == 2 && blockIdx.x == 0 && threadIdx.x == 0)
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace decode_q8
}  // namespace cb
