// cb_kv_append_q8: a step's new K/V into the cache of e4m3 codes with one
// power-of-two scale for each (block, KV head).
//
// "vLLM serving internals", PagedAttention as a virtual memory system: token
// t goes to block slot / 16, offset slot % 16.  Here the tokens of one block
// share a scale, so they are written together: a RUN is a maximal sequence
// of neighbouring tokens at neighbouring slots of one block (1 to 16
// tokens), found by its first token.  One warp writes one run for one head
// of K or V: it holds the run's values in registers, takes their largest
// magnitude, derives the exponent, and writes codes.  The block's old scale
// is read beside the values; the old codes only if that scale has to grow
// (a block's largest value is met early, so few appends do).
//
// With a rotary plan, k turns in registers before its magnitude is taken,
// and the same CTA rotates its tokens' q: the angles of a token are computed
// once for all heads, and k is neither written nor read in between.
//
// Every new element is read once and every code written once; HBM bounds
// large calls and the launch with two dependent loads (slots, then the
// block's scale) small ones.
#include <cuda_runtime.h>

#include <algorithm>

#include "cb_error.h"
#include "launch_common.h"
#include "q8.cuh"
#include "rope.cuh"
#include "rope.h"
#include "validate.h"

namespace cb {
namespace append_q8 {

using rope::Vec;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxTokens = 16;  // tokens of a CTA
enum { kNoRope = -1, kHalf = CB_ROPE_HALF, kInterleaved = CB_ROPE_INTERLEAVED };

struct Params {
  cb_rope_plan plan;
  const void* k_new;
  const void* v_new;
  const int32_t* slot_mapping;
  const int32_t* positions;
  uint8_t* k_cache;
  uint8_t* v_cache;
  uint8_t* k_scales;
  uint8_t* v_scales;
  int64_t scale_stride;
  int64_t num_slots;
  int32_t num_tokens, tokens_per_cta;
  int32_t num_kv_heads;
  rope::Rows q_rows;    // heads 0: no q
  uint32_t* error_word;
};

// Rotate one lane's N elements of a row of D (element offset `at`), whose
// partners in the half layout lie in lane `at` +- rot / 2 of the same row.
// cs: the token's angles as rope::angle_at has them.
template <int kRope, int N>
__device__ __forceinline__ void rotate_lane(float* x, int at, int rot, int lane, const float2* cs) {
  constexpr int kPairs = rope::unit_pairs<N, kRope == kHalf>();
  const int stride = rot / 2 / kPairs;
  if constexpr (kRope == kHalf) {
    const int half = rot / 2;
    const bool lo = at < half, in = at < rot;
    const int partner = lane + (in ? (lo ? half : -half) / N : 0);
    const float2* c = cs + (in ? (lo ? at : at - half) / N : 0);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y = __shfl_sync(0xffffffffu, x[i], partner);
      if (in) {
        float a = lo ? x[i] : y, b = lo ? y : x[i];
        rope::rotate(a, b, c[i * stride]);
        x[i] = lo ? a : b;
      }
    }
  } else {
    if (at < rot) {
#pragma unroll
      for (int i = 0; i < N; i += 2) rope::rotate(x[i], x[i + 1], cs[at / N + i / 2 * stride]);
    }
  }
}

template <typename T, int D, int kRope>
__global__ void __launch_bounds__(kThreads, D * sizeof(T) == 512 ? 2 : kRope == kNoRope ? 4 : 3)
    append_kernel(const __grid_constant__ Params p) {
  constexpr int N = Vec<T>::kN;             // elements of a lane
  constexpr int kLanes = D / N;             // lanes of a row
  constexpr int kRows = 32 / kLanes;        // rows of a warp at once
  constexpr int kSteps = q8::kPage / kRows; // steps of a full block
  static_assert(kLanes <= 32, "a row must fit a warp");
  // slots of this CTA's tokens, of the one before and of those a run that
  // starts here can reach
  __shared__ int32_t slots[1 + kMaxTokens + q8::kPage];
  extern __shared__ float2 cs[];            // [tokens_per_cta + 15][rot_dim / 2]
  // the attention launch that follows (when it asks for it) may start now;
  // it reads the cache only after this grid has completed
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t0 = (int)blockIdx.x * p.tokens_per_cta;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int reach = p.tokens_per_cta + q8::kPage - 1;
  if (threadIdx.x < reach + 1) {
    const int t = t0 - 1 + (int)threadIdx.x;
    int s = t >= 0 && t < p.num_tokens ? p.slot_mapping[t] : -1;
    if (s >= 0 && s >= p.num_slots) {
      // the token's own CTA reports it; for everybody it is padding
      if (threadIdx.x >= 1 && threadIdx.x <= p.tokens_per_cta) set_error(p.error_word, CB_DEVERR_SLOT_RANGE);
      s = -1;
    }
    slots[threadIdx.x] = s;
  }
  const int rot = kRope == kNoRope ? 0 : p.plan.rot_dim;
  const int pairs = rot / 2;
  __syncthreads();
  if constexpr (kRope != kNoRope) {
    // angles of this CTA's tokens, and of the tokens behind them that belong
    // to its last run
    const int last = slots[p.tokens_per_cta];
    for (int i = threadIdx.x; i < reach * pairs; i += kThreads) {
      const int tl = i / pairs, t = t0 + tl;
      if (t >= p.num_tokens) break;
      const int over = tl - (p.tokens_per_cta - 1);
      if (over > 0 && (last < 0 || (last & 15) + over > 15 || slots[1 + tl] != last + over)) continue;
      const int pair = i - tl * pairs;
      cs[tl * pairs + rope::angle_at<N, kRope == kHalf>(pair, pairs)] =
          rope::turn_of(p.plan.turns[pair], p.positions[t], p.plan.amplitude, false);
    }
    __syncthreads();
  }

  const int sub = lane / kLanes, at = (lane - sub * kLanes) * N;  // row of a step, element offset
  const int Hkv = p.num_kv_heads;
  const int tokens = min(p.tokens_per_cta, p.num_tokens - t0);
  // tasks (token, head of K or V), dealt over the warps of the CTAs that
  // share these tokens
  const int worker = (int)blockIdx.y * kWarps + warp, workers = (int)gridDim.y * kWarps;
  for (int task = worker; task < tokens * Hkv * 2; task += workers) {
    const int tl = task / (Hkv * 2), w = task - tl * (Hkv * 2);
    const int slot = slots[1 + tl], before = slots[tl];
    if (slot < 0) continue;
    const int off = slot & (q8::kPage - 1), block = slot >> 4;
    if (off > 0 && before == slot - 1) continue;              // inside a run
    if (before >= 0 && (before >> 4) == block) {              // neighbours out of order
      if (w == 0 && lane == 0) set_error(p.error_word, CB_DEVERR_SLOT_ORDER);
      continue;
    }
    // tokens of the run: lane i looks at the i-th slot
    const bool follows = lane < q8::kPage - off && slots[1 + tl + (lane < q8::kPage ? lane : 0)] == slot + lane;
    const int count = __ffs(~__ballot_sync(0xffffffffu, follows)) - 1;
    const bool is_v = w >= Hkv;
    const int h = is_v ? w - Hkv : w;
    const T* src = static_cast<const T*>(is_v ? p.v_new : p.k_new) + ((int64_t)(t0 + tl) * Hkv + h) * D + at;
    uint8_t* scale = (is_v ? p.v_scales : p.k_scales) + (int64_t)block * p.scale_stride + h;
    const int was = off > 0 ? q8::exp_of(*scale) : q8::kMinExp;
    uint4 raw[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = i * kRows + sub;
      raw[i] = row < count ? __ldg(reinterpret_cast<const uint4*>(src + (int64_t)row * Hkv * D))
                           : make_uint4(0, 0, 0, 0);
    }
    // the values are unpacked (and turned) twice, for their largest magnitude
    // and for their codes: kept in between, they would take twice the
    // registers of the raw ones, and fewer CTAs would fit an SM
    auto values = [&](int i, float* x) {
      Vec<T>::load(raw[i], x);
      if constexpr (kRope != kNoRope) {
        if (!is_v) rotate_lane<kRope, N>(x, at, rot, lane, cs + (tl + min(i * kRows + sub, count - 1)) * pairs);
      }
    };
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i * kRows < count) {
        float x[N];
        values(i, x);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float m = fabsf(x[e]);
          amax = m <= 3.402823466e38f ? fmaxf(amax, m) : amax;  // not an infinity, not NaN
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const int e = max(q8::exp_for(amax), was);
    uint8_t* page = (is_v ? p.v_cache : p.k_cache) + ((int64_t)block * Hkv + h) * (q8::kPage * D);
    if (off > 0 && e > was) {
      // the codes before the run move to the larger scale
      uint4* old = reinterpret_cast<uint4*>(page);
      for (int i = lane; i < off * (D / 16); i += 32) {
        uint4 v = old[i];
        v.x = q8::shrink4(v.x, e - was);
        v.y = q8::shrink4(v.y, e - was);
        v.z = q8::shrink4(v.z, e - was);
        v.w = q8::shrink4(v.w, e - was);
        old[i] = v;
      }
    }
    const float f = q8::exp2i(-e);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      if (i * kRows < count) {
        float x[N];
        values(i, x);
        const int row = i * kRows + sub;
        uint8_t* dst = page + (off + row) * D + at;
        const uint32_t lo = q8::codes2(x[0] * f, x[1] * f) | (q8::codes2(x[2] * f, x[3] * f) << 16);
        if constexpr (N == 8) {
          const uint32_t hi = q8::codes2(x[4] * f, x[5] * f) | (q8::codes2(x[6] * f, x[7] * f) << 16);
          if (row < count) *reinterpret_cast<uint2*>(dst) = make_uint2(lo, hi);
        } else {
          if (row < count) *reinterpret_cast<uint32_t*>(dst) = lo;
        }
      }
    }
    if (lane == 0) *scale = (uint8_t)(e + 127);
  }

  if constexpr (kRope != kNoRope) {
    // q of this CTA's tokens, a unit of the rows to a thread
    constexpr int kAhead = 2;
    const uint32_t items = (uint32_t)tokens * p.q_rows.heads * p.q_rows.units;
    const uint32_t step = gridDim.y * kThreads;
    for (uint32_t n = blockIdx.y * kThreads + threadIdx.x; n < items; n += kAhead * step) {
      rope::Unit<T, N> w[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (n + i * step < items) rope::load_unit<T, N, kRope == kHalf>(p.q_rows, t0, n + i * step, w[i]);
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (n + i * step < items)
          rope::store_unit<T, N, kRope == kHalf>(cs, pairs / rope::unit_pairs<N, kRope == kHalf>(), w[i]);
    }
  }
}

template <typename T, int D, int kRope>
cb_status launch(Params& p, cudaStream_t stream) {
  if constexpr (kRope != kNoRope) {
    rope::Rows& r = p.q_rows;
    if (r.heads > 0) {
      rope::cut_rows(&r, Vec<T>::kN, kRope == kHalf);
      const uint64_t items = (uint64_t)p.tokens_per_cta * r.heads * r.units;
      if (items * (uint64_t)(r.units > r.heads ? r.units : r.heads) >= 0x100000000ull)
        return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q8: %d query heads", r.heads);
    }
  }
  const int64_t ctas = ((int64_t)p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta;
  const size_t smem = kRope == kNoRope ? 0
                                       : (size_t)(p.tokens_per_cta + q8::kPage - 1) * (p.plan.rot_dim / 2) * sizeof(float2);
  // CTAs that share the same tokens: one for every 8 (head of K or V)s, a warp
  // for each, so that a run's heads are written side by side
  const int share = std::min(std::max(p.num_kv_heads * 2 / kWarps, 1), 8);
  append_kernel<T, D, kRope><<<dim3((unsigned)ctas, (unsigned)share), kThreads, smem, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "cb_kv_append_q8 launch: %s", cudaGetErrorString(e));
  return CB_OK;
}

template <typename T, int D>
cb_status dispatch(Params& p, bool with_rope, cudaStream_t stream) {
  if (!with_rope) return launch<T, D, kNoRope>(p, stream);
  return p.plan.layout == CB_ROPE_HALF ? launch<T, D, kHalf>(p, stream)
                                       : launch<T, D, kInterleaved>(p, stream);
}

}  // namespace append_q8
}  // namespace cb

extern "C" cb_status cb_kv_append_q8(const cb_append_q8_args* args, cb_stream_t stream) {
  using cb::fail;
  using namespace cb::append_q8;
  if (!args) return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: args is NULL");
  const cb_append_q8_args& a = *args;
  if (a.num_tokens < 0 || a.num_blocks <= 0 || a.num_kv_heads <= 0 || a.head_dim <= 0 || a.block_size <= 0)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: sizes must be positive");
  if (a.dtype != CB_DTYPE_F32 && a.dtype != CB_DTYPE_BF16)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: unknown dtype");
  if (a.block_size != cb::q8::kPage) return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q8: block_size must be 16");
  if (a.head_dim != 64 && a.head_dim != 128)
    return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q8: head_dim must be 64 or 128");
  if (a.rope) {
    cb_status st = cb::check_rope_plan(a.rope, a.head_dim, "cb_kv_append_q8");
    if (st != CB_OK) return st;
    if (a.rope->rot_dim % 16 != 0)
      return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q8: rot_dim must be a multiple of 16");
    if (a.q && a.num_q_heads <= 0) return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: num_q_heads must be positive");
  } else if (a.q) {
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: q is rotated only with a rotary plan");
  }
  const int64_t stride = a.scale_stride ? a.scale_stride : a.num_kv_heads;
  if (stride < a.num_kv_heads)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: scale_stride is less than num_kv_heads");
  if (a.num_tokens == 0) return CB_OK;
  if (!a.k_new || !a.v_new || !a.slot_mapping || !a.k_cache || !a.v_cache || !a.k_scales || !a.v_scales ||
      (a.rope && !a.positions) || (a.q && !a.q_out))
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: NULL pointer");
  const uintptr_t align = (uintptr_t)a.k_new | (uintptr_t)a.v_new | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache |
                          (uintptr_t)a.q | (uintptr_t)a.q_out;
  if (align & 15u) return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q8: pointers must be 16-byte aligned");
  if ((int64_t)a.num_tokens * (a.num_kv_heads > a.num_q_heads ? a.num_kv_heads : a.num_q_heads) >= ((int64_t)1 << 31) ||
      a.num_kv_heads > (1 << 20) || a.num_q_heads > (1 << 20))
    return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q8: more than 2^31 rows in one call");
  if (cb::validate_enabled()) {
    cb_status vs = cb::validate_append_q8_call(a.slot_mapping, a.num_tokens, a.num_blocks, a.block_size,
                                               (cudaStream_t)stream);
    if (vs != CB_OK) return vs;
  }
  Params p{};
  if (a.rope) p.plan = *a.rope;
  p.k_new = a.k_new;
  p.v_new = a.v_new;
  p.slot_mapping = a.slot_mapping;
  p.positions = a.positions;
  p.k_cache = static_cast<uint8_t*>(a.k_cache);
  p.v_cache = static_cast<uint8_t*>(a.v_cache);
  p.k_scales = a.k_scales;
  p.v_scales = a.v_scales;
  p.scale_stride = stride;
  p.num_slots = (int64_t)a.num_blocks * a.block_size;
  p.num_tokens = a.num_tokens;
  p.num_kv_heads = a.num_kv_heads;
  if (a.q) {
    p.q_rows.head_dim = a.head_dim;
    p.q_rows.rot_dim = p.plan.rot_dim;
    p.q_rows.hq = p.q_rows.heads = a.num_q_heads;
    p.q_rows.q = a.q;
    p.q_rows.q_out = a.q_out;
    p.q_rows.q_stride = p.q_rows.q_out_stride = (int64_t)a.num_q_heads * a.head_dim;
  }
  p.error_word = a.error_word;
  p.tokens_per_cta = a.num_tokens <= 1024 ? 1 : kMaxTokens;
  const bool f32 = a.dtype == CB_DTYPE_F32;
  const cudaStream_t s = (cudaStream_t)stream;
  if (a.head_dim == 64)
    return f32 ? dispatch<float, 64>(p, a.rope, s) : dispatch<__nv_bfloat16, 64>(p, a.rope, s);
  return f32 ? dispatch<float, 128>(p, a.rope, s) : dispatch<__nv_bfloat16, 128>(p, a.rope, s);
}
