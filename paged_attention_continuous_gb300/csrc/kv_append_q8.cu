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
// (a block's largest value is met early, so few appends do).  The runs of a
// CTA's tokens are counted first and (run, head) dealt to the warps: dealt
// by token instead, some warps wrote two runs one after the other while
// others had none (the 6.9k tokens below took 14.9 us).
//
// With a rotary plan, k turns in registers before its magnitude is taken, a
// lane holding both elements of its pairs, and k is neither written nor read
// in between.  CTAs of their own rotate the tokens' q: with q after k in the
// same CTAs, or partners in two lanes and exchanged by shuffles, the call
// below took 48 us.
//
// Every new element is read once and every code written once; HBM bounds
// large calls and the launch with two dependent loads (slots, then the
// block's scale) small ones.  Measured on the GPU alone, bf16, 8 heads of
// 128: 6.9k tokens of 16 chunks 10.9 us (3.9 TB/s), 96 tokens with 32 heads
// of q turned 4.5 us, the 6.9k with 32 heads of q turned 33.8 us (4.6 TB/s);
// float32 17.7 us and 57.2 (5.2 TB/s).
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
constexpr int kPad = 8;         // angles left out behind a token's, so that rows side by side read other banks
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
  // CTAs of the same tokens (grid y): kv_ctas for k, as many for v, and with
  // q one for every q_tokens tokens
  int32_t kv_ctas, q_tokens;
  rope::Rows q_rows;    // heads 0: no q
  uint32_t* error_word;
};

// The codes of N values, in one store.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* dst, const float (&x)[N], float f) {
  const uint32_t lo = q8::codes2(x[0] * f, x[1] * f) | (q8::codes2(x[2] * f, x[3] * f) << 16);
  if constexpr (N == 8)
    *reinterpret_cast<uint2*>(dst) =
        make_uint2(lo, q8::codes2(x[4] * f, x[5] * f) | (q8::codes2(x[6] * f, x[7] * f) << 16));
  else
    *reinterpret_cast<uint32_t*>(dst) = lo;
}

// CTAs an SM should hold: four, where the registers of a run allow it (the
// 6.9k tokens with q turned 35.9 us with four, 37.9 with three, before runs
// were dealt to warps).  float32 runs take twice the registers of bfloat16
// ones.  The 6.9k tokens in float32 with 1 / 2 / 3 CTAs: 128 dims 17.5 / 17.7
// / 18.0 us, with q and k turned 62.1 / 62.0 / 56.8; 64 dims 9.8 / 9.7 / 9.7,
// and 8.3 with four, turned 36.8 / 36.8 / 30.5.
template <typename T, int D, int kRope>
constexpr int resident() { return sizeof(T) == 2 ? 4 : kRope != kNoRope ? 3 : D == 64 ? 4 : 2; }

template <typename T, int D, int kRope>
__global__ void __launch_bounds__(kThreads, resident<T, D, kRope>())
    append_kernel(const __grid_constant__ Params p) {
  constexpr int N = Vec<T>::kN;              // elements of a vector; a lane holds two of a row
  constexpr int kLanes = D / N / 2;          // lanes of a row
  constexpr int kRows = 32 / kLanes;         // rows of a warp at once
  constexpr int kSteps = q8::kPage / kRows;  // steps of a full block
  // slots of this CTA's tokens, of the one before and of those a run that
  // starts here can reach
  __shared__ int32_t slots[1 + kMaxTokens + q8::kPage];
  extern __shared__ float2 cs[];             // [tokens_per_cta + 15][rot_dim / 2 + kPad]
  // the attention launch that follows (when it asks for it) may start now;
  // it reads the cache only after this grid has completed
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t0 = (int)blockIdx.x * p.tokens_per_cta;
  if constexpr (kRope != kNoRope) {
    if ((int)blockIdx.y >= 2 * p.kv_ctas) {
      const int q0 = t0 + ((int)blockIdx.y - 2 * p.kv_ctas) * p.q_tokens;
      if (q0 < p.num_tokens)
        rope::rotate_rows<T, Vec<T>::kN, kRope == kHalf, kThreads>(
            p.q_rows, p.plan, p.positions, q0, min(p.q_tokens, p.num_tokens - q0), false, cs);
      return;
    }
  }
  const bool is_v = (int)blockIdx.y >= p.kv_ctas;
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
  __syncthreads();
  // the runs that start at this CTA's tokens: lane i looks at the i-th token
  const int tokens = min(p.tokens_per_cta, p.num_tokens - t0);
  bool starts = false;
  if (lane < tokens) {
    const int slot = slots[1 + lane], before = slots[lane];
    const bool inside = slot % q8::kPage != 0 && before == slot - 1;
    starts = slot >= 0 && !inside;
    if (starts && before >= 0 && before / q8::kPage == slot / q8::kPage) {  // neighbours out of order
      set_error(p.error_word, CB_DEVERR_SLOT_ORDER);
      starts = false;
    }
  }
  const uint32_t run_starts = __ballot_sync(0xffffffffu, starts);
  const int nth = __popc(run_starts & ((1u << lane) - 1u));  // of the run that starts at the lane's token
  // tasks (run, head), dealt over the warps of the CTAs that share these tokens
  const int Hkv = p.num_kv_heads;
  const int num_tasks = __popc(run_starts) * Hkv;
  const int worker0 = ((int)blockIdx.y - (is_v ? p.kv_ctas : 0)) * kWarps;
  if (worker0 >= num_tasks) return;
  const int pairs = kRope == kNoRope ? 0 : p.plan.rot_dim / 2;
  const int angles = pairs + kPad;  // of a token
  if constexpr (kRope != kNoRope) {
    if (!is_v) {
      // angles of this CTA's tokens, and of the tokens behind them that
      // belong to its last run
      const int last = slots[p.tokens_per_cta];
      for (int i = threadIdx.x; i < reach * pairs; i += kThreads) {
        const int tl = i / pairs, t = t0 + tl;
        if (t >= p.num_tokens) break;
        const int over = tl - (p.tokens_per_cta - 1);
        if (over > 0 && (last < 0 || (last & 15) + over > 15 || slots[1 + tl] != last + over)) continue;
        const int pair = i - tl * pairs;
        cs[tl * angles + rope::angle_at<N, kRope == kHalf>(pair, pairs)] =
            rope::turn_of(p.plan.turns[pair], p.positions[t], p.plan.amplitude, false);
      }
      __syncthreads();
    }
  }

  // The lane's vectors of a row, at elements a and b: two halves of a row,
  // or for k in the half layout a vector of first elements and that of their
  // partners, then (where the row is not turned) two neighbours.
  const int sub = lane / kLanes, j = lane - sub * kLanes;
  int a = j * N, b = a + D / 2;
  if (kRope == kHalf && !is_v) {
    b = a + pairs;
    if (a >= pairs) {
      a += a;
      b = a + N;
    }
  }
  const int64_t row_stride = (int64_t)Hkv * D;
  for (int task = worker0 + warp; task < num_tasks; task += p.kv_ctas * kWarps) {
    const int run = task / Hkv, h = task - run * Hkv;
    const int tl = __ffs(__ballot_sync(0xffffffffu, starts && nth == run)) - 1;
    const int slot = slots[1 + tl];
    const int off = slot & (q8::kPage - 1), block = slot >> 4;
    // tokens of the run: lane i looks at the i-th slot
    const bool follows = lane < q8::kPage - off && slots[1 + tl + (lane < q8::kPage ? lane : 0)] == slot + lane;
    const int count = __ffs(~__ballot_sync(0xffffffffu, follows)) - 1;
    const T* src = static_cast<const T*>(is_v ? p.v_new : p.k_new) + (t0 + tl) * row_stride + h * D;
    uint8_t* scale = (is_v ? p.v_scales : p.k_scales) + (int64_t)block * p.scale_stride + h;
    const int was = off > 0 ? q8::exp_of(*scale) : q8::kMinExp;
    uint4 raw[kSteps][2];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int row = i * kRows + sub;
      const T* r = src + row * row_stride;
      raw[i][0] = row < count ? __ldg(reinterpret_cast<const uint4*>(r + a)) : make_uint4(0, 0, 0, 0);
      raw[i][1] = row < count ? __ldg(reinterpret_cast<const uint4*>(r + b)) : make_uint4(0, 0, 0, 0);
    }
    // the values are unpacked (and turned) twice, for their largest magnitude
    // and for their codes: kept in between, they would take twice the
    // registers of the raw ones, and fewer CTAs would fit an SM
    auto values = [&](int i, float* x, float* y) {
      Vec<T>::load(raw[i][0], x);
      Vec<T>::load(raw[i][1], y);
      if constexpr (kRope != kNoRope) {
        if (!is_v) {
          const float2* c = cs + (tl + min(i * kRows + sub, count - 1)) * angles + j;
          const int stride = pairs / rope::unit_pairs<N, kRope == kHalf>();
          if constexpr (kRope == kHalf) {
            if (j < stride) {
#pragma unroll
              for (int e = 0; e < N; ++e) rope::rotate(x[e], y[e], c[e * stride]);
            }
          } else {
            if (j < stride) {
#pragma unroll
              for (int e = 0; e < N; e += 2) rope::rotate(x[e], x[e + 1], c[e / 2 * stride]);
            }
            if (j + kLanes < stride) {
#pragma unroll
              for (int e = 0; e < N; e += 2) rope::rotate(y[e], y[e + 1], c[e / 2 * stride + kLanes]);
            }
          }
        }
      }
    };
    // the largest finite magnitude: fmaxf passes over NaN, and infinities
    // are rare enough for a second look at all values
    auto largest = [&](float above) {
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        if (i * kRows < count) {
          float x[N], y[N];
          values(i, x, y);
#pragma unroll
          for (int e = 0; e < N; ++e) {
            const float m = fabsf(x[e]), n = fabsf(y[e]);
            if (above > 0.f) {
              amax = m < above ? fmaxf(amax, m) : amax;
              amax = n < above ? fmaxf(amax, n) : amax;
            } else {
              amax = fmaxf(amax, fmaxf(m, n));
            }
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      return amax;
    };
    float amax = largest(0.f);
    if (isinf(amax)) amax = largest(amax);
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
        float x[N], y[N];
        values(i, x, y);
        const int row = i * kRows + sub;
        uint8_t* dst = page + (off + row) * D;
        if (row < count) {
          store_codes(dst + a, x, f);
          store_codes(dst + b, y, f);
        }
      }
    }
    if (lane == 0) *scale = (uint8_t)(e + 127);
  }
}

template <typename T, int D, int kRope>
cb_status launch(Params& p, cudaStream_t stream) {
  if constexpr (kRope != kNoRope) {
    rope::Rows& r = p.q_rows;
    if (r.heads > 0) {
      rope::cut_rows(&r, Vec<T>::kN, kRope == kHalf);
      const uint64_t items = (uint64_t)std::min(p.tokens_per_cta, 4) * r.heads * r.units;
      if (items * (uint64_t)(r.units > r.heads ? r.units : r.heads) >= 0x100000000ull)
        return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q8: %d query heads", r.heads);
    }
  }
  const int64_t ctas = ((int64_t)p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta;
  const size_t smem =
      kRope == kNoRope ? 0 : (size_t)(p.tokens_per_cta + q8::kPage - 1) * (p.plan.rot_dim / 2 + kPad) * sizeof(float2);
  // a warp for every head of a run, so that its heads are written side by
  // side; 16 tokens mostly hold the starts of one or two runs
  p.kv_ctas = std::min(std::max(p.num_kv_heads * (p.tokens_per_cta > 1 ? 2 : 1) / kWarps, 1), 16);
  p.q_tokens = std::min(p.tokens_per_cta, 4);
  const int q_ctas = p.q_rows.heads > 0 ? p.tokens_per_cta / p.q_tokens : 0;
  append_kernel<T, D, kRope><<<dim3((unsigned)ctas, (unsigned)(2 * p.kv_ctas + q_ctas)), kThreads, smem, stream>>>(p);
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
  // Decode steps bring runs of one token and want a warp for each, chunks
  // runs of 16 whose other tokens leave warps idle; the call cannot tell them
  // apart.  96 decodes take 4.5 / 6.0 / 16.4 us with 1 / 4 / 16 tokens to a CTA,
  // 600 10.0 / 9.7 / 16.6, 1024 16.2 / 14.8 / 21.2, 2048 32.0 / 28.2 / 27.9; a
  // chunk of 600 tokens 4.6 / 4.1 / 3.1, four of 500 8.1 / 6.1 / 4.5.
  p.tokens_per_cta = a.num_tokens <= 256 ? 1 : a.num_tokens <= 1024 ? 4 : kMaxTokens;
  const bool f32 = a.dtype == CB_DTYPE_F32;
  const cudaStream_t s = (cudaStream_t)stream;
  if (a.head_dim == 64)
    return f32 ? dispatch<float, 64>(p, a.rope, s) : dispatch<__nv_bfloat16, 64>(p, a.rope, s);
  return f32 ? dispatch<float, 128>(p, a.rope, s) : dispatch<__nv_bfloat16, 128>(p, a.rope, s);
}
