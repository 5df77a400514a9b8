// cb_rope: rotary positions of q and k, and cb_rope_plan_init.
//
// One pass over q and k: each element is read once and written once, so HBM
// bounds it (at small token counts, the launch).  A CTA takes a few tokens:
// its threads compute the tokens' cosines and sines once into shared memory
// -- the only work per (token, pair), shared by every head of q and k -- and
// then move vectors of 16 bytes.  In the half layout a thread owns the two
// vectors that hold the two halves of 8 (bf16) or 4 (f32) pairs; in the
// interleaved one a vector holds whole pairs, and a thread owns two that lie
// half a row apart (one vector to a thread: 51.2 us where it takes 47.2
// below).  The first vectors are loaded before the angles are computed, so
// their latencies overlap.
// Measured on the GPU alone, bf16, 128 dims: 8192 tokens of 64 + 8 heads 47.2
// us interleaved with half of the dims rotated (6.4 TB/s, 96% of the measured
// copy rate; every element, rotated or not, is read and written), 47.8 in the
// half layout and 49.1 interleaved with all rotated; 64 tokens of 32 + 8
// heads 2.5 us; float32, 4096 tokens of 64 + 8 heads 47.5 us in either layout.
#include <cuda_runtime.h>

#include <cmath>

#include "cb_error.h"
#include "launch_common.h"
#include "rope.cuh"
#include "rope.h"

namespace cb {
namespace rope {

constexpr int kThreads = 256;

struct Params {
  cb_rope_plan plan;
  Rows rows;
  const int32_t* positions;
  int32_t num_tokens, tokens_per_cta;
  int32_t inverse;
};

template <typename T, int N, bool kHalf>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Params p) {
  extern __shared__ float2 cs[];  // [tokens_per_cta][rot_dim / 2]
  const int t0 = (int)blockIdx.x * p.tokens_per_cta;
  const int tokens = min(p.tokens_per_cta, p.num_tokens - t0);
  rotate_rows<T, N, kHalf, kThreads>(p.rows, p.plan, p.positions, t0, tokens, p.inverse != 0, cs);
}

template <typename T, int N, bool kHalf>
cb_status launch(Params& p, cudaStream_t stream) {
  Rows& r = p.rows;
  cut_rows(&r, N, kHalf);
  // tokens per CTA: one while the tokens fit the SMs' resident CTAs once
  // (latency: 64 tokens 2.5 us, 3.8 with four; 608 3.3 and 4.0), then four, so
  // that a CTA's loads cover its set-up (2048 tokens 10.3 us with one, 9.2)
  p.tokens_per_cta = p.num_tokens <= 8 * sm_count_current_device() ? 1 : 4;
  const uint64_t items = (uint64_t)p.tokens_per_cta * r.heads * r.units;
  if (items * (uint64_t)(r.units > r.heads ? r.units : r.heads) >= 0x100000000ull)
    return fail(CB_ERR_UNSUPPORTED, "cb_rope: %d heads of %d dims", r.heads, r.head_dim);
  const int64_t ctas = ((int64_t)p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta;
  const size_t smem = (size_t)p.tokens_per_cta * (r.rot_dim / 2) * sizeof(float2);
  rope_kernel<T, N, kHalf><<<(unsigned)ctas, kThreads, smem, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "cb_rope launch: %s", cudaGetErrorString(e));
  return CB_OK;
}

template <typename T>
cb_status dispatch(Params& p, cudaStream_t stream) {
  constexpr int N = Vec<T>::kN;
  const int D = p.plan.head_dim, rot = p.plan.rot_dim;
  const bool half = p.plan.layout == CB_ROPE_HALF;
  // vectors fit when rows, strides and pointers are multiples of 16 bytes
  // and the rotated part splits into whole vectors (of each half)
  const Rows& r = p.rows;
  uintptr_t al = 0;
  int64_t lengths = D | (half ? rot / 2 : rot);
  if (r.hq) {
    al |= (uintptr_t)r.q | (uintptr_t)r.q_out;
    lengths |= r.q_stride | r.q_out_stride;
  }
  if (r.heads > r.hq) {
    al |= (uintptr_t)r.k | (uintptr_t)r.k_out;
    lengths |= r.k_stride | r.k_out_stride;
  }
  const bool vec = (al & 15u) == 0 && lengths % N == 0;
  if (vec) return half ? launch<T, N, true>(p, stream) : launch<T, N, false>(p, stream);
  return half ? launch<T, 1, true>(p, stream) : launch<T, 1, false>(p, stream);
}

}  // namespace rope

cb_status check_rope_plan(const cb_rope_plan* plan, int head_dim, const char* what) {
  if (!plan) return fail(CB_ERR_INVALID_ARG, "%s: plan is NULL", what);
  if (plan->head_dim <= 0 || plan->rot_dim < 2 || plan->rot_dim % 2 != 0 ||
      plan->rot_dim > plan->head_dim || plan->rot_dim > 2 * CB_ROPE_MAX_PAIRS ||
      (plan->layout != CB_ROPE_HALF && plan->layout != CB_ROPE_INTERLEAVED))
    return fail(CB_ERR_INVALID_ARG, "%s: the rotary plan's dims or layout are out of range", what);
  if (head_dim > 0 && plan->head_dim != head_dim)
    return fail(CB_ERR_INVALID_ARG, "%s: the rotary plan is for heads of %d dims, not %d", what,
                plan->head_dim, head_dim);
  return CB_OK;
}

}  // namespace cb

extern "C" cb_status cb_rope_plan_init(const cb_rope_config* config, cb_rope_plan* plan) {
  using cb::fail;
  if (!config || !plan) return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: NULL pointer");
  const cb_rope_config& c = *config;
  cb_rope_plan out{};
  out.head_dim = c.head_dim;
  out.rot_dim = c.rot_dim;
  out.layout = c.layout;
  cb_status st = cb::check_rope_plan(&out, 0, "cb_rope_plan_init");
  if (st != CB_OK) return st;
  if (c.scaling < CB_ROPE_NONE || c.scaling > CB_ROPE_BANDS)
    return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: unknown scaling %d", c.scaling);
  if (!(c.base > 1.0) || !std::isfinite(c.base))
    return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: base must be > 1");
  if (c.scaling != CB_ROPE_NONE && (!(c.factor >= 1.0) || !std::isfinite(c.factor)))
    return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: factor must be >= 1");
  const bool parts = c.scaling == CB_ROPE_PARTS, bands = c.scaling == CB_ROPE_BANDS;
  if ((parts || bands) && (!(c.original_positions >= 1.0) || !std::isfinite(c.original_positions)))
    return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: original_positions must be >= 1");
  if (parts && !(c.beta_slow > 0.0 && c.beta_fast > c.beta_slow && std::isfinite(c.beta_fast)))
    return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: beta_fast > beta_slow > 0 is wanted");
  if (bands && !(c.low_freq_factor > 0.0 && c.high_freq_factor > c.low_freq_factor &&
                 std::isfinite(c.high_freq_factor)))
    return fail(CB_ERR_INVALID_ARG,
                "cb_rope_plan_init: high_freq_factor > low_freq_factor > 0 is wanted");
  if (c.scaling == CB_ROPE_NTK && c.rot_dim == 2)
    return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: the base cannot be scaled with one pair");
  if (!(c.amplitude >= 0.0) || !std::isfinite(c.amplitude))
    return fail(CB_ERR_INVALID_ARG, "cb_rope_plan_init: amplitude must be >= 0");
  const double two_pi = 6.283185307179586476925;
  const double rot = c.rot_dim;
  double base = c.base;
  if (c.scaling == CB_ROPE_NTK) base *= std::pow(c.factor, rot / (rot - 2.0));
  double lo = 0.0, hi = 0.0;
  if (parts) {
    auto at = [&](double n) {
      return rot * std::log(c.original_positions / (two_pi * n)) / (2.0 * std::log(base));
    };
    lo = std::fmax(std::floor(at(c.beta_fast)), 0.0);
    // (rot - 1, not the last pair's rot / 2 - 1: a ramp that reaches past the
    // pairs keeps its slope)
    hi = std::fmin(std::ceil(at(c.beta_slow)), rot - 1);
    if (hi < lo)
      return fail(CB_ERR_INVALID_ARG,
                  "cb_rope_plan_init: the ramp would end (%.0f) before it starts (%.0f): original_positions "
                  "does not go with base and betas", hi, lo);
    if (hi == lo) hi = lo + 0.001;
  }
  double amplitude = parts && c.factor > 1.0 ? 0.1 * std::log(c.factor) + 1.0 : 1.0;
  if (c.amplitude > 0.0) amplitude = c.amplitude;
  out.amplitude = (float)amplitude;
  for (int i = 0; i < c.rot_dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / rot);
    if (c.scaling == CB_ROPE_LINEAR) f /= c.factor;
    if (parts || bands) {
      double k = parts ? 1.0 - (i - lo) / (hi - lo)
                       : (c.original_positions * f / two_pi - c.low_freq_factor) /
                             (c.high_freq_factor - c.low_freq_factor);
      k = std::fmin(std::fmax(k, 0.0), 1.0);
      f *= k + (1.0 - k) / c.factor;
    }
    out.turns[i] = (uint64_t)(std::ldexp(f / two_pi, 64) + 0.5);  // f <= 1: below 2^62
  }
  *plan = out;
  return CB_OK;
}

extern "C" cb_status cb_rope(const cb_rope_args* args, cb_stream_t stream) {
  using cb::fail;
  if (!args) return fail(CB_ERR_INVALID_ARG, "cb_rope: args is NULL");
  const cb_rope_args& a = *args;
  cb_status st = cb::check_rope_plan(a.plan, 0, "cb_rope");
  if (st != CB_OK) return st;
  if (a.num_tokens < 0 || (a.q && a.num_q_heads <= 0) || (a.k && a.num_kv_heads <= 0))
    return fail(CB_ERR_INVALID_ARG, "cb_rope: sizes must be positive");
  if (a.dtype != CB_DTYPE_F32 && a.dtype != CB_DTYPE_BF16)
    return fail(CB_ERR_INVALID_ARG, "cb_rope: unknown dtype");
  if (a.num_tokens == 0) return CB_OK;
  if (!a.q && !a.k) return fail(CB_ERR_INVALID_ARG, "cb_rope: neither q nor k is given");
  if (!a.positions || (a.q && !a.q_out) || (a.k && !a.k_out))
    return fail(CB_ERR_INVALID_ARG, "cb_rope: NULL pointer");
  if ((a.q && a.num_q_heads > (1 << 20)) || (a.k && a.num_kv_heads > (1 << 20)))
    return fail(CB_ERR_UNSUPPORTED, "cb_rope: more than 2^20 heads");
  cb::rope::Params p{};
  p.plan = *a.plan;
  p.positions = a.positions;
  p.num_tokens = a.num_tokens;
  p.inverse = a.inverse;
  cb::rope::Rows& r = p.rows;
  r.head_dim = p.plan.head_dim;
  r.rot_dim = p.plan.rot_dim;
  r.hq = a.q ? a.num_q_heads : 0;
  r.heads = r.hq + (a.k ? a.num_kv_heads : 0);
  const int64_t D = r.head_dim;
  auto stride = [&](int64_t s, int32_t heads) { return s ? s : heads * D; };
  r.q = a.q;
  r.q_out = a.q_out;
  r.k = a.k;
  r.k_out = a.k_out;
  r.q_stride = stride(a.q_stride, a.num_q_heads);
  r.q_out_stride = stride(a.q_out_stride, a.num_q_heads);
  r.k_stride = stride(a.k_stride, a.num_kv_heads);
  r.k_out_stride = stride(a.k_out_stride, a.num_kv_heads);
  if ((a.q && (r.q_stride < a.num_q_heads * D || r.q_out_stride < a.num_q_heads * D)) ||
      (a.k && (r.k_stride < a.num_kv_heads * D || r.k_out_stride < a.num_kv_heads * D)))
    return fail(CB_ERR_INVALID_ARG, "cb_rope: a stride is less than a token's heads");
  const uintptr_t elem = a.dtype == CB_DTYPE_F32 ? 4 : 2;
  if ((((uintptr_t)a.q | (uintptr_t)a.q_out | (uintptr_t)a.k | (uintptr_t)a.k_out) & (elem - 1)) != 0)
    return fail(CB_ERR_INVALID_ARG, "cb_rope: pointers must be aligned to their element");
  return a.dtype == CB_DTYPE_F32 ? cb::rope::dispatch<float>(p, (cudaStream_t)stream)
                                 : cb::rope::dispatch<__nv_bfloat16>(p, (cudaStream_t)stream);
}
