// cb_rope: rotary positions of q and k, and cb_rope_plan_init.
//
// One pass over q and k: each element is read once and written once, so HBM
// bounds it (at small token counts, the launch).  A CTA takes a few tokens:
// its threads compute the tokens' cosines and sines once into shared memory
// -- the only work per (token, pair), shared by every head of q and k -- and
// then move vectors of 16 bytes.  In the half layout a thread owns the two
// vectors that hold the two halves of 8 (bf16) or 4 (f32) pairs; in the
// interleaved one a vector holds whole pairs.  The first vectors are loaded
// before the angles are computed, so their latencies overlap.
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
  const int32_t* positions;
  int32_t num_tokens, tokens_per_cta;
  int32_t hq, heads;            // heads of q (0 without q), of q and k together
  int32_t units;                // work units of one head row
  int32_t rot_units;            // the first rot_units of them rotate, the rest copy
  uint32_t units_magic, heads_magic;  // ceil(2^32 / x)
  int32_t inverse;
  const void* q;
  void* q_out;
  const void* k;
  void* k_out;
  int64_t q_stride, q_out_stride, k_stride, k_out_stride;  // elements
};

// n / d for n d < 2^32, magic = ceil(2^32 / d) (0 for d = 1)
__device__ __forceinline__ uint32_t div_by(uint32_t n, uint32_t magic) {
  return magic ? __umulhi(n, magic) : n;
}

// A unit of work: N elements at `a`, and their partners at `b` when it
// rotates in the half layout (or N = 1, for rows that vectors do not fit: one
// pair, or one element to copy).  pair < 0: a unit that is only copied.
template <typename T, int N>
struct Unit {
  const T* in;
  T* out;
  int a, b, pair;
  float x[N], y[N];
};

template <typename T, int N, bool kHalf>
__device__ __forceinline__ void load_unit(const Params& p, int t0, uint32_t n, Unit<T, N>& w) {
  const int D = p.plan.head_dim, rot = p.plan.rot_dim;
  const uint32_t row = div_by(n, p.units_magic);
  const int u = (int)(n - row * (uint32_t)p.units);
  const uint32_t tl = div_by(row, p.heads_magic);
  const int head = (int)(row - tl * (uint32_t)p.heads);
  const int64_t t = t0 + (int)tl;
  if (head < p.hq) {
    w.in = static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)head * D;
    w.out = static_cast<T*>(p.q_out) + t * p.q_out_stride + (int64_t)head * D;
  } else {
    w.in = static_cast<const T*>(p.k) + t * p.k_stride + (int64_t)(head - p.hq) * D;
    w.out = static_cast<T*>(p.k_out) + t * p.k_out_stride + (int64_t)(head - p.hq) * D;
  }
  w.b = -1;
  if (u >= p.rot_units) {
    w.a = rot + (u - p.rot_units) * N;
    w.pair = -1;
  } else {
    const int angles = (int)tl * (rot / 2);  // this token's angles in shared memory
    if (kHalf) {
      w.a = u * N;
      w.b = w.a + rot / 2;
      w.pair = angles + w.a;
    } else if (N > 1) {
      w.a = u * N;
      w.pair = angles + w.a / 2;
    } else {
      w.a = 2 * u;
      w.b = w.a + 1;
      w.pair = angles + u;
    }
  }
  if constexpr (N > 1) {
    Vec<T>::load(*reinterpret_cast<const uint4*>(w.in + w.a), w.x);
    if (kHalf && w.b >= 0) Vec<T>::load(*reinterpret_cast<const uint4*>(w.in + w.b), w.y);
  } else {
    w.x[0] = to_float(w.in[w.a]);
    if (w.b >= 0) w.y[0] = to_float(w.in[w.b]);
  }
}

template <typename T, int N, bool kHalf>
__device__ __forceinline__ void store_unit(const float2* cs, Unit<T, N>& w) {
  if (w.pair >= 0) {
    if constexpr (kHalf || N == 1) {
#pragma unroll
      for (int i = 0; i < N; ++i) rotate(w.x[i], w.y[i], cs[w.pair + i]);
    } else {
#pragma unroll
      for (int i = 0; i + 1 < N; i += 2) rotate(w.x[i], w.x[i + 1], cs[w.pair + i / 2]);
    }
  } else if (w.in == w.out) {
    return;  // in place: nothing to copy
  }
  if constexpr (N > 1) {
    *reinterpret_cast<uint4*>(w.out + w.a) = Vec<T>::store(w.x);
    if (kHalf && w.b >= 0) *reinterpret_cast<uint4*>(w.out + w.b) = Vec<T>::store(w.y);
  } else {
    from_float(w.out + w.a, w.x[0]);
    if (w.b >= 0) from_float(w.out + w.b, w.y[0]);
  }
}

template <typename T, int N, bool kHalf>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Params p) {
  extern __shared__ float2 cs[];  // [tokens_per_cta][rot_dim / 2]
  const int t0 = (int)blockIdx.x * p.tokens_per_cta;
  const int tokens = min(p.tokens_per_cta, p.num_tokens - t0);
  const uint32_t items = (uint32_t)tokens * p.heads * p.units;
  constexpr int kAhead = N > 1 ? 2 : 1;
  Unit<T, N> w[kAhead];
  uint32_t n = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (n + i * kThreads < items) load_unit<T, N, kHalf>(p, t0, n + i * kThreads, w[i]);
  const int pairs = p.plan.rot_dim / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int tl = i / pairs;
    cs[i] = turn_of(p.plan.turns[i - tl * pairs], p.positions[t0 + tl], p.plan.amplitude, p.inverse != 0);
  }
  __syncthreads();
  while (true) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (n + i * kThreads < items) store_unit<T, N, kHalf>(cs, w[i]);
    n += kAhead * kThreads;
    if (n >= items) break;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (n + i * kThreads < items) load_unit<T, N, kHalf>(p, t0, n + i * kThreads, w[i]);
  }
}

template <typename T, int N, bool kHalf>
cb_status launch(Params& p, cudaStream_t stream) {
  const int D = p.plan.head_dim, rot = p.plan.rot_dim;
  p.rot_units = kHalf ? rot / 2 / N : N > 1 ? rot / N : rot / 2;
  p.units = p.rot_units + (D - rot) / N;
  auto magic = [](int d) { return d == 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d); };
  p.units_magic = magic(p.units);
  p.heads_magic = magic(p.heads);
  // tokens per CTA: one while the tokens fit the SMs' resident CTAs once
  // (latency), then four, so that a CTA's loads cover its set-up
  p.tokens_per_cta = p.num_tokens <= 8 * sm_count_current_device() ? 1 : 4;
  const uint64_t items = (uint64_t)p.tokens_per_cta * p.heads * p.units;
  if (items * (uint64_t)(p.units > p.heads ? p.units : p.heads) >= 0x100000000ull)
    return fail(CB_ERR_UNSUPPORTED, "cb_rope: %d heads of %d dims", p.heads, D);
  const int64_t ctas = ((int64_t)p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta;
  const size_t smem = (size_t)p.tokens_per_cta * (rot / 2) * sizeof(float2);
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
  uintptr_t al = 0;
  int64_t lengths = D | (half ? rot / 2 : rot);
  if (p.hq) {
    al |= (uintptr_t)p.q | (uintptr_t)p.q_out;
    lengths |= p.q_stride | p.q_out_stride;
  }
  if (p.heads > p.hq) {
    al |= (uintptr_t)p.k | (uintptr_t)p.k_out;
    lengths |= p.k_stride | p.k_out_stride;
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
    hi = std::fmin(std::ceil(at(c.beta_slow)), rot / 2 - 1);
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
  p.hq = a.q ? a.num_q_heads : 0;
  p.heads = p.hq + (a.k ? a.num_kv_heads : 0);
  const int64_t D = p.plan.head_dim;
  auto stride = [&](int64_t s, int32_t heads) { return s ? s : heads * D; };
  p.q = a.q;
  p.q_out = a.q_out;
  p.k = a.k;
  p.k_out = a.k_out;
  p.q_stride = stride(a.q_stride, a.num_q_heads);
  p.q_out_stride = stride(a.q_out_stride, a.num_q_heads);
  p.k_stride = stride(a.k_stride, a.num_kv_heads);
  p.k_out_stride = stride(a.k_out_stride, a.num_kv_heads);
  if ((a.q && (p.q_stride < a.num_q_heads * D || p.q_out_stride < a.num_q_heads * D)) ||
      (a.k && (p.k_stride < a.num_kv_heads * D || p.k_out_stride < a.num_kv_heads * D)))
    return fail(CB_ERR_INVALID_ARG, "cb_rope: a stride is less than a token's heads");
  const uintptr_t elem = a.dtype == CB_DTYPE_F32 ? 4 : 2;
  if ((((uintptr_t)a.q | (uintptr_t)a.q_out | (uintptr_t)a.k | (uintptr_t)a.k_out) & (elem - 1)) != 0)
    return fail(CB_ERR_INVALID_ARG, "cb_rope: pointers must be aligned to their element");
  return a.dtype == CB_DTYPE_F32 ? cb::rope::dispatch<float>(p, (cudaStream_t)stream)
                                 : cb::rope::dispatch<__nv_bfloat16>(p, (cudaStream_t)stream);
}
