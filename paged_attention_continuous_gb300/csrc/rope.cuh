// Rotary positions: the angle and the rotation of one pair, shared by the
// cb_rope kernel and the append into the 8-bit cache.
//
// A pair (a, b) at position p turns by p * f.  The plan holds f as a 64-bit
// fraction of a turn, so p * turns mod 2^64 is the angle as a fraction of a
// turn with an error of |p| * 2^-65 turns: no range reduction is left to do
// at any position, and no 64-bit floating point (which this chip has little
// of).  Its top 32 bits, as a signed number of half turns in [-1, 1), go to
// sincospif: the error of that float is at most 2^-25 half turns.  A table
// of cosines would be read instead for every token; computed once per
// (token, pair) and shared by all heads in shared memory, the angles cost
// less than that read and need no memory that grows with the context.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "device_utils.cuh"

namespace cb {
namespace rope {

// (amplitude cos, amplitude sin) of one pair at position pos
__device__ __forceinline__ float2 turn_of(uint64_t turns, int32_t pos, float amplitude, bool inverse) {
  const uint64_t angle = turns * (uint64_t)(int64_t)pos;
  const float half_turns = __int2float_rn((int32_t)(angle >> 32)) * 4.656612873077393e-10f;  // 2^-31
  float s, c;
  sincospif(half_turns, &s, &c);
  return make_float2(c * amplitude, (inverse ? -s : s) * amplitude);
}

__device__ __forceinline__ void rotate(float& a, float& b, float2 cs) {
  const float x = a * cs.x - b * cs.y;
  b = b * cs.x + a * cs.y;
  a = x;
}

// 16 bytes of T as floats and back (rounded to nearest even)
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void load(const uint4& w, float* f) {
    const float2 a = bf16x2_to_float2(w.x), b = bf16x2_to_float2(w.y);
    const float2 c = bf16x2_to_float2(w.z), d = bf16x2_to_float2(w.w);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
    f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    return make_uint4(float2_to_bf16x2(f[0], f[1]), float2_to_bf16x2(f[2], f[3]),
                      float2_to_bf16x2(f[4], f[5]), float2_to_bf16x2(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void load(const uint4& w, float* f) {
    f[0] = __uint_as_float(w.x); f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z); f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 store(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
};

__device__ __forceinline__ float to_float(float x) { return x; }
__device__ __forceinline__ float to_float(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_float(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_float(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// ---- rows of q (and k) as units of work ------------------------------------
// The rows of a few tokens, cut into units that one thread moves.  In the
// half layout (and for single elements): rot_units per head row that rotate,
// then units that are only copied.  Interleaved vectors: vector u of a row and
// the one half a row further on, of which the first rot_units rotate.
struct Rows {
  int32_t head_dim, rot_dim;
  int32_t hq, heads;                  // heads of q (0 without q), of q and k together
  int32_t units, rot_units;           // of one head row
  uint32_t units_magic, heads_magic;  // ceil(2^32 / x)
  const void* q;
  void* q_out;
  const void* k;
  void* k_out;
  int64_t q_stride, q_out_stride, k_stride, k_out_stride;  // elements from token to token
};

// Fills units, rot_units and the magics for units of N elements.
inline void cut_rows(Rows* r, int n, bool half) {
  r->rot_units = half ? r->rot_dim / 2 / n : n > 1 ? r->rot_dim / n : r->rot_dim / 2;
  r->units = !half && n > 1 ? (r->head_dim / n + 1) / 2 : r->rot_units + (r->head_dim - r->rot_dim) / n;
  auto magic = [](int d) { return d == 1 ? 0u : (uint32_t)((0x100000000ull + d - 1) / d); };
  r->units_magic = magic(r->units);
  r->heads_magic = magic(r->heads);
}

// Pairs of a unit of N elements, and where the angle of pair i lies in shared
// memory: the i-th pairs of all units side by side, so that neighbouring
// threads read neighbouring words.
template <int N, bool kHalf>
constexpr int unit_pairs() { return N == 1 || kHalf ? N : N / 2; }
template <int N, bool kHalf>
__device__ __forceinline__ int angle_at(int i, int pairs) {
  constexpr int g = unit_pairs<N, kHalf>();
  return i % g * (pairs / g) + i / g;
}

// n / d for n d < 2^32, magic = ceil(2^32 / d) (0 for d = 1)
__device__ __forceinline__ uint32_t div_by(uint32_t n, uint32_t magic) {
  return magic ? __umulhi(n, magic) : n;
}

// A unit of work: N elements at `a`, and at `b` (unless negative) their
// partners in the half layout, other N elements in the interleaved one, or (N
// = 1, for rows that vectors do not fit) the other of a pair.  pair < 0: what
// is only copied.
template <typename T, int N>
struct Unit {
  T* out;
  int a, b, pair, pair_b;
  bool same;        // in place
  uint4 x, y;       // N elements each, as they lie in memory (N = 1: one float)
};

template <typename T, int N, bool kHalf>
__device__ __forceinline__ void load_unit(const Rows& p, int t0, uint32_t n, Unit<T, N>& w) {
  const int D = p.head_dim, rot = p.rot_dim;
  const uint32_t row = div_by(n, p.units_magic);
  const int u = (int)(n - row * (uint32_t)p.units);
  const uint32_t tl = div_by(row, p.heads_magic);
  const int head = (int)(row - tl * (uint32_t)p.heads);
  const int64_t t = t0 + (int)tl;
  const T* in;
  if (head < p.hq) {
    in = static_cast<const T*>(p.q) + t * p.q_stride + (int64_t)head * D;
    w.out = static_cast<T*>(p.q_out) + t * p.q_out_stride + (int64_t)head * D;
  } else {
    in = static_cast<const T*>(p.k) + t * p.k_stride + (int64_t)(head - p.hq) * D;
    w.out = static_cast<T*>(p.k_out) + t * p.k_out_stride + (int64_t)(head - p.hq) * D;
  }
  w.same = in == w.out;
  w.b = -1;
  const int angles = (int)tl * (rot / 2);  // this token's in shared memory
  if constexpr (!kHalf && N > 1) {
    const int v = u + p.units;
    w.a = u * N;
    w.b = v * N < D ? v * N : -1;
    w.pair = u < p.rot_units ? angles + u : -1;
    w.pair_b = v < p.rot_units ? angles + v : -1;
  } else if (u >= p.rot_units) {
    w.a = rot + (u - p.rot_units) * N;
    w.pair = -1;
  } else {
    w.pair = angles + u;  // the unit's first angle
    if (kHalf) {
      w.a = u * N;
      w.b = w.a + rot / 2;
    } else {
      w.a = 2 * u;
      w.b = w.a + 1;
    }
  }
  if constexpr (N > 1) {
    w.x = *reinterpret_cast<const uint4*>(in + w.a);
    if (w.b >= 0) w.y = *reinterpret_cast<const uint4*>(in + w.b);
  } else {
    w.x.x = __float_as_uint(to_float(in[w.a]));
    if (w.b >= 0) w.y.x = __float_as_uint(to_float(in[w.b]));
  }
}

template <typename T, int N, bool kHalf>
__device__ __forceinline__ void store_unit(const float2* cs, int stride, const Unit<T, N>& w) {
  if (w.pair < 0 && w.same) return;  // in place: nothing to copy
  if constexpr (N == 1) {
    float x = __uint_as_float(w.x.x), y = __uint_as_float(w.y.x);
    if (w.pair >= 0) rotate(x, y, cs[w.pair]);
    from_float(w.out + w.a, x);
    if (w.b >= 0) from_float(w.out + w.b, y);
  } else if constexpr (kHalf) {
    if (w.pair < 0) {
      *reinterpret_cast<uint4*>(w.out + w.a) = w.x;
      return;
    }
    float x[N], y[N];
    Vec<T>::load(w.x, x);
    Vec<T>::load(w.y, y);
#pragma unroll
    for (int i = 0; i < N; ++i) rotate(x[i], y[i], cs[w.pair + i * stride]);
    *reinterpret_cast<uint4*>(w.out + w.b) = Vec<T>::store(y);
    *reinterpret_cast<uint4*>(w.out + w.a) = Vec<T>::store(x);
  } else {
    auto vector = [&](uint4 raw, int at, int pair) {
      if (pair >= 0) {
        float x[N];
        Vec<T>::load(raw, x);
#pragma unroll
        for (int i = 0; i < N; i += 2) rotate(x[i], x[i + 1], cs[pair + i / 2 * stride]);
        raw = Vec<T>::store(x);
      }
      if (pair >= 0 || !w.same) *reinterpret_cast<uint4*>(w.out + at) = raw;
    };
    vector(w.x, w.a, w.pair);
    if (w.b >= 0) vector(w.y, w.b, w.pair_b);
  }
}

// Rotates the rows of tokens t0 .. t0 + tokens: all kThreads threads of a CTA,
// a unit to a thread at a time.  The first units are loaded before the angles
// (cs: tokens * rot_dim / 2 of them, in shared memory), so that their
// latencies overlap.
template <typename T, int N, bool kHalf, int kThreads>
__device__ __forceinline__ void rotate_rows(const Rows& rows, const cb_rope_plan& plan, const int32_t* positions,
                                            int t0, int tokens, bool inverse, float2* cs) {
  constexpr int kAhead = N == 1 ? 1 : 2;  // 64 bytes of loads in flight per thread
  const uint32_t items = (uint32_t)tokens * rows.heads * rows.units;
  Unit<T, N> w[kAhead];
  uint32_t n = threadIdx.x;
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (n + i * kThreads < items) load_unit<T, N, kHalf>(rows, t0, n + i * kThreads, w[i]);
  const int pairs = plan.rot_dim / 2;
  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int tl = i / pairs, pair = i - tl * pairs;
    cs[tl * pairs + angle_at<N, kHalf>(pair, pairs)] =
        turn_of(plan.turns[pair], positions[t0 + tl], plan.amplitude, inverse);
  }
  __syncthreads();
  while (true) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (n + i * kThreads < items) store_unit<T, N, kHalf>(cs, pairs / unit_pairs<N, kHalf>(), w[i]);
    n += kAhead * kThreads;
    if (n >= items) break;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (n + i * kThreads < items) load_unit<T, N, kHalf>(rows, t0, n + i * kThreads, w[i]);
  }
}

}  // namespace rope
}  // namespace cb
