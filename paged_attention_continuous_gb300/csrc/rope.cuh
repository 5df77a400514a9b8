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

}  // namespace rope
}  // namespace cb
