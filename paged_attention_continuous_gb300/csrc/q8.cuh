// The 8-bit cache's number format: e4m3 codes, one power-of-two scale for
// each (block, KV head), stored as the byte exponent + 127.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "device_utils.cuh"

namespace cb {
namespace q8 {

constexpr int kPage = 16;              // tokens of a block
constexpr int kMinExp = -40, kMaxExp = 40;

// Exponent of a scale byte; bytes outside the range count as its ends, so
// that any byte gives a finite scale and products of two scales stay far
// inside float32.
__device__ __forceinline__ int exp_of(uint32_t byte) {
  return min(max((int)byte - 127, kMinExp), kMaxExp);
}

// 2^e, |e| <= 126
__device__ __forceinline__ float exp2i(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Least e with amax <= 448 * 2^e, in [kMinExp, kMaxExp].  448 = 1.75 * 2^8:
// an amax m * 2^k with 1 <= m < 2 needs k - 8, or k - 7 if m > 1.75.  Zero
// and float32 subnormals give kMinExp.
__device__ __forceinline__ int exp_for(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return min(max(e, kMinExp), kMaxExp);
}

// Two scaled values to e4m3 codes (low byte first), to nearest even, finite
// ones saturating at 448; an infinity becomes NaN (x + 0 * x is NaN then,
// and x otherwise).
__device__ __forceinline__ uint32_t codes2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(fmaf(hi, 0.f, hi)), "f"(fmaf(lo, 0.f, lo)));
  return r;
}

// Two codes (low byte first) to a pair of halves, exactly.
__device__ __forceinline__ uint32_t halves2(uint16_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(codes));
  return r;
}

// Four codes to two pairs of halves.
__device__ __forceinline__ void halves4(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// Two halves to codes, to nearest even.
__device__ __forceinline__ uint16_t codes_of_halves(uint32_t h) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
  return r;
}

__device__ __forceinline__ float2 floats2(uint16_t codes) {
  const uint32_t h = halves2(codes);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// Four codes moved to a scale 2^k times larger, k >= 1: code * 2^-k rounded
// to nearest even (exact unless the result is an e4m3 subnormal).  From k =
// 19 on every code becomes zero, and 2^-k stays a half up to there.
__device__ __forceinline__ uint32_t shrink4(uint32_t codes, int k) {
  const __half2 f = __float2half2_rn(exp2i(-min(k, 24)));
  uint32_t lo = halves2((uint16_t)(codes & 0xffffu)), hi = halves2((uint16_t)(codes >> 16));
  __half2 a = __hmul2(*reinterpret_cast<__half2*>(&lo), f);
  __half2 b = __hmul2(*reinterpret_cast<__half2*>(&hi), f);
  return (uint32_t)codes_of_halves(*reinterpret_cast<uint32_t*>(&a)) |
         ((uint32_t)codes_of_halves(*reinterpret_cast<uint32_t*>(&b)) << 16);
}

}  // namespace q8
}  // namespace cb
