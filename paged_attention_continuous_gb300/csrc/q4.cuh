// The 4-bit cache's number format: a block's page of one KV head is 17 rows
// of D / 2 bytes, 16 of codes and one of scale bytes, [16 tokens][D / 32].
//
// A group of 32 neighbouring dims of a token shares a scale s, the half whose
// bits are byte << 7: five bits of exponent and three of mantissa, so that a
// byte becomes an operand by one shift, and s keeps four bits at every size
// from 2^-14 to 240 (a power of two would cost up to a bit of every code).
// A value is (n - 8) s with n the code, 1 to 15: at most 3 + 4 bits, so a
// half and a bfloat16 exactly, and the matrix instructions see the cache's
// values without a rounding.  Byte 0xff is a half that is not a number: a
// group that held an element that is not finite reads as NaN.
//
// Codes lie so that pairs of halves cost one logic operation each.  The codes
// of dims 8 j .. 8 j + 7 are a 32-bit word: the even dims its low 16 bits, the
// odd ones its high 16, ascending from the low four, each sixteen then rotated
// left by two.  Bits 5..2 of a sixteen are then its first code and bits 9..6 its
// second, in the middle and at the top of a half's mantissa; with the two bytes
// exchanged the same places hold its third and fourth.  So a word gives the pairs
// of neighbouring dims, in their order, and a 32-bit word of the same sixteen of
// two tokens gives pairs of tokens.  With exponents put above them they are the
// halves 16 + n and 256 + n, and one fused multiply-add gives (16 + n) s - 24 s
// or (256 + n) s - 264 s = (n - 8) s.  Both constants are halves exactly (24 s
// has 6 bits, 264 s ten), which is why s ends at 240.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "device_utils.cuh"

namespace cb {
namespace q4 {

constexpr int kPage = 16;             // tokens of a block
constexpr int kGroup = 32;            // dims that share a scale
constexpr uint32_t kTopByte = 0xb7;   // the largest scale, 240
constexpr uint32_t kNanByte = 0xff;
constexpr int kTopCode = 7;           // of n - 8

constexpr int row_bytes(int D) { return D / 2; }
constexpr int page_bytes(int D) { return (kPage + 1) * (D / 2); }
// where a token's scales begin in a page
__host__ __device__ constexpr int scales_at(int D, int token) { return kPage * (D / 2) + token * (D / kGroup); }

__device__ __forceinline__ float scale_of(uint32_t byte) {
  return __half2float(__ushort_as_half((unsigned short)(byte << 7)));
}

// Least byte with amax <= 7.5 s (kTopByte if there is none): every element
// then lies within half a step of its value.  The quotient is taken a little
// too large, so that its first bits (cut off by the conversion to a half, whose
// top byte and a half they are, subnormal or not) are those of that byte or of
// the one before.
__device__ __forceinline__ uint32_t byte_for(float amax) {
  const float q = amax * (2.f / 15.f * 1.0000003f);
  uint32_t b = min((uint32_t)__half_as_ushort(__float2half_rz(q)) >> 7, kTopByte);
  b += 7.5f * scale_of(b) < amax ? 1u : 0u;
  return min(b, kTopByte);
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two sixteens (the even dims' codes and the odd ones'), rotated left by two bits
// each.
__device__ __forceinline__ uint32_t turn_units(uint32_t w) {
  return (w << 2 & 0xfffcfffcu) | (w >> 14 & 0x00030003u);
}

// The codes of eight neighbouring dims: x / s to nearest even, -7 to 7, plus 8.
// Rounded by adding 1.5 * 2^23, whose sum has the whole number in its low bits;
// x times the reciprocal may be off next to a border, but the remainder x - r s
// is exact and says which side x is on: past half a step, or at it with r odd,
// r moves by one.  (Magnitudes past 7 s count as 7 s.)
struct Rounder {
  float s, inv, half, below, most;  // below: the float before half
  __device__ __forceinline__ explicit Rounder(uint32_t byte) {
    s = scale_of(byte);
    inv = rcp_approx(s);
    half = 0.5f * s;
    below = __uint_as_float(__float_as_uint(half) - 1u);
    most = (float)kTopCode * s;
  }
  __device__ __forceinline__ int code(float x) const {
    constexpr float kMagic = 12582912.f;
    x = fminf(fmaxf(x, -most), most);
    const float y = fmaf(x, inv, kMagic), d = fmaf(kMagic - y, s, x);
    int n = __float_as_int(y);
    if (fabsf(d) > ((n & 1) ? below : half)) n += (__float_as_int(d) >> 31) | 1;
    return n;  // its low 16 bits: those of the rounded number
  }
  __device__ __forceinline__ uint32_t four(const float* x) const {  // of every other dim
    return (uint32_t)(code(x[0]) + code(x[2]) * 16 + code(x[4]) * 256 + code(x[6]) * 4096 + 0x8888) & 0xffffu;
  }
  __device__ __forceinline__ uint32_t word(const float (&x)[8]) const {
    return turn_units(four(x) | four(x + 1) << 16);
  }
};

// The same of bfloat16 elements, two at a time.  192 is 1.5 * 2^7; the remainder
// is exact here too (x, and r s of seven bits, differ by at most x's own size
// or by 64 of its last bits), and the reciprocal's error of 2^-9 moves no
// quotient by more than 0.015.  `wide`: some magnitude may pass 7 s.
struct RounderBf16 {
  uint32_t s, inv, half, most;
  bool wide;
  __device__ __forceinline__ RounderBf16(uint32_t byte, float amax) {
    const float f = scale_of(byte);
    s = float2_to_bf16x2(f, f);
    const float i = rcp_approx(f);
    inv = float2_to_bf16x2(i, i);
    half = float2_to_bf16x2(0.5f * f, 0.5f * f);
    most = float2_to_bf16x2((float)kTopCode * f, (float)kTopCode * f);
    wide = amax >= 7.5f * f;
  }
  __device__ __forceinline__ uint32_t two(uint32_t x) const {  // at bits 3..0 of either half
    const auto v = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const auto u = [](__nv_bfloat162 w) { return *reinterpret_cast<const uint32_t*>(&w); };
    if (wide) x = u(__hmin2(__hmax2(v(x), v(most ^ 0x80008000u)), v(most)));
    const __nv_bfloat162 magic = v(0x43404340u);
    const __nv_bfloat162 y = __hfma2(v(x), v(inv), magic);
    const uint32_t d = u(__hfma2(__hsub2(magic, y), v(s), v(x)));
    // (positive numbers: the one before half has bits one less)
    const uint32_t past = __hgt2_mask(v(d & 0x7fff7fffu), v(half - (u(y) & 0x00010001u)));
    return (u(__hadd2(y, v(((d & 0x80008000u) | 0x3f803f80u) & past))) ^ 0x00080008u) & 0x000f000fu;
  }
  __device__ __forceinline__ uint32_t word(const uint4& x) const {
    return turn_units(two(x.x) | two(x.y) << 4 | two(x.z) << 8 | two(x.w) << 12);
  }
};
constexpr uint32_t kZeroUnit = 0x2222u;  // four codes of 8

// The multiplier and the two addends of a scale (or of a pair of scales).
struct Scale {
  __half2 s, c24, c264;
};
__device__ __forceinline__ Scale scale_from(__half2 s) {
  return Scale{s, __hmul2(s, __float2half2_rn(-24.f)), __hmul2(s, __float2half2_rn(-264.f))};
}
// A byte's scale, twice.
__device__ __forceinline__ Scale scale_twice(uint32_t byte) {
  const uint32_t w = byte * 0x00800080u;
  return scale_from(*reinterpret_cast<const __half2*>(&w));
}

// Byte i (0 or 1) of either half of a word: two tokens' scales.
__device__ __forceinline__ Scale scale_pair(uint32_t two, int i) {
  const uint32_t w = (i == 0 ? two << 7 : two >> 1) & 0x7f807f80u;
  return scale_from(*reinterpret_cast<const __half2*>(&w));
}

// The exponents that go above the fields, kept in registers: a logic operation
// takes one constant, the mask.
struct Exponents {
  uint32_t mid = 0x5c005c00u, top = 0x4c004c00u;
  __device__ __forceinline__ Exponents() { asm volatile("" : "+r"(mid), "+r"(top)); }
};

__device__ __forceinline__ uint32_t fields(uint32_t w, uint32_t mask, uint32_t exps) {
  uint32_t r;  // (w & mask) | exps
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(w), "r"(mask), "r"(exps));
  return r;
}
__device__ __forceinline__ uint32_t fma_fields(uint32_t f, __half2 s, __half2 c) {
  const __half2 v = __hfma2(*reinterpret_cast<__half2*>(&f), s, c);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Four pairs of halves of a word whose two 16-bit halves hold four codes each:
// out[i] = (code i of the low one, code i of the high one) under the scale's
// low and high half.
__device__ __forceinline__ void halves8(uint32_t w, const Scale& s, const Exponents& e, uint32_t (&out)[4]) {
  const uint32_t x = __byte_perm(w, 0u, 0x2301);
  out[0] = fma_fields(fields(w, 0x003c003cu, e.mid), s.s, s.c264);
  out[1] = fma_fields(fields(w, 0x03c003c0u, e.top), s.s, s.c24);
  out[2] = fma_fields(fields(x, 0x003c003cu, e.mid), s.s, s.c264);
  out[3] = fma_fields(fields(x, 0x03c003c0u, e.top), s.s, s.c24);
}

// The eight values of a word, ascending dims.
__device__ __forceinline__ void values8(uint32_t w, uint32_t byte, float (&x)[8]) {
  uint32_t h[4];
  halves8(w, scale_twice(byte), Exponents(), h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}

}  // namespace q4
}  // namespace cb
