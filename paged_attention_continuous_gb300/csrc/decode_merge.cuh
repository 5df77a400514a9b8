// Split tickets and the merge of split partials, shared by the decode kernels
// over the 8-bit and the 4-bit caches.
#pragma once

#include <cstdint>

#include "decode_launch.h"
#include "device_utils.cuh"

namespace cb {
namespace decode {

// Of four elements of every other one of eight dims (the odd ones, or those from
// the first on, whose others the lane `away` bits aside has): the four in the
// same places of the eight in order, which are its last or first ones.
__device__ __forceinline__ float4 exchange_odd(float4 v, bool odd, int away) {
  const float a = __shfl_xor_sync(0xffffffffu, odd ? v.x : v.z, away);
  const float b = __shfl_xor_sync(0xffffffffu, odd ? v.y : v.w, away);
  return odd ? make_float4(a, v.z, b, v.w) : make_float4(v.x, a, v.y, b);
}

// Merge the n >= 2 split partials of one item group (row, heads h0 .. h0 +
// heads), whose slots start at s0, into the rows of query token q0: per head
// o = sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s, in split order.
// kH heads at once, kB splits in flight.  kOdd: a part's places 8 i .. 8 i + 3 hold
// the even dims of its eight, the next four the odd ones.
template <typename T, int D, int kH, int kB, bool kOdd = false>
__device__ __forceinline__ void merge_splits(const float* part_ml, const float* part_acc, void* out, int Hq,
                                             int h0, int heads, int s0, int n, int q0) {
  const int lane = threadIdx.x & 31;
  constexpr int kV = D / 4;      // lanes that own 4 elements each
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
      if constexpr (kOdd) o[h] = exchange_odd(o[h], lane & 1, 1);
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

// The same as a call: it is rare.  Its caller keeps nothing alive across it;
// more splits in flight take registers that the caller would spill.
template <typename T, int D>
__device__ __noinline__ void merge_splits_call(const float* part_ml, const float* part_acc, void* out, int Hq,
                                               int h0, int heads, int s0, int n, int q0) {
  merge_splits<T, D, 4, 4>(part_ml, part_acc, out, Hq, h0, heads, s0, n, q0);
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

}  // namespace decode
}  // namespace cb
