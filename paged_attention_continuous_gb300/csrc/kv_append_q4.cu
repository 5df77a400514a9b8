// cb_kv_append_q4: a step's new K/V into the cache of 4-bit codes with one
// scale for each 32 dims of a token and KV head.
//
// "vLLM serving internals", PagedAttention as a virtual memory system: token
// t goes to block slot / 16, offset slot % 16.  Scales belong to tokens, so
// tokens are written independently of each other, in any order.
//
// A thread quantises a word of K and the same word of V (in large calls several):
// 8 neighbouring dims of a token and head (one or two 16-byte loads, a 4-byte
// store each); the threads of a group find its largest magnitude by shuffles and
// the first of them stores the scale.  With a rotary plan a CTA's tokens' angles are computed
// once, in shared memory, and a thread reads the partners of its dims itself
// (the half layout: from the line that another thread of the row reads too), so
// nothing is exchanged before the magnitude is taken; other CTAs rotate the
// tokens' q.
//
// Every new element is read once and every code written once.  What bounds it:
// in large calls the arithmetic (float32 and turned words take more than
// bfloat16's), in small ones the launch with one dependent access.  Measured in a
// replayed row of calls, 8 heads of 128: 8521 tokens 10.7 us, of which HBM needs
// 6.5, 32768 tokens 31.4 (5.4 TB/s); float32 19.4 of 11.7 and 62.6 of 44.8; 96 tokens
// with 32 heads of q turned 2.5, 8521 of those 42 of 27 (float32 62 of 53).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "cb_error.h"
#include "launch_common.h"
#include "q4.cuh"
#include "rope.cuh"
#include "rope.h"
#include "validate.h"

namespace cb {
namespace append_q4 {

using rope::Vec;

constexpr int kThreads = 256;
constexpr int kMaxTokens = 32;  // tokens of a CTA
enum { kNoRope = -1, kHalf = CB_ROPE_HALF, kInterleaved = CB_ROPE_INTERLEAVED };

struct Params {
  cb_rope_plan plan;
  const void* k_new;
  const void* v_new;
  const int32_t* slot_mapping;
  const int32_t* positions;
  uint8_t* k_cache;
  uint8_t* v_cache;
  int64_t num_slots;
  int32_t num_tokens, tokens_per_cta;
  int32_t num_kv_heads;
  uint32_t row_units_magic;  // ceil(2^32 / units of a token's K), see rope::div_by
  int32_t q_tokens;     // tokens of a CTA that rotates q
  rope::Rows q_rows;    // heads 0: no q
  uint32_t* error_word;
};

// Eight elements as they lie in memory.
template <typename T>
struct Word {
  static constexpr int kN = 8 / Vec<T>::kN;
  uint4 raw[kN];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kN; ++i) raw[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) Vec<T>::load(raw[i], x + i * Vec<T>::kN);
  }
};

__device__ __forceinline__ float max_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Bits of the largest magnitude of a word as a float: as bits, magnitudes
// order like whole numbers, infinity and NaN last.
__device__ __forceinline__ uint32_t top_of(const float (&x)[8]) {
  float m = max_nan(fabsf(x[0]), fabsf(x[1]), fabsf(x[2]));
  m = max_nan(m, fabsf(x[3]), fabsf(x[4]));
  return __float_as_uint(max_nan(max_nan(m, fabsf(x[5]), fabsf(x[6])), fabsf(x[7]), 0.f));
}
__device__ __forceinline__ uint32_t top_of(const uint4& x) {
  const uint32_t m = 0x7fff7fffu;
  const uint32_t a = __vmaxu2(__vmaxu2(x.x & m, x.y & m), __vmaxu2(x.z & m, x.w & m));
  return max(a & 0xffff0000u, a << 16);
}

// Quantises kW words (floats, or bfloat16s as they lie in memory) of a group,
// whose others the neighbouring lanes have, and stores them if `in`.
template <int D, int kW, typename X>
__device__ __forceinline__ void put(const X (&x)[kW], bool in, uint8_t* page, int token, int u) {
  uint32_t top = top_of(x[0]);
#pragma unroll
  for (int i = 1; i < kW; ++i) top = max(top, top_of(x[i]));
#pragma unroll
  for (int o = 1; o < 4 / kW; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (!in) return;
  const uint32_t byte = top < 0x7f800000u ? q4::byte_for(__uint_as_float(top)) : q4::kNanByte;
  uint32_t word[kW];
#pragma unroll
  for (int i = 0; i < kW; ++i) word[i] = q4::kZeroUnit | q4::kZeroUnit << 16;
  if (byte - 1u < q4::kTopByte) {
    if constexpr (std::is_same<X, uint4>::value) {
      const q4::RounderBf16 r(byte, __uint_as_float(top));
#pragma unroll
      for (int i = 0; i < kW; ++i) word[i] = r.word(x[i]);
    } else {
      const q4::Rounder r(byte);
#pragma unroll
      for (int i = 0; i < kW; ++i) word[i] = r.word(x[i]);
    }
  }
  uint8_t* at = page + token * q4::row_bytes(D) + 4 * kW * u;
  if constexpr (kW == 1) *reinterpret_cast<uint32_t*>(at) = word[0];
  else if constexpr (kW == 2) *reinterpret_cast<uint2*>(at) = make_uint2(word[0], word[1]);
  else *reinterpret_cast<uint4*>(at) = make_uint4(word[0], word[1], word[2], word[3]);
  if (u % (4 / kW) == 0) page[q4::scales_at(D, token) + u * kW / 4] = (uint8_t)byte;
}

// kW: words of K and of V that a thread quantises (1 with a rotary plan).
template <typename T, int D, int kRope, int kW>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ Params p) {
  constexpr int kUnits = D / 8 / kW;         // of a row
  extern __shared__ float2 cs[];             // [tokens_per_cta][rot_dim / 2]
  // the attention launch that follows (when it asks for it) may start now;
  // it reads the cache only after this grid has completed
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int t0 = (int)blockIdx.x * p.tokens_per_cta;
  const int tokens = min(p.tokens_per_cta, p.num_tokens - t0);
  if constexpr (kRope != kNoRope) {
    if (blockIdx.y >= 1) {
      const int q0 = ((int)blockIdx.y - 1) * p.q_tokens;
      if (q0 < tokens)
        rope::rotate_rows<T, Vec<T>::kN, kRope == kHalf, kThreads>(
            p.q_rows, p.plan, p.positions, t0 + q0, min(p.q_tokens, tokens - q0), false, cs);
      return;
    }
  }
  const int Hkv = p.num_kv_heads;
  const int row_units = Hkv * kUnits, units = tokens * row_units;
  const int pairs = kRope == kNoRope ? 0 : p.plan.rot_dim / 2;
  bool angles = kRope == kNoRope;
  // (whole warps: the shuffles want all lanes)
  for (int first = (int)(threadIdx.x & ~31u); first < units || !angles; first += kThreads) {
    const int i = first + (int)(threadIdx.x & 31);
    bool in = i < units;
    // (the quotient holds where a CTA has several tokens, of few words each)
    const int tl = in && tokens > 1 ? (int)rope::div_by((uint32_t)i, p.row_units_magic) : 0;
    const int at = in ? i - tl * row_units : 0, h = at / kUnits, u = at - h * kUnits, w = u * kW;
    const int64_t e = (((int64_t)t0 + tl) * Hkv + h) * D + 8 * w;
    Word<T> k[kW], partner, v[kW];
    int slot = -1;
    const bool turns = kRope != kNoRope && 8 * w < 2 * pairs, low = 8 * w < pairs;
    if (in) {
      slot = __ldg(p.slot_mapping + t0 + tl);
#pragma unroll
      for (int j = 0; j < kW; ++j) {
        k[j].load(static_cast<const T*>(p.k_new) + e + 8 * j);
        v[j].load(static_cast<const T*>(p.v_new) + e + 8 * j);
      }
      if (kRope == kHalf && turns) partner.load(static_cast<const T*>(p.k_new) + e + (low ? pairs : -pairs));
    }
    if constexpr (kRope != kNoRope) {
      if (!angles) {
        for (int a = threadIdx.x; a < tokens * pairs; a += kThreads) {
          const int ta = a / pairs;
          cs[a] = rope::turn_of(p.plan.turns[a - ta * pairs], p.positions[t0 + ta], p.plan.amplitude, false);
        }
        __syncthreads();
        angles = true;
      }
    }
    if (slot >= 0 && slot >= p.num_slots) {
      set_error(p.error_word, CB_DEVERR_SLOT_RANGE);
      slot = -1;
    }
    in = slot >= 0;
    const int64_t page = ((int64_t)(max(slot, 0) >> 4) * Hkv + h) * q4::page_bytes(D);
    const int token = slot & (q4::kPage - 1);
    const auto put_words = [&](const Word<T> (&y)[kW], uint8_t* cache) {
      if constexpr (sizeof(T) == 2) {
        uint4 x[kW];
#pragma unroll
        for (int j = 0; j < kW; ++j) x[j] = y[j].raw[0];
        put<D, kW>(x, in, cache + page, token, u);
      } else {
        float x[kW][8] = {};
#pragma unroll
        for (int j = 0; j < kW; ++j)
          if (in) y[j].values(x[j]);
        put<D, kW>(x, in, cache + page, token, u);
      }
    };
    if constexpr (kRope == kNoRope) {
      put_words(k, p.k_cache);
    } else {
      float turned[1][8] = {};
      float (&x)[8] = turned[0];
      if (in) k[0].values(x);
      if (in && turns) {
        if constexpr (kRope == kHalf) {
          float y[8];
          partner.values(y);
          const float2* c = cs + tl * pairs + (low ? 8 * w : 8 * w - pairs);
#pragma unroll
          for (int j = 0; j < 8; ++j) x[j] = low ? x[j] * c[j].x - y[j] * c[j].y : x[j] * c[j].x + y[j] * c[j].y;
        } else {
          const float2* c = cs + tl * pairs + 4 * w;
#pragma unroll
          for (int j = 0; j < 4; ++j) rope::rotate(x[2 * j], x[2 * j + 1], c[j]);
        }
      }
      put<D, 1>(turned, in, p.k_cache + page, token, u);
    }
    put_words(v, p.v_cache);
  }
}

template <typename T, int D, int kRope, int kW>
cb_status launch(Params& p, cudaStream_t stream) {
  static_assert(kW == 1 || kRope == kNoRope, "a thread turns one word");
  const uint32_t row_units = (uint32_t)p.num_kv_heads * (D / 8 / kW);  // (2 or more)
  p.row_units_magic = (uint32_t)((0x100000000ull + row_units - 1) / row_units);
  // a unit for each thread, of whole tokens
  p.tokens_per_cta = std::min(std::max(kThreads / (int)row_units, 1), kMaxTokens);
  int q_ctas = 0;
  if constexpr (kRope != kNoRope) {
    rope::Rows& r = p.q_rows;
    if (r.heads > 0) {
      rope::cut_rows(&r, Vec<T>::kN, kRope == kHalf);
      p.q_tokens = std::min(p.tokens_per_cta, 4);
      q_ctas = (p.tokens_per_cta + p.q_tokens - 1) / p.q_tokens;
      const uint64_t items = (uint64_t)p.q_tokens * r.heads * r.units;
      if (items * (uint64_t)(r.units > r.heads ? r.units : r.heads) >= 0x100000000ull)
        return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q4: %d query heads", r.heads);
    }
  }
  const unsigned ctas = (unsigned)(((int64_t)p.num_tokens + p.tokens_per_cta - 1) / p.tokens_per_cta);
  const size_t smem = kRope == kNoRope ? 0 : (size_t)p.tokens_per_cta * (p.plan.rot_dim / 2) * sizeof(float2);
  append_kernel<T, D, kRope, kW><<<dim3(ctas, (unsigned)(1 + q_ctas)), kThreads, smem, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "cb_kv_append_q4 launch: %s", cudaGetErrorString(e));
  return CB_OK;
}

template <typename T, int D>
cb_status dispatch(Params& p, bool with_rope, cudaStream_t stream) {
  // Words of one group in one thread share its scale and what places them, and
  // leave fewer threads: 8 heads of 128 dims, bfloat16, one / two / four words,
  // 512 tokens 2.5 / 2.5 / 3.3 us, 2048 4.6 / 4.1 / 4.3, 8521 14.6 / 11.9 / 10.7;
  // float32 3.2 / 3.4 / 5.5, 6.1 / 6.4 / 9.8, 21.9 / 19.5 / 36.8.
  constexpr int kMany = sizeof(T) == 2 ? 4 : 2;
  if (!with_rope && (int64_t)p.num_tokens * p.num_kv_heads * (D / 8) >= 1 << 18)
    return launch<T, D, kNoRope, kMany>(p, stream);
  if (!with_rope) return launch<T, D, kNoRope, 1>(p, stream);
  return p.plan.layout == CB_ROPE_HALF ? launch<T, D, kHalf, 1>(p, stream) : launch<T, D, kInterleaved, 1>(p, stream);
}

}  // namespace append_q4
}  // namespace cb

extern "C" cb_status cb_kv_append_q4(const cb_append_q4_args* args, cb_stream_t stream) {
  using cb::fail;
  using namespace cb::append_q4;
  if (!args) return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q4: args is NULL");
  const cb_append_q4_args& a = *args;
  if (a.num_tokens < 0 || a.num_blocks <= 0 || a.num_kv_heads <= 0 || a.head_dim <= 0 || a.block_size <= 0)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q4: sizes must be positive");
  if (a.dtype != CB_DTYPE_F32 && a.dtype != CB_DTYPE_BF16)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q4: unknown dtype");
  if (a.block_size != cb::q4::kPage) return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q4: block_size must be 16");
  if (a.head_dim != 64 && a.head_dim != 128)
    return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q4: head_dim must be 64 or 128");
  if (a.rope) {
    cb_status st = cb::check_rope_plan(a.rope, a.head_dim, "cb_kv_append_q4");
    if (st != CB_OK) return st;
    if (a.rope->rot_dim % 16 != 0)
      return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q4: rot_dim must be a multiple of 16");
    if (a.q && a.num_q_heads <= 0) return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q4: num_q_heads must be positive");
  } else if (a.q) {
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q4: q is rotated only with a rotary plan");
  }
  if (a.num_tokens == 0) return CB_OK;
  if (!a.k_new || !a.v_new || !a.slot_mapping || !a.k_cache || !a.v_cache || (a.rope && !a.positions) ||
      (a.q && !a.q_out))
    return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q4: NULL pointer");
  const uintptr_t align = (uintptr_t)a.k_new | (uintptr_t)a.v_new | (uintptr_t)a.k_cache | (uintptr_t)a.v_cache |
                          (uintptr_t)a.q | (uintptr_t)a.q_out;
  if (align & 15u) return fail(CB_ERR_INVALID_ARG, "cb_kv_append_q4: pointers must be 16-byte aligned");
  if ((int64_t)a.num_tokens * (a.num_kv_heads > a.num_q_heads ? a.num_kv_heads : a.num_q_heads) >= ((int64_t)1 << 31) ||
      a.num_kv_heads > (1 << 20) || a.num_q_heads > (1 << 20))
    return fail(CB_ERR_UNSUPPORTED, "cb_kv_append_q4: more than 2^31 rows in one call");
  if (cb::validate_enabled()) {
    cb_status vs = cb::validate_append_call(a.slot_mapping, a.num_tokens, a.num_blocks, a.block_size,
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
  const bool f32 = a.dtype == CB_DTYPE_F32;
  const cudaStream_t s = (cudaStream_t)stream;
  if (a.head_dim == 64)
    return f32 ? dispatch<float, 64>(p, a.rope, s) : dispatch<__nv_bfloat16, 64>(p, a.rope, s);
  return f32 ? dispatch<float, 128>(p, a.rope, s) : dispatch<__nv_bfloat16, 128>(p, a.rope, s);
}
