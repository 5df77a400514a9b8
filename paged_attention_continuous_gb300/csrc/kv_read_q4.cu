// cb_kv_read_q4: tokens of a 4-bit cache as rows of bfloat16 or float32.
//
// The reverse of cb_kv_append_q4: token t's K and V come from block slot / 16,
// offset slot % 16.  Values are (n - 8) s exactly (seven bits).
//
// A thread expands a word of K and the same word of V, 8 neighbouring dims of a
// head, for kTokens tokens: 4 bytes of codes and a scale byte each become 16 or
// 32 bytes, which a warp stores as whole lines.  HBM bounds it, and in it the
// rows written (four fifths of the traffic in bfloat16): 32768 tokens of 8 heads of 128
// dims 29.8 us, 5.7 TB/s, 84% of the measured copy rate (float32 67 us, 4.5 TB/s; 8521
// tokens 8.2 and 21.2).  Each access waits for
// its token's slot, so a thread has several tokens' on the way.
#include <cuda_runtime.h>

#include <algorithm>

#include "cb_error.h"
#include "q4.cuh"
#include "rope.cuh"
#include "validate.h"

namespace cb {
namespace read_q4 {

constexpr int kThreads = 128;

struct Params {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* slot_mapping;
  void* k_out;
  void* v_out;
  int64_t num_slots;
  int32_t num_tokens, num_kv_heads;
  int32_t sets;            // of kTokens tokens to a CTA
  uint32_t* error_word;
};

template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&x)[8]) {
  constexpr int N = rope::Vec<T>::kN;
#pragma unroll
  for (int i = 0; i < 8 / N; ++i) __stcs(reinterpret_cast<uint4*>(p) + i, rope::Vec<T>::store(x + i * N));
}

template <typename T, int D, int kTokens>
__global__ void __launch_bounds__(kThreads) read_kernel(const Params p) {
  constexpr int kWords = D / 8;
  const int row_words = p.num_kv_heads * kWords;
  const int set = p.sets > 1 ? (int)threadIdx.x / row_words : 0;
  if (set >= p.sets) return;
  const int64_t t0 = ((int64_t)blockIdx.x * p.sets + set) * kTokens;
  int slots[kTokens];
#pragma unroll
  for (int k = 0; k < kTokens; ++k) {
    // padding, and tokens past the last: their rows stay as they are
    slots[k] = t0 + k < p.num_tokens ? __ldg(p.slot_mapping + t0 + k) : -1;
    if (slots[k] >= 0 && slots[k] >= p.num_slots) {
      set_error(p.error_word, CB_DEVERR_SLOT_RANGE);
      slots[k] = -1;
    }
  }
  for (int i = (int)threadIdx.x - set * row_words; i < row_words; i += kThreads) {
    const int h = i / kWords, w = i - h * kWords;
    uint32_t kw[kTokens], vw[kTokens], ks[kTokens], vs[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      const int slot = max(slots[k], 0), token = slot & (q4::kPage - 1);
      const int64_t page = ((int64_t)(slot >> 4) * p.num_kv_heads + h) * q4::page_bytes(D);
      const int64_t code = page + token * q4::row_bytes(D) + 4 * w, scale = page + q4::scales_at(D, token) + w / 4;
      if (slots[k] >= 0) {
        kw[k] = __ldg(reinterpret_cast<const uint32_t*>(p.k_cache + code));
        vw[k] = __ldg(reinterpret_cast<const uint32_t*>(p.v_cache + code));
        ks[k] = __ldg(p.k_cache + scale);
        vs[k] = __ldg(p.v_cache + scale);
      }
    }
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
      if (slots[k] < 0) continue;
      const int64_t e = ((t0 + k) * row_words + i) * 8;
      float x[8];
      q4::values8(kw[k], ks[k], x);
      store8(static_cast<T*>(p.k_out) + e, x);
      q4::values8(vw[k], vs[k], x);
      store8(static_cast<T*>(p.v_out) + e, x);
    }
    if (p.sets > 1) break;  // a set's words have a thread each
  }
}

template <typename T, int D, int kTokens>
void launch_sets(const Params& p, cudaStream_t stream) {
  const int64_t per_cta = (int64_t)p.sets * kTokens;
  read_kernel<T, D, kTokens><<<(unsigned)((p.num_tokens + per_cta - 1) / per_cta), kThreads, 0, stream>>>(p);
}

// One token to a thread spreads few tokens over more SMs, four keep more
// loads on the way (8 heads of 128 dims, bfloat16: 16 tokens 4.7 / 5.1 us,
// 1536 5.1 / 5.3, 8768 10.4 / 10.2, 32768 31.6 / 28.0, in one replayed call each;
// eight are slower again).
template <typename T, int D>
void launch(Params& p, cudaStream_t stream) {
  p.sets = std::max(kThreads / (p.num_kv_heads * (D / 8)), 1);
  if (p.num_tokens < 8192) launch_sets<T, D, 1>(p, stream);
  else launch_sets<T, D, 4>(p, stream);
}

}  // namespace read_q4
}  // namespace cb

extern "C" cb_status cb_kv_read_q4(const cb_read_q4_args* args, cb_stream_t stream_) {
  using cb::fail;
  using namespace cb::read_q4;
  if (!args) return fail(CB_ERR_INVALID_ARG, "cb_kv_read_q4: args is NULL");
  const cb_read_q4_args& a = *args;
  if (a.num_tokens < 0 || a.num_blocks <= 0 || a.num_kv_heads <= 0 || a.head_dim <= 0 || a.block_size <= 0)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_read_q4: sizes must be positive");
  if (a.dtype != CB_DTYPE_F32 && a.dtype != CB_DTYPE_BF16)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_read_q4: unknown dtype");
  if (a.block_size != cb::q4::kPage) return fail(CB_ERR_UNSUPPORTED, "cb_kv_read_q4: block_size must be 16");
  if (a.head_dim != 64 && a.head_dim != 128)
    return fail(CB_ERR_UNSUPPORTED, "cb_kv_read_q4: head_dim must be 64 or 128");
  if (a.num_tokens == 0) return CB_OK;
  if (!a.k_cache || !a.v_cache || !a.slot_mapping || !a.k_out || !a.v_out)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_read_q4: NULL pointer");
  if (((uintptr_t)a.k_cache | (uintptr_t)a.v_cache | (uintptr_t)a.k_out | (uintptr_t)a.v_out) & 15u)
    return fail(CB_ERR_INVALID_ARG, "cb_kv_read_q4: pointers must be 16-byte aligned");
  if ((int64_t)a.num_tokens * a.num_kv_heads >= ((int64_t)1 << 31) || a.num_kv_heads > (1 << 20))
    return fail(CB_ERR_UNSUPPORTED, "cb_kv_read_q4: more than 2^31 rows in one call");
  const cudaStream_t stream = (cudaStream_t)stream_;
  if (cb::validate_enabled()) {
    cb_status vs = cb::validate_append_call(a.slot_mapping, a.num_tokens, a.num_blocks, a.block_size, stream);
    if (vs != CB_OK) return vs;
  }
  Params p{};
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.slot_mapping = a.slot_mapping;
  p.k_out = a.k_out;
  p.v_out = a.v_out;
  p.num_slots = (int64_t)a.num_blocks * a.block_size;
  p.num_tokens = a.num_tokens;
  p.num_kv_heads = a.num_kv_heads;
  p.error_word = a.error_word;
  if (a.dtype == CB_DTYPE_F32) {
    if (a.head_dim == 64) launch<float, 64>(p, stream);
    else launch<float, 128>(p, stream);
  } else {
    if (a.head_dim == 64) launch<__nv_bfloat16, 64>(p, stream);
    else launch<__nv_bfloat16, 128>(p, stream);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "cb_kv_read_q4 launch: %s", cudaGetErrorString(e));
  return CB_OK;
}
