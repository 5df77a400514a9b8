// cb_paged_attention_q4: paged attention over the 4-bit cache: checks and
// dispatch.
//
// The definition is cb_paged_attention's ("Chunked Prefill", How chunked
// prefill works) with an element of key j or value j read as (n - 8) s, n its
// code and s its group's scale.
#include <cuda_runtime.h>

#include "attention_packed.h"
#include "cb_error.h"
#include "decode_q4.h"
#include "launch_common.h"
#include "prefill_q4.h"
#include "q4.cuh"
#include "rope.cuh"
#include "row_checks.h"
#include "validate.h"

namespace cb {
namespace q4 {

struct RowsParams {
  const void* q;
  void* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens;
  const int32_t* block_tables;
  int32_t row_begin, row_end;   // rows handled; others' tokens are skipped
  int32_t num_rows, num_decodes, num_tokens;
  int32_t num_blocks, max_blocks_per_seq;
  int32_t num_q_heads, num_kv_heads;
  float scale_log2;
  int32_t window;
  uint32_t* error_word;
};

// One warp per (token, query head), keys walked one at a time with an online
// softmax in float32: any group size, head dim and query type.
template <typename T, int D>
__global__ void __launch_bounds__(256) rows_kernel(const RowsParams p) {
  constexpr int kPairs = D / 64;   // a lane's pairs of dims
  const int lane = threadIdx.x & 31;
  const int64_t wid = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  const int Hq = p.num_q_heads, Hkv = p.num_kv_heads;
  if (blockIdx.x == 0) {
    // rows that are no rows: the other kernels' checks of lengths and queries
    for (int r = p.row_begin + (int)threadIdx.x; r < p.row_end; r += (int)blockDim.x) {
      const int q0 = p.cu_seqlens_q[r], q_len = p.cu_seqlens_q[r + 1] - q0, L = p.seq_lens[r];
      if (q_len == 0 && L == 0) continue;  // padding
      if (r < p.num_decodes) {
        if (q_len != 1 || !row_tokens_fit(q0, 1, p.num_tokens)) set_error(p.error_word, CB_DEVERR_DECODE_QLEN);
        if (!row_length_fits(L, kPage, p.max_blocks_per_seq)) set_error(p.error_word, CB_DEVERR_SEQ_RANGE);
      } else if (q_len < 1 || !row_tokens_fit(q0, q_len, p.num_tokens)) {
        set_error(p.error_word, CB_DEVERR_SEQ_RANGE);
      }
    }
  }
  if (wid >= (int64_t)p.num_tokens * Hq) return;
  const int t = (int)(wid / Hq), h = (int)(wid % Hq);
  // the last row whose queries start at or before t
  int lo = 0, hi = p.num_rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (p.cu_seqlens_q[mid] <= t) lo = mid; else hi = mid - 1;
  }
  const int r = lo, q0 = p.cu_seqlens_q[r], q1 = p.cu_seqlens_q[r + 1];
  if (t < q0 || t >= q1 || r < p.row_begin || r >= p.row_end) return;
  const int L = p.seq_lens[r], q_len = q1 - q0;
  if ((r < p.num_decodes && q_len != 1) || !row_tokens_fit(q0, q_len, p.num_tokens)) return;  // flagged above
  if (L < q_len || !row_length_fits(L, kPage, p.max_blocks_per_seq)) {
    if (lane == 0) set_error(p.error_word, CB_DEVERR_SEQ_RANGE);
    return;
  }
  const int pos = L - q_len + (t - q0), g = h / (Hq / Hkv);
  const T* qrow = static_cast<const T*>(p.q) + ((int64_t)t * Hq + h) * D + lane * (2 * kPairs);
  float qf[2 * kPairs], acc[2 * kPairs];
#pragma unroll
  for (int e = 0; e < 2 * kPairs; ++e) {
    qf[e] = rope::to_float(qrow[e]) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int k_lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
  const int word = lane * kPairs / 4, first = lane * kPairs % 4;  // of the lane's pairs
  const auto values = [&](const uint8_t* page, int token, float (&x)[2 * kPairs]) {
    float y[8];
    values8(*reinterpret_cast<const uint32_t*>(page + token * row_bytes(D) + 4 * word),
            page[scales_at(D, token) + word / 4], y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int e = 0; e < kPairs; ++e)
        if (i == first + e) {
          x[2 * e] = y[2 * i];
          x[2 * e + 1] = y[2 * i + 1];
        }
    }
  };
  for (int pg = k_lo / kPage; pg <= pos / kPage; ++pg) {
    const int blk = p.block_tables[(int64_t)r * p.max_blocks_per_seq + pg];
    // (a page that cannot be read counts as zeros, as in the other kernels)
    const bool there = blk >= 0 && blk < p.num_blocks;
    if (!there && lane == 0) set_error(p.error_word, CB_DEVERR_BLOCK_RANGE);
    const int64_t page = there ? ((int64_t)blk * Hkv + g) * page_bytes(D) : 0;
    const int i1 = min(kPage, pos + 1 - pg * kPage);
    for (int i = max(0, k_lo - pg * kPage); i < i1; ++i) {
      float k[2 * kPairs] = {}, v[2 * kPairs] = {};
      if (there) {
        values(p.k_cache + page, i, k);
        values(p.v_cache + page, i, v);
      }
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < 2 * kPairs; ++e) dot = fmaf(qf[e], k[e], dot);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      const float mn = fmaxf(m, dot);
      const float a = exp2f(m - mn), w = exp2f(dot - mn);
      l = l * a + w;
#pragma unroll
      for (int e = 0; e < 2 * kPairs; ++e) acc[e] = fmaf(w, v[e], acc[e] * a);
      m = mn;
    }
  }
  T* orow = static_cast<T*>(p.out) + ((int64_t)t * Hq + h) * D + lane * (2 * kPairs);
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < 2 * kPairs; ++e) rope::from_float(orow + e, acc[e] * inv);
}

namespace {

template <typename T, int D>
cb_status launch_rows(const RowsParams& p, cudaStream_t stream) {
  const int64_t blocks = ((int64_t)p.num_tokens * p.num_q_heads + 7) / 8;
  if (blocks >= ((int64_t)1 << 31)) return fail(CB_ERR_UNSUPPORTED, "more than 2^34 query rows");
  rows_kernel<T, D><<<(unsigned)blocks, 256, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "rows kernel launch: %s", cudaGetErrorString(e));
  return CB_OK;
}

}  // namespace
}  // namespace q4
}  // namespace cb

extern "C" cb_status cb_paged_attention_q4(const cb_attention_args* args, cb_stream_t stream_) {
  using cb::fail;
  if (!args) return fail(CB_ERR_INVALID_ARG, "args is NULL");
  const cb_attention_args& a = *args;
  const cudaStream_t stream = (cudaStream_t)stream_;
  cb_status st = cb::check_attention(a);
  if (st != CB_OK) return st;
  if (a.num_reqs == 0 || a.num_tokens == 0) return CB_OK;
  if (cb::validate_enabled()) {
    st = cb::validate_attention_call(a, stream);
    if (st != CB_OK) return st;
  }
  bool decodes_left, prefills_left;
  st = cb::attend_packed(
      a, stream,
      [&](const cb::prefill_packed::Parts& parts, uint32_t* ew) { return cb::prefill_q4::launch(a, parts, ew, stream); },
      [&](const cb::decode::Scratch& scratch, uint32_t* ew, cb::decode::After after) {
        return cb::decode_q4::dispatch(a, scratch, ew, stream, after);
      },
      &decodes_left, &prefills_left);
  if (st != CB_OK || (!decodes_left && !prefills_left)) return st;
  const int nd = a.num_decodes;
  cb::q4::RowsParams p{};
  p.q = a.q;
  p.out = a.out;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens = a.seq_lens;
  p.block_tables = a.block_tables;
  p.row_begin = decodes_left ? 0 : nd;
  p.row_end = prefills_left ? a.num_reqs : nd;
  p.num_rows = a.num_reqs;
  p.num_decodes = a.num_decodes;
  p.num_tokens = a.num_tokens;
  p.num_blocks = a.num_blocks;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.window = a.sliding_window;
  p.error_word = static_cast<uint32_t*>(a.workspace);
  using namespace cb::q4;
  if (a.dtype == CB_DTYPE_F32)
    return a.head_dim == 64 ? launch_rows<float, 64>(p, stream) : launch_rows<float, 128>(p, stream);
  return a.head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(p, stream)
                          : launch_rows<__nv_bfloat16, 128>(p, stream);
}
