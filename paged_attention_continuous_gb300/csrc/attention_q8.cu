// cb_paged_attention_q8: paged attention over the 8-bit cache (e4m3 codes,
// one power-of-two scale for each (block, KV head)): checks and dispatch.
//
// The definition is cb_paged_attention's ("Chunked Prefill", How chunked
// prefill works) with key j of head g read as code * 2^ek(block, g) and
// value j as code * 2^ev(block, g).
#include <cuda_runtime.h>

#include "attention_common.h"
#include "cb_error.h"
#include "decode_q8.h"
#include "launch_common.h"
#include "prefill_q8.h"
#include "q8.cuh"
#include "rope.cuh"
#include "row_checks.h"
#include "validate.h"

namespace cb {
namespace q8 {

struct RowsParams {
  const void* q;
  void* out;
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  int64_t scale_stride;
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
  constexpr int kDPL = D / 32;
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
  const T* qrow = static_cast<const T*>(p.q) + ((int64_t)t * Hq + h) * D + lane * kDPL;
  float qf[kDPL], acc[kDPL];
#pragma unroll
  for (int e = 0; e < kDPL; ++e) {
    qf[e] = rope::to_float(qrow[e]) * p.scale_log2;
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  const int k_lo = p.window > 0 && pos + 1 > p.window ? pos + 1 - p.window : 0;
  for (int pg = k_lo / kPage; pg <= pos / kPage; ++pg) {
    const int blk = p.block_tables[(int64_t)r * p.max_blocks_per_seq + pg];
    if (blk < 0 || blk >= p.num_blocks) {
      if (lane == 0) set_error(p.error_word, CB_DEVERR_BLOCK_RANGE);
      continue;
    }
    const int64_t page = ((int64_t)blk * Hkv + g) * (kPage * D) + lane * kDPL;
    const float ks = exp2i(exp_of(p.k_scales[(int64_t)blk * p.scale_stride + g]));
    const float vs = exp2i(exp_of(p.v_scales[(int64_t)blk * p.scale_stride + g]));
    const int i1 = min(kPage, pos + 1 - pg * kPage);
    for (int i = max(0, k_lo - pg * kPage); i < i1; ++i) {
      const uint16_t* kr = reinterpret_cast<const uint16_t*>(p.k_cache + page + i * D);
      const uint16_t* vr = reinterpret_cast<const uint16_t*>(p.v_cache + page + i * D);
      float dot = 0.f;
#pragma unroll
      for (int e = 0; e < kDPL; e += 2) {
        const float2 k2 = floats2(kr[e / 2]);
        dot = fmaf(qf[e], k2.x, fmaf(qf[e + 1], k2.y, dot));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, o);
      dot *= ks;
      const float mn = fmaxf(m, dot);
      const float a = exp2f(m - mn), w = exp2f(dot - mn);
      l = l * a + w;
#pragma unroll
      for (int e = 0; e < kDPL; e += 2) {
        const float2 v2 = floats2(vr[e / 2]);
        acc[e] = fmaf(w, v2.x * vs, acc[e] * a);
        acc[e + 1] = fmaf(w, v2.y * vs, acc[e + 1] * a);
      }
      m = mn;
    }
  }
  T* orow = static_cast<T*>(p.out) + ((int64_t)t * Hq + h) * D + lane * kDPL;
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < kDPL; ++e) rope::from_float(orow + e, acc[e] * inv);
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
}  // namespace q8
}  // namespace cb

extern "C" cb_status cb_paged_attention_q8(const cb_attention_args* args, const uint8_t* k_scales,
                                           const uint8_t* v_scales, int64_t scale_stride,
                                           cb_stream_t stream_) {
  using cb::fail;
  if (!args) return fail(CB_ERR_INVALID_ARG, "args is NULL");
  const cb_attention_args& a = *args;
  const cudaStream_t stream = (cudaStream_t)stream_;
  cb_status st = cb::check_attention(a);
  if (st != CB_OK) return st;
  if (a.num_reqs == 0 || a.num_tokens == 0) return CB_OK;
  if (!k_scales || !v_scales) return fail(CB_ERR_INVALID_ARG, "NULL scales");
  if (scale_stride == 0) scale_stride = a.num_kv_heads;
  if (scale_stride < a.num_kv_heads)
    return fail(CB_ERR_INVALID_ARG, "scale_stride is less than num_kv_heads");
  if (cb::validate_enabled()) {
    st = cb::validate_attention_call(a, stream);
    if (st != CB_OK) return st;
  }
  // Decode rows run the split-KV kernel, the others the prefill kernel; what
  // those two do not take (KV heads shared by very many query heads; for
  // decodes more than 64 items to a split) runs the row kernel.  The prefill rows come first: the decode kernel then takes
  // the SMs that they leave, item by item, from the last wave's start on (96
  // decodes and 2.9k prompt tokens 218 us, 232 in the other order; with 512
  // tokens behind 4k 179 and 212, behind 15k 257 and 385; 64 decodes and 600
  // tokens 75 and 75).
  using cb::decode::After;
  uint32_t* ew = static_cast<uint32_t*>(a.workspace);
  const int nd = a.num_decodes;
  // Splits of few prefill rows leave their parts in the last places of the
  // workspace, at most half of them; the decodes' are the ones before.
  const cb::WsLayout L = cb::ws_layout(a.num_reqs, a.num_q_heads, a.num_kv_heads, a.head_dim);
  cb::decode::Scratch scratch = cb::decode_scratch(a, L);
  cb::prefill_q8::Parts parts{cb::prefill_q8::splits(a, L.slots / 2), nullptr, nullptr};
  if (parts.splits > 1) {
    scratch.slots -= (int64_t)a.num_tokens * parts.splits;
    parts.ml = scratch.part_ml + scratch.slots * a.num_q_heads * 2;
    parts.acc = scratch.part_acc + scratch.slots * a.num_q_heads * a.head_dim;
  }
  bool decodes_left = nd > 0, prefills_left = nd < a.num_reqs;
  if (prefills_left) {
    st = cb::prefill_q8::launch(a, k_scales, v_scales, scale_stride, parts, ew, stream);
    if (st != CB_OK && st != CB_ERR_UNSUPPORTED) return st;
    prefills_left = st != CB_OK;
  }
  const bool prefilled = nd < a.num_reqs && !prefills_left;
  if (decodes_left) {
    const After after = prefilled ? After::kPrefill : a.after_append ? After::kAppend : After::kStream;
    st = cb::decode_q8::dispatch(a, k_scales, v_scales, scale_stride, scratch, ew, stream, after);
    if (st != CB_OK && st != CB_ERR_UNSUPPORTED) return st;
    decodes_left = st != CB_OK;
  }
  if (prefilled && parts.splits > 1) {
    st = cb::prefill_q8::join(a, parts, stream);
    if (st != CB_OK) return st;
  }
  if (!decodes_left && !prefills_left) return CB_OK;
  cb::q8::RowsParams p{};
  p.q = a.q;
  p.out = a.out;
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.scale_stride = scale_stride;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens = a.seq_lens;
  p.block_tables = a.block_tables;
  p.row_begin = decodes_left ? 0 : nd;
  p.row_end = prefills_left ? a.num_reqs : nd;
  p.num_rows = a.num_reqs;
  p.num_decodes = nd;
  p.num_tokens = a.num_tokens;
  p.num_blocks = a.num_blocks;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.window = a.sliding_window;
  p.error_word = static_cast<uint32_t*>(a.workspace);
  using namespace cb::q8;
  if (a.dtype == CB_DTYPE_F32)
    return a.head_dim == 64 ? launch_rows<float, 64>(p, stream) : launch_rows<float, 128>(p, stream);
  return a.head_dim == 64 ? launch_rows<__nv_bfloat16, 64>(p, stream)
                          : launch_rows<__nv_bfloat16, 128>(p, stream);
}
