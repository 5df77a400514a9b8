// Split-KV decode over the 8-bit cache: instantiations and launch.
#include "decode_q8.h"

#include <atomic>

#include "cb_error.h"
#include "decode_q8.cuh"
#include "launch_common.h"
#include "tensor_map.h"

namespace cb {
namespace decode_q8 {

namespace {

constexpr size_t kSmemLimit = 226 * 1024;  // of 227 KB; the plan has static words too

template <typename T, int D, int kNT>
cb_status launch(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                 int64_t scale_stride, int parts, int part_heads, const decode::Scratch& s,
                 uint32_t* error_word, cudaStream_t stream, decode::After after) {
  // Two stages of two pages to a warp keep 128 KB of an SM in flight with 128
  // dims, 64 KB with 64.  More change little: 64 requests of up to 4k tokens,
  // 128 dims 63.3 us with two and 64.0 with three, 64 dims 54.0 and 53.6 with
  // four; 128 of up to 32k tokens 636 and 633, 64 dims 513 and 507; float32
  // queries 72.4 and 73.1, 707 and 712.
  constexpr int kStages = 2;
  using Lay = Layout<D, kStages>;
  auto kern = decode_kernel<T, D, kNT, kStages>;
  constexpr size_t smem = Lay::total(kWarps);
  static_assert(smem <= kSmemLimit, "decode stages do not fit shared memory");
  static std::atomic<uint8_t> attr_set[kMaxDevices];
  cb_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem, attr_set);
  if (st != CB_OK) return st;
  Params p{};
  const int64_t rows = (int64_t)a.num_blocks * a.num_kv_heads * kPageTokens;
  st = cached_cache_map(&p.tmap_k, a.k_cache, rows, D, 1);
  if (st != CB_OK) return st;
  st = cached_cache_map(&p.tmap_v, a.v_cache, rows, D, 1);
  if (st != CB_OK) return st;
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.scale_stride = scale_stride;
  p.q = a.q;
  p.out = a.out;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens = a.seq_lens;
  p.block_tables = a.block_tables;
  p.num_tokens = a.num_tokens;
  p.num_blocks = a.num_blocks;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.parts = parts;
  p.part_heads = part_heads;
  const double scale_log2 = (double)a.scale * 1.4426950408889634;
  p.scale_log2 = (float)scale_log2;
  p.scale_log2_low = p.scale_log2 != 0.f ? (float)((scale_log2 - p.scale_log2) / p.scale_log2) : 0.f;
  p.window = a.sliding_window;
  p.error_word = error_word;
  p.work_counter = s.work_counter;
  p.done = s.done;
  p.max_slots = (int32_t)(s.slots < (1 << 30) ? s.slots : (1 << 30));
  p.part_ml = s.part_ml;
  p.part_acc = s.part_acc;
  p.wait_ns = wait_limit_ns();
  p.withhold_item = withheld_decode_item();
  for (int r0 = 0; r0 < a.num_decodes; r0 += decode::kPlanMax) {
    p.row_begin = r0;
    p.num_rows = a.num_decodes - r0 < decode::kPlanMax ? a.num_decodes - r0 : decode::kPlanMax;
    // the first launch may overlap the kernel queued just before it; later
    // ones share this call's workspace with the one before and follow it
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)sm_count_current_device(), 1, 1);
    cfg.blockDim = dim3(kWarps * 32, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    const decode::After mode = r0 == 0 ? after : decode::After::kStream;
    p.pdl_mode = (int32_t)mode;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = mode != decode::After::kStream ? 1 : 0;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess) return fail(CB_ERR_CUDA, "decode kernel launch: %s", cudaGetErrorString(e));
  }
  return CB_OK;
}

}  // namespace

cb_status dispatch(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                   int64_t scale_stride, const decode::Scratch& s, uint32_t* error_word,
                   cudaStream_t stream, decode::After after) {
  const int G = a.num_q_heads / a.num_kv_heads;
  const int parts = (G + kMaxHeads - 1) / kMaxHeads;
  const int heads = (G + parts - 1) / parts;  // of a part
  if (a.num_kv_heads * parts > 64) return CB_ERR_UNSUPPORTED;  // tickets, and the plan's divisions
  if ((int64_t)a.num_blocks * a.num_kv_heads * kPageTokens >= ((int64_t)1 << 31)) return CB_ERR_UNSUPPORTED;
#define CB_DEC(T, DD, NT)                                                                        \
  if (a.head_dim == DD && (heads > 8) == (NT == 2))                                              \
    return launch<T, DD, NT>(a, k_scales, v_scales, scale_stride, parts, heads, s, error_word, stream, after);
  if (a.dtype == CB_DTYPE_F32) {
    CB_DEC(float, 64, 1) CB_DEC(float, 64, 2) CB_DEC(float, 128, 1) CB_DEC(float, 128, 2)
  } else {
    CB_DEC(__nv_bfloat16, 64, 1) CB_DEC(__nv_bfloat16, 64, 2)
    CB_DEC(__nv_bfloat16, 128, 1) CB_DEC(__nv_bfloat16, 128, 2)
  }
#undef CB_DEC
  return CB_ERR_UNSUPPORTED;
}

}  // namespace decode_q8
}  // namespace cb
