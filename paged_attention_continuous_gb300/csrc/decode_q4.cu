// Split-KV decode over the 4-bit cache: instantiations and launch.
#include "decode_q4.h"

#include <atomic>

#include "cb_error.h"
#include "decode_q4.cuh"
#include "launch_common.h"

namespace cb {
namespace decode_q4 {

namespace {

constexpr size_t kSmemLimit = 226 * 1024;  // of 227 KB; the plan has static words too

// Stages of a warp, and pages of a stage.
constexpr int kStages = 2, kPages = 4;

// Warps of a CTA: by the registers of an item's outputs and queries, what leaves
// none of a warp's others in memory.  Measured, 8 KV heads, 12 warps / 8: 64
// requests of up to 8k tokens, 32 bfloat16 heads of 64 dims (24 registers) 53.5 / 60
// us, float32 (32) 61.7 / 70, 128 bfloat16 heads of 64 (48) 71.4 / 75.5.  128
// requests of up to 32k tokens, 64 float32 heads of 128 dims (64) 714 / 553, 128
// bfloat16 heads of 128 (96) 801 / 592.  (Three stages are no faster, stages of two
// pages slower.)
template <typename T, int D, int kNT>
struct Shape {
  static constexpr int kRegs = D * kNT / 4 + D * kNT / 8 * (int)(sizeof(T) / 2);
  static constexpr int kWarps = kRegs < 64 ? 12 : 8;
};

template <typename T, int D, int kNT, int kWarps>
cb_status launch(const cb_attention_args& a, int parts, int part_heads, const decode::Scratch& s,
                 uint32_t* error_word, cudaStream_t stream, decode::After after) {
  using Lay = Layout<D, kStages, kPages, kWarps>;
  auto kern = decode_kernel<T, D, kNT, kWarps, kStages, kPages>;
  constexpr size_t smem = Lay::total;
  static_assert(smem <= kSmemLimit, "decode stages do not fit shared memory");
  static std::atomic<uint8_t> attr_set[kMaxDevices];
  cb_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), smem, attr_set);
  if (st != CB_OK) return st;
  Params p{};
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
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

cb_status dispatch(const cb_attention_args& a, const decode::Scratch& s, uint32_t* error_word,
                   cudaStream_t stream, decode::After after) {
  const int G = a.num_q_heads / a.num_kv_heads;
  // query heads of an item: 16, but 8 where the outputs and the queries' two
  // pieces of 16 heads would pass the registers
  const int most = a.dtype == CB_DTYPE_F32 && a.head_dim == 128 ? 8 : 16;
  const int parts = (G + most - 1) / most;
  const int heads = (G + parts - 1) / parts;  // of a part
  if (a.num_kv_heads * parts > 64) return CB_ERR_UNSUPPORTED;  // tickets, and the plan's divisions
  if ((int64_t)a.num_blocks * a.num_kv_heads >= ((int64_t)1 << 31)) return CB_ERR_UNSUPPORTED;
  // Few pages (at most this many of all KV heads' together) are read sooner by
  // eight warps with more registers: 8 requests of up to 512 tokens 12.0 us, 13.5
  // with twelve, 16 of up to 2k 17.3 / 18.9, 8 of up to 8k 24.2 / 27.4; 64 of up to
  // 4k 51.7 / 49.4.  (Twelve beside a prefill grid, where long rows beside long
  // chunks want them: 96 of up to 8k and 512 tokens behind 4k 159 / 154; with 512
  // fresh tokens 16 of up to 4k take 38 / 40, 2 of 8k 28 / 31.)
  // The lengths are the caller's bound: a captured step declares its table's
  // width, and with one of 128k tokens these few take 13.5, 19.4 and 30 us.
  const int64_t pages = (int64_t)a.num_decodes * a.num_kv_heads * parts * blocks_of(a.max_seq_len, q4::kPage);
  const bool few = pages <= 32768 && after != decode::After::kPrefill;
#define CB_DEC(T, DD, NT)                                                                          \
  if (a.head_dim == DD && (heads > 8) == (NT == 2))                                                \
    return few ? launch<T, DD, NT, 8>(a, parts, heads, s, error_word, stream, after)               \
               : launch<T, DD, NT, Shape<T, DD, NT>::kWarps>(a, parts, heads, s, error_word, stream, after);
  if (a.dtype == CB_DTYPE_F32) {
    CB_DEC(float, 64, 1) CB_DEC(float, 64, 2) CB_DEC(float, 128, 1)
  } else {
    CB_DEC(__nv_bfloat16, 64, 1) CB_DEC(__nv_bfloat16, 64, 2)
    CB_DEC(__nv_bfloat16, 128, 1) CB_DEC(__nv_bfloat16, 128, 2)
  }
#undef CB_DEC
  return CB_ERR_UNSUPPORTED;
}

}  // namespace decode_q4
}  // namespace cb
