// Prefill-chunk attention over the 8-bit cache on tcgen05 tensor cores.
//
// The definition is the prefill kernel's ("Chunked Prefill", How chunked
// prefill works): query i of a chunk that starts at position s attends keys
// 0..s+i (with a window W the last W of them), key j of KV head g being code
// * 2^ek(block, g) and value j code * 2^ev(block, g).
//
// One CTA = (prefill row, KV head, a pair of 128-row query tiles); a tile
// packs floor(128 / G) tokens x the G query heads of the KV head.  Keys
// stream in tiles of 128 (eight blocks).  The tensor cores bound it (4 D
// FLOP for each query head and visible key); the codes ask for what the
// 16-bit kernel does not have:
//
//   * Four converter warps read the pages' codes from global memory into
//     registers, a tile ahead, expand them to halves (every e4m3 number is
//     one exactly: one conversion for two codes) and store them in the
//     swizzled layout that the matrix instructions read.  No raw codes pass
//     through shared memory.
//   * Both products are kind::f16 with half operands: Q rows are scaled by a
//     power of two to the halves' range (so bfloat16 queries are halves
//     exactly; elements under 2^-29 of the row's largest lose bits).
//   * The scales stay out of the operands.  A score's factor is its block's
//     2^ek times the row's; a weight is 2^(x + ev - m) with x the score in
//     powers of two, so that weight times code is the value's part, and the
//     running reference m is over x + ev.  The sum of weights adds each
//     block's sum times 2^-ev.  Weights are halves: scores go through
//     ex2.f16x2 (an exponent in [-8, 8] is off by 2^-9 at most), 8 times
//     finer than bfloat16 exponents for the same instructions.  A weight
//     below 2^-24 is zero; a block whose values are more than 2^4 smaller
//     than the largest so far gets its part of the sum from float32
//     exponentials instead, where x counts and x + ev does not.
//   * float32 queries: Q and the weights are split into two halves each (22
//     bits), one query tile per CTA (the second tile's place holds the low
//     halves), float32 exponentials.
//   * A value code that is NaN must not reach rows that do not see its key
//     (weight 0 times NaN is NaN): in tiles that some row of the CTA sees only
//     in part, converters store such codes as 0 and note the first and last
//     key for each dim; the epilogue writes NaN where a row sees one.
//
// Tensor memory: S0 | S1 | O0 | O1 at columns 0, 128, 256, 384; P_t is
// written over S_t as half pairs and read from there as the A operand.
//
// Warp roles (512 threads, registers redistributed):
//   0-3 / 4-7  softmax of query tile 0 / 1 (thread = row): 184 registers
//   10, 11     MMA issuers of the two tiles (8, 9 idle; 10 owns TMEM): 48
//   12-15      converters: 96
// Per KV tile j an issuer queues P.V(j-1) and then Q.K(j).  Every wait is
// bounded (CB_DEVERR_TIMEOUT).
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "cb_error.h"
#include "device_utils.cuh"
#include "launch_common.h"
#include "mma_utils.cuh"
#include "prefill_q8.h"
#include "q8.cuh"
#include "rope.cuh"
#include "tcgen05.cuh"

namespace cb {
namespace prefill_q8 {

constexpr int kBM = 128;            // query rows per tile
constexpr int kBN = 128;            // keys per KV tile
constexpr int kPage = 16;
constexpr int kPages = kBN / kPage; // blocks of a KV tile
constexpr int kStagesK = 3;
constexpr int kStagesV = 2;
constexpr int kScaleSlots = 8;      // tiles whose scales are kept (see below)
constexpr int kMmaWarp = 10;
constexpr int kConvWarp = 12;
constexpr int kThreads = 512;
constexpr int kRegsSoftmax = 184, kRegsMma = 48, kRegsConv = 96;
static_assert(128 * (2 * kRegsSoftmax + kRegsMma + kRegsConv) <= 65536, "register split");
constexpr uint32_t kHalf = 128 * 128;  // 128 rows of 64 halves
constexpr uint32_t kTmemCols = 512;
constexpr float kTop = 4.f;         // weight exponent at the reference
constexpr float kLag = 4.f;         // the reference moves when passed by more
constexpr float kSpread = 4.f;      // value exponents this far below the largest: float32 sums
__host__ __device__ constexpr uint32_t col_s(int t) { return t ? 128u : 0u; }
__host__ __device__ constexpr uint32_t col_o(int t) { return t ? 384u : 256u; }

struct Bars {
  uint64_t k_full[kStagesK];   // K tile expanded (one arrival per converter warp)
  uint64_t v_full[kStagesV];
  uint64_t k_empty[kStagesK];  // last Q.K of the stage done
  uint64_t v_empty[kStagesV];  // last P.V of the stage done
  uint64_t s_full[2], p_full[2], o_done[2], drain[2];
  uint32_t tmem_base, abort;
  int32_t row, pair;
  // factor 2^ek and exponent ev of the blocks of recent KV tiles: the slot of
  // tile j is rewritten for tile j + 8, which is expanded only after Q.K(j +
  // 5), and that only after the softmax of tile j + 4
  float ks[kScaleSlots][kPages];
  float ev[kScaleSlots][kPages];
  int32_t nan_first[128], nan_last[128];  // by dim: keys whose value is NaN
};

template <int D>
struct Smem {
  static constexpr uint32_t kTile = kBM * D * 2;  // Q, K or V tile of halves
  static constexpr uint32_t q = 0;                // Q0 | Q1 (float32: high | low)
  static constexpr uint32_t k = q + 2 * kTile;
  static constexpr uint32_t v = k + kStagesK * kTile;
  static constexpr uint32_t bars = v + kStagesV * kTile;
  static constexpr uint32_t total = bars + sizeof(Bars) + 1024;  // + alignment of the base
};
static_assert(Smem<128>::total <= 227 * 1024, "shared memory");

struct Params {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  int64_t scale_stride;
  const void* q;
  void* out;
  const int32_t* cu_seqlens_q;
  const int32_t* seq_lens;
  const int32_t* block_tables;
  int32_t row_begin, num_rows, num_tokens;
  int32_t num_blocks, max_blocks_per_seq, num_q_heads, num_kv_heads, group;
  float scale_log2;
  int32_t window;
  uint32_t* error_word;
  uint64_t wait_ns;
  int32_t withhold_tile;      // test hook: CTA 0 never announces this K tile (-1: none)
};

__device__ __forceinline__ void abort_cta(Bars* B, uint32_t* error_word) {
  if (atomicExch(&B->abort, 1u) == 0u) set_error(error_word, CB_DEVERR_TIMEOUT);
}

__device__ __forceinline__ bool wait_or_abort(uint64_t* bar, uint32_t parity, Bars* B,
                                              uint32_t* error_word, uint64_t limit_ns) {
  if (mbar_wait(bar, parity, limit_ns)) return true;
  abort_cta(B, error_word);
  return false;
}

// 2^x of a pair of halves; 2^-inf = 0
__device__ __forceinline__ uint32_t ex2_f16x2(uint32_t x) {
  uint32_t y;
  asm("ex2.approx.f16x2 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint32_t add_f16x2(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("add.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}
__device__ __forceinline__ uint32_t halves(float lo, float hi) {
  return decode::as_u32(__floats2half2_rn(lo, hi));
}
__device__ __forceinline__ float2 floats(uint32_t h) {
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t swz(uint32_t row, uint32_t chunk) {
  return row * 128u + ((chunk ^ (row & 7u)) << 4);
}
__device__ __forceinline__ uint4 ld_codes(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ void order_after_previous_grid() {
  if (blockIdx.x == 0 && threadIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Any e4m3 NaN (0x7f or 0xff) among four codes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1) prefill_kernel(const __grid_constant__ Params p) {
  constexpr bool kF32 = std::is_same<T, float>::value;
  constexpr int kTiles = kF32 ? 1 : 2;            // query tiles of a CTA
  constexpr uint32_t kTile = Smem<D>::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  Bars* B = reinterpret_cast<Bars*>(smem + Smem<D>::bars);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  // the decode rows of the same call, when launched after this grid with
  // programmatic serialization, may start at once on the SMs it leaves idle
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int G = p.group;
  const int tpt = kBM / G;                        // tokens per query tile
  const int tpp = kTiles * tpt;                   // of a CTA
  const int Hkv = p.num_kv_heads;
  const int g = (int)(blockIdx.x % (unsigned)Hkv);
  // ---- which (row, pair) this CTA serves: warp 0 scans the rows' pair
  // counts; every row's latest (heaviest) pair comes first
  if (warp == 0) {
    const int x = (int)(blockIdx.x / (unsigned)Hkv);
    const int num_pairs = (int)(gridDim.x / (unsigned)Hkv);
    int run = 0, row = -1, pair = 0;
    bool bad = false;
    for (int b = 0; b < p.num_rows; b += 32) {
      const int i = b + lane;
      int cnt = 0;
      if (i < p.num_rows) {
        const int rr = p.row_begin + i;
        const int ql = p.cu_seqlens_q[rr + 1] - p.cu_seqlens_q[rr];
        if (ql < 0 || (ql == 0 && p.seq_lens[rr] != 0)) bad = true;
        cnt = ql > 0 ? (ql + tpp - 1) / tpp : 0;
      }
      int incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      const bool mine = cnt > 0 && x >= run + incl - cnt && x < run + incl;
      const uint32_t hit = __ballot_sync(0xffffffffu, mine);
      if (hit) {
        const int src = __ffs(hit) - 1;
        row = __shfl_sync(0xffffffffu, i, src);
        const int first = __shfl_sync(0xffffffffu, run + incl - cnt, src);
        const int n = __shfl_sync(0xffffffffu, cnt, src);
        pair = n - 1 - (x - first);
      }
      run += __shfl_sync(0xffffffffu, incl, 31);
    }
    bad = __any_sync(0xffffffffu, bad) || run > num_pairs;
    if (lane == 0) {
      if (bad && blockIdx.x == 0) set_error(p.error_word, CB_DEVERR_SEQ_RANGE);
      B->row = row;
      B->pair = pair;
    }
  }
  __syncthreads();
  if (B->row < 0) {                               // past the last pair
    order_after_previous_grid();
    return;
  }
  const int r = p.row_begin + B->row;
  const int mp = B->pair;
  const int q0 = p.cu_seqlens_q[r];
  const int q_len = p.cu_seqlens_q[r + 1] - q0;
  const int L = p.seq_lens[r];
  const int W = p.max_blocks_per_seq;
  if (q0 < 0 || q0 + q_len > p.num_tokens || L < q_len || (L + kPage - 1) / kPage > W) {
    if (threadIdx.x == 0 && mp == 0 && g == 0) set_error(p.error_word, CB_DEVERR_SEQ_RANGE);
    order_after_previous_grid();
    return;
  }
  const int tok0 = mp * tpp;                      // first token of the CTA
  const bool has_t1 = kTiles == 2 && tok0 + tpt < q_len;
  const int start = L - q_len;
  const int last_tok = min(tok0 + tpp - 1, q_len - 1);
  const int n_tiles = (start + last_tok) / kBN + 1;
  const int npages = (L + kPage - 1) / kPage;
  // with a window, the first query reads keys from key_lo on: KV tiles j_lo ..
  const int key_lo = p.window > 0 ? max(0, start + tok0 - p.window + 1) : 0;
  const int j_lo = key_lo / kBN;
  const int lo_pg = key_lo / kPage;
  const int nt = n_tiles - j_lo;

  if (threadIdx.x == 0) {
    const uint32_t issuers = has_t1 ? 2u : 1u;
    for (int s = 0; s < kStagesK; ++s) {
      mbar_init(&B->k_full[s], 4);
      mbar_init(&B->k_empty[s], issuers);
    }
    for (int s = 0; s < kStagesV; ++s) {
      mbar_init(&B->v_full[s], 4);
      mbar_init(&B->v_empty[s], issuers);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&B->s_full[t], 1);
      mbar_init(&B->p_full[t], 4);
      mbar_init(&B->o_done[t], 1);
      mbar_init(&B->drain[t], 1);
    }
    B->abort = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < 128) {
    B->nan_first[threadIdx.x] = 0x7fffffff;
    B->nan_last[threadIdx.x] = -1;
  }
  if (warp == kMmaWarp) {
    tc::tmem_alloc(&B->tmem_base, kTmemCols);
    tc::tmem_relinquish();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = B->tmem_base;

  if (warp >= kConvWarp) {
    // ------------------------------------------------------------ converters
    tc::regs_dec<kRegsConv>();
    // Thread ct of 128 owns a 16-byte chunk of a page row: D = 128, one page
    // a round; D = 64, two.
    constexpr int kChunks = D / 16;                // chunks of a row
    constexpr int kPerRound = 128 / (kPage * kChunks);  // pages of a round
    constexpr int kRounds = kPages / kPerRound;
    const int ct = threadIdx.x - kConvWarp * 32;
    const int c = ct % kChunks, prow = ct / kChunks % kPage, psub = ct / (kChunks * kPage);
    // the lane's two 16-byte stores: dims 16 c .. 16 c + 7 and the next 8; at
    // D = 128 the upper half's lanes store theirs in the other order, so that
    // the 8 lanes of a row never meet in a bank
    const int first = D == 128 ? c >> 2 : 0;
    const uint32_t hbase = (uint32_t)(c / 4) * kHalf;
    const int ch0 = (2 * c + first) & 7, ch1 = (2 * c + 1 - first) & 7;
    auto page_of = [&](int j, int i) { return j * kPages + i; };
    // lane i < 8: block of page i of tile j (-1: none, read as zeros)
    auto block_ids = [&](int j) {
      const int pg = page_of(j, lane);
      const bool in = lane < kPages && j < n_tiles && pg < npages && pg >= lo_pg;
      int b = in ? __ldg(p.block_tables + (int64_t)r * W + pg) : -1;
      if (in && (b < 0 || b >= p.num_blocks)) {
        b = -1;
        set_error(p.error_word, CB_DEVERR_BLOCK_RANGE);
      }
      return b;
    };
    auto load = [&](const uint8_t* cache, int ids, uint4* raw) {
#pragma unroll
      for (int i = 0; i < kRounds; ++i) {
        const int b = __shfl_sync(0xffffffffu, ids, i * kPerRound + psub);
        raw[i] = b >= 0 ? ld_codes(cache + ((int64_t)b * Hkv + g) * (kPage * D) + prow * D + c * 16)
                        : make_uint4(0, 0, 0, 0);
      }
    };
    auto store = [&](uint8_t* tile, int i, uint4 w) {
      const uint32_t row = (uint32_t)((i * kPerRound + psub) * kPage + prow);
      uint4 a, b;
      q8::halves4(w.x, a.x, a.y);
      q8::halves4(w.y, a.z, a.w);
      q8::halves4(w.z, b.x, b.y);
      q8::halves4(w.w, b.z, b.w);
      uint8_t* base = tile + hbase;
      *reinterpret_cast<uint4*>(base + swz(row, ch0)) = first ? b : a;
      *reinterpret_cast<uint4*>(base + swz(row, ch1)) = first ? a : b;
    };
    uint4 kr[kRounds], vr[kRounds];
    int ids = block_ids(j_lo);
    load(p.k_cache, ids, kr);
    load(p.v_cache, ids, vr);
    bool ok = true;
    for (int jj = 0; jj < nt && ok; ++jj) {
      const int j = j_lo + jj;
      const int next = block_ids(j + 1);
      // scales of this tile: lane i < 8 its K scale, lane 8 + i its V scale
      int e = 0;
      {
        // (a block that is not read takes the first one's that is, so that it
        // does not widen the tile's range of exponents)
        const uint32_t read = __ballot_sync(0xffffffffu, ids >= 0) & 0xffu;
        const int own = __shfl_sync(0xffffffffu, ids, lane & 7);
        const int any = __shfl_sync(0xffffffffu, ids, read ? __ffs(read) - 1 : 0);
        const int b = own >= 0 ? own : any;
        if (warp == kConvWarp && lane < 2 * kPages && b >= 0)
          e = q8::exp_of((lane < kPages ? p.k_scales : p.v_scales)[(int64_t)b * p.scale_stride + g]);
      }
      // ---- K
      const int sk = jj % kStagesK;
      if (jj >= kStagesK) {
        ok = __all_sync(0xffffffffu, mbar_wait(&B->k_empty[sk], ((jj / kStagesK) - 1) & 1, p.wait_ns));
        if (!ok) { abort_cta(B, p.error_word); break; }
      }
      if (*reinterpret_cast<volatile uint32_t*>(&B->abort)) break;
      uint8_t* kt = smem + Smem<D>::k + sk * kTile;
#pragma unroll
      for (int i = 0; i < kRounds; ++i) store(kt, i, kr[i]);
      if (warp == kConvWarp && lane < 2 * kPages) {
        if (lane < kPages) B->ks[jj % kScaleSlots][lane] = q8::exp2i(e);
        else B->ev[jj % kScaleSlots][lane - kPages] = (float)e;
      }
      fence_proxy_async_smem();
      __syncwarp();
      // test hook: the withheld tile is never announced, so the bounded waits
      // on it run out
      if (lane == 0 && !(blockIdx.x == 0 && jj == p.withhold_tile)) mbar_arrive(&B->k_full[sk]);
      load(p.k_cache, next, kr);                   // in flight while V is expanded
      // ---- V
      const int sv = jj % kStagesV;
      if (jj >= kStagesV) {
        ok = __all_sync(0xffffffffu, mbar_wait(&B->v_empty[sv], ((jj / kStagesV) - 1) & 1, p.wait_ns));
        if (!ok) { abort_cta(B, p.error_word); break; }
      }
      uint8_t* vt = smem + Smem<D>::v + sv * kTile;
      const int kbase = j * kBN;
      const int end = L - kbase;                   // rows past the sequence become zeros
      // some row of the CTA does not see all keys of this tile
      const bool part = kbase + kBN - 1 > start + tok0 ||
                        (p.window > 0 && kbase < start + last_tok - p.window + 1);
      if (!part) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) store(vt, i, vr[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          const int row = (i * kPerRound + psub) * kPage + prow;
          uint4 w = vr[i];
          if (row >= end) w = make_uint4(0, 0, 0, 0);
          if (nan_codes(w.x) | nan_codes(w.y) | nan_codes(w.z) | nan_codes(w.w)) {
            uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int b = 0; b < 16; ++b)
              if (((x[b >> 2] >> (8 * (b & 3))) & 0x7fu) == 0x7fu) {
                x[b >> 2] &= ~(0xffu << (8 * (b & 3)));
                atomicMin(&B->nan_first[16 * c + b], kbase + row);
                atomicMax(&B->nan_last[16 * c + b], kbase + row);
              }
            w = make_uint4(x[0], x[1], x[2], x[3]);
          }
          store(vt, i, w);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->v_full[sv]);
      load(p.v_cache, next, vr);
      ids = next;
    }
  } else if (warp >= 8) {
    // ------------------------------------------------------------------ MMA
    tc::regs_dec<kRegsMma>();
    if (warp >= kMmaWarp) {
      asm volatile("bar.sync 1, 320;" ::: "memory");  // Q is in shared memory
      tc::fence_after_sync();
      const int t = warp - kMmaWarp;
      if (lane == 0 && (t == 0 || has_t1)) {
        constexpr uint32_t idesc_qk = tc::idesc_f16_f32(kBM, kBN, 0);
        constexpr uint32_t idesc_pv = tc::idesc_f16_f32(kBM, D, 1);
        const uint64_t aq = tc::smem_desc_sw128(smem_addr(smem + Smem<D>::q) + t * kTile, 16, 1024);
        const uint64_t dk0 = tc::smem_desc_sw128(smem_addr(smem + Smem<D>::k), 16, 1024);
        const uint64_t dv0 = tc::smem_desc_sw128(smem_addr(smem + Smem<D>::v), kHalf, 1024);
        constexpr uint32_t kTileDesc = kTile >> 4;
        bool ok = true;
        for (int jj = 0; jj <= nt && ok; ++jj) {
          if (jj >= 1) {
            const int jr = jj - 1, sp = jr % kStagesV;
            ok = wait_or_abort(&B->p_full[t], jr & 1, B, p.error_word, p.wait_ns) &&
                 wait_or_abort(&B->v_full[sp], (jr / kStagesV) & 1, B, p.error_word, p.wait_ns);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t bv = dv0 + sp * kTileDesc;
#pragma unroll
            for (int piece = 0; piece < (kF32 ? 2 : 1); ++piece)
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk)
                tc::mma_f16_ts(tmem + col_o(t), tmem + col_s(t) + piece * 64 + kk * 8, bv + (kk * 2048 >> 4),
                               idesc_pv, (jr > 0 || kk > 0 || piece > 0) ? 1u : 0u);
            tc::mma_commit(&B->v_empty[sp]);
            if (jj == nt) tc::mma_commit(&B->o_done[t]);
          }
          if (jj < nt) {
            const int s = jj % kStagesK;
            ok = wait_or_abort(&B->k_full[s], (jj / kStagesK) & 1, B, p.error_word, p.wait_ns);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t bk = dk0 + s * kTileDesc;
#pragma unroll
            for (int piece = 0; piece < (kF32 ? 2 : 1); ++piece)
#pragma unroll
              for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                tc::mma_f16(tmem + col_s(t), aq + piece * kTileDesc + off, bk + off, idesc_qk,
                            (kk > 0 || piece > 0) ? 1u : 0u);
              }
            tc::mma_commit(&B->s_full[t]);
            tc::mma_commit(&B->k_empty[s]);
          }
        }
        // drain: all issued MMAs complete before tensor memory is released
        tc::mma_commit(&B->drain[t]);
        mbar_wait(&B->drain[t], 0, p.wait_ns);
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    tc::regs_inc<kRegsSoftmax>();
    const int t = warp >> 2;                      // query tile
    const int row = threadIdx.x & 127;            // == TMEM lane
    const int tl = row / G;
    const int tok = tok0 + t * tpt + tl;
    const int head = g * G + (row - tl * G);
    const bool valid = t < kTiles && tl < tpt && tok < q_len;
    const int pos = start + (valid ? tok : q_len - 1);
    float hs = 1.f;                               // score factor of the row
    if (t < kTiles) {
      // Q row -> halves in shared memory, the largest magnitude at [2^14,
      // 2^15); the scale's sign goes with Q, and a scale of 0 makes Q zero
      const T* src = static_cast<const T*>(p.q) + ((int64_t)(q0 + (valid ? tok : q_len - 1)) * p.num_q_heads +
                                                   (valid ? head : g * G)) * D;
      float amax = 0.f;
      if (valid) {
#pragma unroll 4
        for (int i = 0; i < D / 8; ++i) {
          float x[8];
          if constexpr (kF32) {
            rope::Vec<float>::load(__ldg(reinterpret_cast<const uint4*>(src) + 2 * i), x);
            rope::Vec<float>::load(__ldg(reinterpret_cast<const uint4*>(src) + 2 * i + 1), x + 4);
          } else {
            rope::Vec<__nv_bfloat16>::load(__ldg(reinterpret_cast<const uint4*>(src) + i), x);
          }
#pragma unroll
          for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
        }
      }
      // zeros, or a row that is not finite (nor are its scores): factor 1
      const int k = amax > 0.f && amax <= 3.402823466e38f ? max((int)(__float_as_uint(amax) >> 23) - 127, -110) : 14;
      const float up = p.scale_log2 == 0.f ? 0.f : p.scale_log2 < 0.f ? -q8::exp2i(14 - k) : q8::exp2i(14 - k);
      hs = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2) * q8::exp2i(k - 14);
      uint8_t* qs = smem + Smem<D>::q + t * kTile;
#pragma unroll 4
      for (int i = 0; i < D / 8; ++i) {
        float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (valid) {
          if constexpr (kF32) {
            rope::Vec<float>::load(__ldg(reinterpret_cast<const uint4*>(src) + 2 * i), x);
            rope::Vec<float>::load(__ldg(reinterpret_cast<const uint4*>(src) + 2 * i + 1), x + 4);
          } else {
            rope::Vec<__nv_bfloat16>::load(__ldg(reinterpret_cast<const uint4*>(src) + i), x);
          }
        }
        uint32_t h[4], lo[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[2 * e] * up, b = x[2 * e + 1] * up;
          h[e] = halves(a, b);
          const float2 f = floats(h[e]);
          lo[e] = halves(a - f.x, b - f.y);
        }
        const uint32_t at = (i >> 3) * kHalf + swz(row, i & 7);
        *reinterpret_cast<uint4*>(qs + at) = make_uint4(h[0], h[1], h[2], h[3]);
        if constexpr (kF32) *reinterpret_cast<uint4*>(qs + kTile + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
      }
      fence_proxy_async_smem();
    }
    asm volatile("bar.sync 1, 320;" ::: "memory");
    const bool active = t == 0 || has_t1;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t colS = col_s(t), colO = col_o(t);
    float m_run = -INFINITY, l_run = 0.f, e_run = -INFINITY;
    bool ok = active;
    // keys before key_row are outside this row's window
    const int key_row = p.window > 0 ? pos - p.window + 1 : -(1 << 30);
    for (int jj = 0; jj < nt && ok; ++jj) {
      // the two warpgroups take turns, so that each runs alone on the SM's
      // exponential and FMA units while the tensor core works for the other
      if (has_t1 && (t == 1 || jj >= 1)) {
        const bool tw = __all_sync(0xffffffffu, t == 0 ? mbar_wait(&B->p_full[1], (jj - 1) & 1, p.wait_ns)
                                                     : mbar_wait(&B->p_full[0], jj & 1, p.wait_ns));
        if (!tw) { abort_cta(B, p.error_word); ok = false; break; }
      }
      // S(j) ready implies that the tile's scales are in shared memory: they
      // were stored before the arrivals that the issuer waited for
      const bool w = __all_sync(0xffffffffu, mbar_wait(&B->s_full[t], jj & 1, p.wait_ns));
      if (!w) { abort_cta(B, p.error_word); ok = false; break; }
      tc::fence_after_sync();
      const int kbase = (j_lo + jj) * kBN;
      const int lim = pos - kbase;                // key kbase+i visible iff lo <= i <= lim
      const int lo = key_row - kbase;
      float sv[kBN];
#pragma unroll
      for (int c = 0; c < kBN / 32; ++c) tc::tmem_ld32(trow + colS + 32 * c, sv + 32 * c);
      tc::tmem_wait_ld();
      if (lim < kBN - 1 || lo > 0) {
#pragma unroll
        for (int i = 0; i < kBN; ++i) sv[i] = (i <= lim && i >= lo) ? sv[i] : -INFINITY;
      }
      float f[kPages], ev[kPages];
#pragma unroll
      for (int b = 0; b < kPages; b += 4) {
        const float4 x = *reinterpret_cast<const float4*>(&B->ks[jj % kScaleSlots][b]);
        const float4 y = *reinterpret_cast<const float4*>(&B->ev[jj % kScaleSlots][b]);
        f[b] = x.x * hs; f[b + 1] = x.y * hs; f[b + 2] = x.z * hs; f[b + 3] = x.w * hs;
        ev[b] = y.x; ev[b + 1] = y.y; ev[b + 2] = y.z; ev[b + 3] = y.w;
      }
      // the row's largest x + ev: each block's largest score, scaled
      float top = -INFINITY;
#pragma unroll
      for (int b = 0; b < kPages; b += 2) {
        float z2[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const float* s = sv + 16 * (b + u);
          const float a = fmax3(fmax3(s[0], s[1], s[2]), fmax3(s[3], s[4], s[5]), fmax3(s[6], s[7], s[8]));
          const float c = fmax3(fmax3(s[9], s[10], s[11]), fmax3(s[12], s[13], s[14]), s[15]);
          z2[u] = fmaf(fmaxf(a, c), f[b + u], ev[b + u]);
        }
        top = fmax3(top, z2[0], z2[1]);
      }
      top -= kTop;
      const bool resc = top - m_run > kLag;       // also on a row's first visible key
      const float alpha = resc ? ex2_approx(m_run - top) : 1.f;
      m_run = resc ? top : m_run;
      // a row with every key so far masked has m = -inf: subtract 0 instead,
      // so that its masked scores give 2^-inf = 0 rather than NaN
      const float m_sub = m_run == -INFINITY ? 0.f : m_run;
      const float e_max = fmax3(fmax3(ev[0], ev[1], ev[2]), fmax3(ev[3], ev[4], ev[5]), fmaxf(ev[6], ev[7]));
      const float e_min = -fmax3(fmax3(-ev[0], -ev[1], -ev[2]), fmax3(-ev[3], -ev[4], -ev[5]), fmaxf(-ev[6], -ev[7]));
      e_run = fmaxf(e_run, e_max);
      float lsum = 0.f;
      if constexpr (kF32) {
#pragma unroll
        for (int b = 0; b < kPages; ++b) {
          const float base = ev[b] - m_sub;
          float bs = 0.f;
          uint32_t hi[8], lw[8];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float p0 = ex2_approx(fmaf(sv[16 * b + i], f[b], base));
            const float p1 = ex2_approx(fmaf(sv[16 * b + i + 1], f[b], base));
            bs += p0 + p1;
            hi[i / 2] = halves(p0, p1);
            const float2 h = floats(hi[i / 2]);
            lw[i / 2] = halves(p0 - h.x, p1 - h.y);
          }
          lsum = fmaf(bs, q8::exp2i(-(int)ev[b]), lsum);
          // (kept in the scores' registers until all are read)
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            sv[16 * b + i] = __uint_as_float(hi[i]);
            sv[16 * b + 8 + i] = __uint_as_float(lw[i]);
          }
        }
#pragma unroll
        for (int b = 0; b < kPages; b += 2) {
          uint32_t pk[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = __float_as_uint(sv[16 * (b + (i >> 3)) + (i & 7)]);
          tc::tmem_st16(trow + colS + 8 * b, pk);
#pragma unroll
          for (int i = 0; i < 16; ++i) pk[i] = __float_as_uint(sv[16 * (b + (i >> 3)) + 8 + (i & 7)]);
          tc::tmem_st16(trow + colS + 64 + 8 * b, pk);
        }
      } else {
        const bool wide = e_run - e_min > kSpread;
        if (wide) {
          // float32 exponentials for the sum (see the header)
#pragma unroll
          for (int b = 0; b < kPages; ++b) {
            const float base = ev[b] - m_sub;
            float bs = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) bs += ex2_approx(fmaf(sv[16 * b + i], f[b], base));
            lsum = fmaf(bs, q8::exp2i(-(int)ev[b]), lsum);
          }
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int b = 2 * h + u;
            const float base = ev[b] - m_sub;
            const float2 f2 = make_float2(f[b], f[b]), b2 = make_float2(base, base);
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float2 z = __ffma2_rn(make_float2(sv[16 * b + i], sv[16 * b + i + 1]), f2, b2);
              pk[8 * u + i / 2] = ex2_f16x2(halves(z.x, z.y));
            }
            if (!wide) {
              // the block's sum in halves (16 weights of at most 2^8)
              const uint32_t* q = pk + 8 * u;
              const uint32_t s4 = add_f16x2(add_f16x2(add_f16x2(q[0], q[1]), add_f16x2(q[2], q[3])),
                                            add_f16x2(add_f16x2(q[4], q[5]), add_f16x2(q[6], q[7])));
              const float2 s2 = floats(s4);
              lsum = fmaf(s2.x + s2.y, q8::exp2i(-(int)ev[b]), lsum);
            }
          }
          tc::tmem_st16(trow + colS + 16 * h, pk);
        }
      }
      l_run = fmaf(l_run, alpha, lsum);
      // S_t(j) ready implies P_t.V(j-1) completed (same issuing thread, in
      // order), so O_t is stable here and may be rescaled.
      if (jj >= 1 && __any_sync(0xffffffffu, resc)) {
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc::tmem_ld32_sync(trow + colO + 32 * c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= alpha;
          tc::tmem_st32(trow + colO + 32 * c, o);
        }
      }
      tc::tmem_wait_st();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->p_full[t]);
    }
    // epilogue: O_t / l -> rows
    if (ok) {
      const bool w = __all_sync(0xffffffffu, mbar_wait(&B->o_done[t], 0, p.wait_ns));
      if (!w) abort_cta(B, p.error_word);
      if (w) {
        tc::fence_after_sync();
        const float inv = 1.f / l_run;
        T* dst = static_cast<T*>(p.out) + ((int64_t)(q0 + tok) * p.num_q_heads + head) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc::tmem_ld32_sync(trow + colO + 32 * c, o);
          if (valid) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              o[e] *= inv;
              const int a = B->nan_first[32 * c + e], b = B->nan_last[32 * c + e];
              if ((a <= pos && a >= key_row) || (b >= 0 && b <= pos && b >= key_row)) o[e] = __int_as_float(0x7fffffff);
            }
            constexpr int N = rope::Vec<T>::kN;
#pragma unroll
            for (int e = 0; e < 32; e += N)
              reinterpret_cast<uint4*>(dst)[(32 * c + e) / N] = rope::Vec<T>::store(o + e);
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
  order_after_previous_grid();
}

namespace {

template <typename T, int D>
cb_status launch_kernel(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                        int64_t scale_stride, uint32_t* error_word, cudaStream_t stream,
                        bool overlap_previous) {
  auto kern = prefill_kernel<T, D>;
  static std::atomic<uint8_t> attr_set[kMaxDevices];
  cb_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), Smem<D>::total, attr_set);
  if (st != CB_OK) return st;
  const int64_t n = ctas(a);
  if (n <= 0) return CB_OK;
  if (n >= ((int64_t)1 << 31)) return CB_ERR_UNSUPPORTED;
  Params p{};
  p.k_cache = static_cast<const uint8_t*>(a.k_cache);
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.scale_stride = scale_stride;
  p.q = a.q;
  p.out = a.out;
  p.cu_seqlens_q = a.cu_seqlens_q;
  p.seq_lens = a.seq_lens;
  p.block_tables = a.block_tables;
  p.row_begin = a.num_decodes;
  p.num_rows = a.num_reqs - a.num_decodes;
  p.num_tokens = a.num_tokens;
  p.num_blocks = a.num_blocks;
  p.max_blocks_per_seq = a.max_blocks_per_seq;
  p.num_q_heads = a.num_q_heads;
  p.num_kv_heads = a.num_kv_heads;
  p.group = a.num_q_heads / a.num_kv_heads;
  p.scale_log2 = a.scale * 1.4426950408889634f;
  p.window = a.sliding_window;
  p.error_word = error_word;
  p.wait_ns = wait_limit_ns();
  p.withhold_tile = withheld_prefill_tile();
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)n, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = Smem<D>::total;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = overlap_previous ? 1 : 0;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "prefill kernel launch: %s", cudaGetErrorString(e));
  return CB_OK;
}

}  // namespace

int64_t ctas(const cb_attention_args& a) {
  const int G = a.num_q_heads / a.num_kv_heads;
  if (G <= 0 || G > kBM || a.num_reqs <= a.num_decodes) return 0;
  const int tpp = (a.dtype == CB_DTYPE_F32 ? 1 : 2) * (kBM / G);
  // every row's pairs: tokens / tpp rounded up per row (decode rows may be
  // padding without tokens, so all tokens may be prefill tokens)
  const int64_t pairs = ((int64_t)a.num_tokens + tpp - 1) / tpp + (a.num_reqs - a.num_decodes);
  return pairs * a.num_kv_heads;
}

cb_status launch(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                 int64_t scale_stride, uint32_t* error_word, cudaStream_t stream,
                 bool overlap_previous) {
  if (a.num_q_heads / a.num_kv_heads > kBM) return CB_ERR_UNSUPPORTED;
#define CB_PRE(T, DD) \
  return launch_kernel<T, DD>(a, k_scales, v_scales, scale_stride, error_word, stream, overlap_previous)
  if (a.dtype == CB_DTYPE_F32) {
    if (a.head_dim == 64) CB_PRE(float, 64);
    CB_PRE(float, 128);
  }
  if (a.head_dim == 64) CB_PRE(__nv_bfloat16, 64);
  CB_PRE(__nv_bfloat16, 128);
#undef CB_PRE
}

}  // namespace prefill_q8
}  // namespace cb
