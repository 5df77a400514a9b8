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
//   * Two producer warps gather the pages' codes through the block table (one
//     TMA box of 16 rows per page) into one raw tile each for K and V.  Four
//     converter warps take a raw tile into registers, which frees it for the
//     next tile's copies at once, expand it to halves (every e4m3 number is
//     one exactly: one conversion for two codes) and store those in the
//     swizzled layout that the matrix instructions read.  (Reading the codes
//     from global memory into the converters' registers instead was 2.3 times
//     slower: with 227 KB of shared memory in use the L1 holds too few
//     outstanding loads.)
//   * Both products are kind::f16 with half operands: Q rows are scaled by a
//     power of two to the halves' range (so bfloat16 queries are halves
//     exactly; elements under 2^-29 of the row's largest lose bits).
//   * The scales stay out of the operands.  A score's factor is its block's
//     2^ek times the row's; a weight is 2^(x + ev - m) with x the score in
//     powers of two, so that weight times code is the value's part, and the
//     running reference m is over x + ev.  The sum of weights adds each
//     block's sum times 2^-ev, in float32 and from the unrounded weights, so
//     that a block of small values counts in it in full; the weights
//     themselves are rounded to halves (2^7 at the reference, 2^15 at most;
//     below 2^-25 they are zero, 2^-32 of the largest).  Exponentials are
//     float32: the unit takes 4 cycles a warp for them and 8 for a pair of
//     halves or bfloat16s, so the packed forms only lose bits.
//   * float32 queries: Q and the weights are split into two halves each (22
//     bits; a weight also to 2^-24, the least half), one query tile per CTA (the second tile's place holds the low
//     halves).  Score exponents are rounded once: scale * log2(e) is a pair
//     of floats, the reference a whole number near the largest exponent.  The
//     tensor core drops bits wherever it adds to a large accumulator, so each
//     tile's P.V starts from zero and the softmax warps add it to the output
//     (largest error at 1000 keys 0.6 to 1.1e-6; 0.9 to 1.7e-6 with one
//     accumulator, 0.4 to 0.9e-6 for a plain float32 form).
//   * A value code that is NaN must not reach rows that do not see its key
//     (weight 0 times NaN is NaN): in tiles that some row of the CTA sees only
//     in part, converters store such codes as 0 and note the first and last
//     key for each dim; the epilogue writes NaN where a row sees one.  Between
//     those two (with a window a row may see neither) it looks at the codes
//     again, which only calls with several such codes in one dim pay for.
//
//   * Few rows with many keys would leave most SMs idle: when the CTAs, counted
//     by their bound (one pair more for each row than its tokens fill: the host
//     does not know the rows), fill less than half of them, each one's KV tiles
//     are split over SMs / bound CTAs (at least four tiles each), which leave
//     float32 parts that a second kernel joins.  One row of 16 tokens counts
//     two pairs where one works, so its splits fill 72 of 152 SMs (64 tokens of
//     64 heads behind 16k: 63 us, 265 without; 16 tokens of 32 heads behind
//     100k: 170 and 1344; 64 of 32 behind 2k: 26 and 44; 64 behind 900, under
//     eight tiles: not split).
//
// What bounds it: the chain of a KV tile, 2.0 us for 128 keys and both query
// tiles.  Its products are 1.4 us at the measured matrix rate, its 32k exponentials
// 0.55 us of the four exponential units each, and shared memory moves codes,
// halves and operands for 1.3 us; the rest is the turns that the two query
// tiles' softmax take with them.  512 tokens of 64 heads behind 16k (128
// CTAs of 152 SMs): 279 us, 1.0 PFLOP/s, 54% of the measured bfloat16 rate
// (with the 16-bit cache, which is read and not expanded, the 16-bit kernel
// takes 237 us where this one takes 273); a CTA costs 7 us beside its tiles.
//
// Tensor memory: S0 | S1 | O0 | O1 at columns 0, 128, 256, 384; P_t is
// written over S_t as half pairs and read from there as the A operand.
//
// Warp roles (512 threads, registers redistributed):
//   0-3 / 4-7  softmax of query tile 0 / 1 (thread = row): 192 registers
//   8, 9       producers of raw K and V tiles: 48
//   10, 11     MMA issuers of the two tiles (10 owns TMEM): 48
//   12-15      converters: 80
// Per KV tile j an issuer queues P.V(j-1) and then Q.K(j).  Every wait is
// bounded (CB_DEVERR_TIMEOUT).
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cb_error.h"
#include "device_utils.cuh"
#include "launch_common.h"
#include "mma_utils.cuh"
#include "prefill_q8.h"
#include "q8.cuh"
#include "rope.cuh"
#include "row_checks.h"
#include "tcgen05.cuh"
#include "tensor_map.h"

namespace cb {
namespace prefill_q8 {

constexpr int kBM = 128;            // query rows per tile
constexpr int kBN = 128;            // keys per KV tile
constexpr int kPage = 16;
constexpr int kPages = kBN / kPage; // blocks of a KV tile
constexpr int kStages = 2;          // tiles of K, and of V, as halves
constexpr int kScaleSlots = 4;      // tiles whose scales are kept (see Bars)
constexpr int kMmaWarp = 10;
constexpr int kConvWarp = 12;
constexpr int kThreads = 512;
constexpr int kRegsSoftmax = 192, kRegsMma = 48, kRegsConv = 80;
static_assert(128 * (2 * kRegsSoftmax + kRegsMma + kRegsConv) <= 65536, "register split");
constexpr uint32_t kHalf = 128 * 128;  // 128 rows of 64 halves
// A CTA costs about 7 us beside its KV tiles, of 2 us each, so a split of the
// keys has at least four of them.
constexpr int kLeastTiles = 4;
constexpr int kMaxSplits = 16;
constexpr uint32_t kTmemCols = 512;
// weight exponent at the reference, which moves when passed by more than the
// lag (float32: exponents near 0 are the most exact)
template <typename T> constexpr float kTop = 7.f;
template <> constexpr float kTop<float> = 0.f;
template <typename T> constexpr float kLag = 8.f;
template <> constexpr float kLag<float> = 2.f;
__host__ __device__ constexpr uint32_t col_s(int t) { return t ? 128u : 0u; }
__host__ __device__ constexpr uint32_t col_o(int t) { return t ? 384u : 256u; }

struct Bars {
  uint64_t raw_full[2];        // the K, V codes of a tile landed
  uint64_t raw_empty[2];       // they are in the converters' registers
  uint64_t k_full[kStages];    // K tile expanded (one arrival per converter warp)
  uint64_t v_full[kStages];
  uint64_t k_empty[kStages];  // last Q.K of the stage done
  uint64_t v_empty[kStages];  // last P.V of the stage done
  uint64_t s_full[2], p_full[2], o_done[2], drain[2];
  uint64_t turn[2][4];         // warp w of softmax t has made its weights of a tile
  uint32_t tmem_base, abort;
  int32_t row, pair;
  // what the CTA works on; the roles read it where they need it (kept in
  // registers from the prologue on, it would spill)
  int32_t seq_len, n_tiles, npages, lo_pg, first_pos, last_pos, table_row, split;
  // Of each block of recent KV tiles: 2^ek, ev, 2^-ev.  The slot of tile j is rewritten for tile j +
  // 4, which is expanded only after Q.K(j + 2) of both query tiles, and that
  // is queued only after their softmax of tile j + 1.
  alignas(16) float scales[kScaleSlots][kPages][4];
  int32_t nan_first[128], nan_last[128];  // by dim: keys whose value is NaN
  int32_t nan_any;
};

template <int D>
struct Smem {
  static constexpr uint32_t kTile = kBM * D * 2;  // Q, K or V tile of halves
  static constexpr uint32_t q = 0;                // Q0 | Q1 (float32: high | low)
  static constexpr uint32_t k = q + 2 * kTile;
  static constexpr uint32_t v = k + kStages * kTile;
  static constexpr uint32_t raw = v + kStages * kTile;    // K codes | V codes
  static constexpr uint32_t kRaw = kBN * D;
  static constexpr uint32_t bars = raw + 2 * kRaw;
  static constexpr uint32_t total = bars + sizeof(Bars) + 1024;  // + alignment of the base
};
static_assert(kScaleSlots > kStages + 1, "a slot outlives its softmax");
static_assert(Smem<128>::total <= 227 * 1024, "shared memory");

struct Params {
  CUtensorMap tmap_k;  // [num_blocks * Hkv * 16 rows][D] bytes, box 16 rows x D
  CUtensorMap tmap_v;
  const uint8_t* v_cache;     // (the epilogue's second look at NaN codes)
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
  float scale_log2_low;       // what float32 leaves of it, as a share of it
  int32_t window;
  uint32_t* error_word;
  // splits of the keys of a (row, pair of query tiles); with more than one,
  // token i of the prefill rows leaves split s's part at slot i * splits + s
  int32_t splits;
  float* part_ml;             // [slots][Hq][2]: reference and sum of weights
  float* part_acc;            // [slots][Hq][D]
  uint64_t wait_ns;
  int32_t withhold_tile;      // test hook: CTA 0 never copies this raw K tile (-1: none)
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
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}
__device__ __forceinline__ float4 lds_float4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}
// s (f + fl) + base, rounded at the size of the result and not of s f; -inf
// stays -inf (whatever the sign of fl)
__device__ __forceinline__ float exponent(float s, float f, float fl, float base) {
  return fmaf(fmaxf(s, -4294967296.f), fl, fmaf(s, f, base));
}
// Any e4m3 NaN (0x7f or 0xff) among four codes.
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}

// A row's tokens and length lie within the call's (and its parts' places).
__device__ __forceinline__ bool row_fits(const Params& p, int q0, int q_len, int L) {
  const int first = p.splits > 1 ? p.cu_seqlens_q[p.row_begin] : 0;
  return first >= 0 && q0 >= first && row_tokens_fit(q0, q_len, p.num_tokens) && L >= q_len &&
         row_length_fits(L, kPage, p.max_blocks_per_seq);
}

// The KV tiles of a (row, pair of query tiles) and of each of its splits.
struct Tiles {
  int key_lo;         // with a window, the first key that the first query sees
  int first, last;    // tiles [first, last)
  int of_split;       // tiles of a split; the last one may have fewer
  int splits;         // that have any
};
// start: cached tokens of the row; [tok0, tok0 + tpp) the pair's tokens
__device__ __forceinline__ Tiles tiles_of(const Params& p, int start, int q_len, int tok0, int tpp) {
  Tiles t;
  t.key_lo = p.window > 0 ? max(0, start + tok0 - p.window + 1) : 0;
  t.first = t.key_lo / kBN;
  t.last = (start + min(tok0 + tpp - 1, q_len - 1)) / kBN + 1;
  const int n = t.last - t.first;
  t.of_split = p.splits > 1 ? max((n + p.splits - 1) / p.splits, kLeastTiles) : n;
  t.splits = p.splits > 1 ? (n + t.of_split - 1) / t.of_split : 1;
  return t;
}

// Some row of the CTA does not see all keys of the tile that starts at kbase.
__device__ __forceinline__ bool seen_in_part(const Params& p, const volatile Bars* B, int kbase) {
  return kbase + kBN - 1 > B->first_pos || (p.window > 0 && kbase < B->last_pos - p.window + 1);
}

// Bit e: a value of dim d0 + e that the row at position pos sees in a tile
// that is seen in part is NaN.  key_row: the first key of the row's window.
template <int D>
__device__ __forceinline__ uint32_t nan_dims(const Params& p, const volatile Bars* B, int g, int d0, int pos,
                                             int key_row) {
  uint32_t mask = 0;
#pragma unroll 1
  for (int e = 0; e < 32; ++e) {
    const int first = B->nan_first[d0 + e], last = B->nan_last[d0 + e];
    bool sees = (first <= pos && first >= key_row) || (last <= pos && last >= key_row && last >= 0);
    if (!sees && first < key_row && last > pos) {
      // neither end of the NaN keys is seen: one between them may be
#pragma unroll 1
      for (int key = key_row; key <= pos && !sees; ++key) {
        if (!seen_in_part(p, B, key / kBN * kBN)) {
          key |= kBN - 1;                         // such a tile's NaN codes were multiplied
          continue;
        }
        const int b = p.block_tables[(int64_t)B->table_row * p.max_blocks_per_seq + key / kPage];
        if (b >= 0 && b < p.num_blocks)
          sees = (p.v_cache[(((int64_t)b * p.num_kv_heads + g) * kPage + key % kPage) * D + d0 + e] & 0x7f) == 0x7f;
      }
    }
    mask |= (uint32_t)sees << e;
  }
  return mask;
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
  // the decode rows of the same call, launched after this grid with
  // programmatic serialization, may start on the SMs that it leaves
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  const int G = p.group;
  const int tpt = kBM / G;                        // tokens per query tile
  const int tpp = kTiles * tpt;                   // of a CTA
  const int Hkv = p.num_kv_heads;
  const unsigned units = gridDim.x / (unsigned)p.splits;     // (row, pair, KV head)s
  const int split = (int)(blockIdx.x / units);
  const unsigned unit = blockIdx.x - split * units;
  const int g = (int)(unit % (unsigned)Hkv);
  // ---- which (row, pair) this CTA serves: warp 0 scans the rows' pair
  // counts; every row's latest (heaviest) pair comes first
  if (warp == 0) {
    const int x = (int)(unit / (unsigned)Hkv);
    const int num_pairs = (int)(units / (unsigned)Hkv);
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
  if (B->row < 0) return;                         // past the last pair
  const int r = p.row_begin + B->row;
  const int mp = B->pair;
  const int q0 = p.cu_seqlens_q[r];
  const int q_len = p.cu_seqlens_q[r + 1] - q0;
  const int L = p.seq_lens[r];
  if (!row_fits(p, q0, q_len, L)) {
    if (threadIdx.x == 0 && mp == 0 && g == 0 && split == 0) set_error(p.error_word, CB_DEVERR_SEQ_RANGE);
    return;
  }
  const int tok0 = mp * tpp;                      // first token of the CTA
  const bool has_t1 = kTiles == 2 && tok0 + tpt < q_len;
  const int start = L - q_len;
  const int last_tok = min(tok0 + tpp - 1, q_len - 1);
  const int npages = blocks_of(L, kPage);
  const Tiles tiles = tiles_of(p, start, q_len, tok0, tpp);
  if (split >= tiles.splits) return;
  const int lo_pg = tiles.key_lo / kPage;
  const int j_lo = tiles.first + split * tiles.of_split;
  const int n_tiles = min(tiles.last, j_lo + tiles.of_split);
  const int nt = n_tiles - j_lo;

  if ((warp == 8 || warp == 9) && lane == 0) tc::prefetch_tensormap(warp == 8 ? &p.tmap_k : &p.tmap_v);
  if (threadIdx.x == 0) {
    const uint32_t issuers = has_t1 ? 2u : 1u;
    for (int h = 0; h < 2; ++h) {
      mbar_init(&B->raw_full[h], 1);
      mbar_init(&B->raw_empty[h], 4);
    }
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&B->k_full[s], 4);
      mbar_init(&B->k_empty[s], issuers);
      mbar_init(&B->v_full[s], 4);
      mbar_init(&B->v_empty[s], issuers);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&B->s_full[t], 1);
      mbar_init(&B->p_full[t], 4);
      mbar_init(&B->o_done[t], 1);
      mbar_init(&B->drain[t], 1);
      for (int w = 0; w < 4; ++w) mbar_init(&B->turn[t][w], 1);
    }
    B->abort = 0;
    B->nan_any = 0;
    B->seq_len = L;
    B->n_tiles = n_tiles;
    B->npages = npages;
    B->lo_pg = lo_pg;
    B->first_pos = start + tok0;
    B->last_pos = start + last_tok;
    B->table_row = r;
    B->split = tiles.splits > 1 ? split : -1;
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
  // Lane i < 8: block of page i of tile j as the table has it, or -1 where the
  // page is not read.
  const volatile Bars* VB = B;
  auto reads_page = [&](int j) {
    const int pg = j * kPages + lane;
    return lane < kPages && j < VB->n_tiles && pg < VB->npages && pg >= VB->lo_pg;
  };
  auto table_ids = [&](int j) {
    return reads_page(j) ? p.block_tables[(int64_t)VB->table_row * p.max_blocks_per_seq + j * kPages + lane] : -1;
  };

  if (warp >= kConvWarp) {
    // ------------------------------------------------------------ converters
    tc::regs_dec<kRegsConv>();
    // Thread ct of 128 owns a 16-byte chunk of a page row: D = 128, one page
    // a round; D = 64, two.  Of every 8 neighbouring lanes 4 have the chunks of
    // one half of a row and 4 the same of another row (D = 128: the row XOR
    // 5), so that they never meet in a bank: neither where they read the
    // codes nor where they write the halves.
    constexpr int kChunks = D / 16;                // chunks of a row
    constexpr int kPerRound = 128 / (kPage * kChunks);  // pages of a round
    constexpr int kRounds = kPages / kPerRound;
    const int ct = threadIdx.x - kConvWarp * 32;
    const int even = ((ct >> 2) & 6) | ((ct >> 2) & 8);
    const int prow = D == 128 ? ((ct & 4) ? even ^ 5 : even) : (ct >> 2) & 15;
    const int c = D == 128 ? ((ct >> 6) << 2) | (ct & 3) : ct & 3;
    const int psub = D == 128 ? 0 : ct >> 6;
    // where the TMA swizzle put the chunk, and where its halves go: dims 16 c
    // .. 16 c + 7 and the next 8 of the row (rows of a round lie 16 rows or 32
    // after those of the last, so the swizzle is the same)
    const uint32_t raw_at = smem_addr(smem + Smem<D>::raw) + (uint32_t)psub * (kPage * D) +
                            (D == 128 ? prow * 128 + ((c ^ (prow & 7)) << 4) : prow * 64 + ((c ^ ((prow >> 1) & 3)) << 4));
    const uint32_t out_at = smem_addr(smem) + (uint32_t)(c / 4) * kHalf + (uint32_t)psub * (kPage * 128);
    const uint32_t out_a = out_at + swz(prow, (2 * c) & 7), out_b = out_at + swz(prow, (2 * c + 1) & 7);
    auto store = [&](uint32_t tile, int i, const uint32_t (&w)[4]) {
      uint32_t a[4], b[4];
      q8::halves4(w[0], a[0], a[1]);
      q8::halves4(w[1], a[2], a[3]);
      q8::halves4(w[2], b[0], b[1]);
      q8::halves4(w[3], b[2], b[3]);
      const uint32_t at = tile + i * (kPerRound * kPage * 128);
      sts128(out_a + at, a);
      sts128(out_b + at, b);
    };
    // raw tile h (0: K, 1: V) of ring turn jj into registers
    auto take = [&](int h, int jj, uint32_t (&w)[kRounds][4]) {
      if (!__all_sync(0xffffffffu, mbar_wait(&B->raw_full[h], jj & 1, p.wait_ns))) return false;
#pragma unroll
      for (int i = 0; i < kRounds; ++i) decode::lds128(raw_at + h * Smem<D>::kRaw + i * (kPerRound * kPage * D), w[i]);
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->raw_empty[h]);
      return true;
    };
    // Scale bytes of a tile (requested one tile ahead): lane i < 8 page i's K,
    // lane 8 + i its V; 1 for a page that is not read.
    auto scale_bytes = [&](int ids) {
      const int b = __shfl_sync(0xffffffffu, ids, lane & 7);
      uint32_t v = 127;
      if (lane < 2 * kPages && b >= 0 && b < p.num_blocks)
        v = (lane < kPages ? p.k_scales : p.v_scales)[(int64_t)b * p.scale_stride + g];
      return v;
    };
    uint32_t bytes = 127;
    int ids_next = -1;
    if (warp == kConvWarp) {
      bytes = scale_bytes(table_ids(j_lo));
      ids_next = table_ids(j_lo + 1);
    }
    bool ok = true;
    uint32_t w[kRounds][4];
    for (int jj = 0; jj < nt && ok; ++jj) {
      const int j = j_lo + jj;
      // ---- K
      const int st = jj % kStages;
      ok = take(0, jj, w);
      if (ok && jj >= kStages)
        ok = __all_sync(0xffffffffu, mbar_wait(&B->k_empty[st], ((jj / kStages) - 1) & 1, p.wait_ns));
      if (!ok) { abort_cta(B, p.error_word); break; }
      if (*reinterpret_cast<volatile uint32_t*>(&B->abort)) break;
      const uint32_t kt = Smem<D>::k + st * kTile;
#pragma unroll
      for (int i = 0; i < kRounds; ++i) store(kt, i, w[i]);
      if (warp == kConvWarp) {
        const int e = q8::exp_of(bytes);
        const int ev = __shfl_sync(0xffffffffu, e, kPages + (lane & 7));
        if (lane < kPages)
          *reinterpret_cast<float4*>(B->scales[jj % kScaleSlots][lane]) =
              make_float4(q8::exp2i(e), (float)ev, q8::exp2i(-ev), 0.f);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->k_full[st]);
      if (warp == kConvWarp) {
        bytes = scale_bytes(ids_next);
        ids_next = table_ids(j + 2);
      }
      // ---- V
      ok = take(1, jj, w);
      if (ok && jj >= kStages)
        ok = __all_sync(0xffffffffu, mbar_wait(&B->v_empty[st], ((jj / kStages) - 1) & 1, p.wait_ns));
      if (!ok) { abort_cta(B, p.error_word); break; }
      const uint32_t vt = Smem<D>::v + st * kTile;
      const int kbase = j * kBN;
      const int end = VB->seq_len - kbase;         // rows past the sequence become zeros
      const bool part = seen_in_part(p, VB, kbase);
      if (!part) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) store(vt, i, w[i]);
      } else {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
          const int row = (i * kPerRound + psub) * kPage + prow;
          uint32_t x[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) x[b] = row < end ? w[i][b] : 0u;
          if (nan_codes(x[0]) | nan_codes(x[1]) | nan_codes(x[2]) | nan_codes(x[3])) {
            *reinterpret_cast<volatile int32_t*>(&B->nan_any) = 1;
#pragma unroll
            for (int b = 0; b < 16; ++b)
              if (((x[b >> 2] >> (8 * (b & 3))) & 0x7fu) == 0x7fu) {
                x[b >> 2] &= ~(0xffu << (8 * (b & 3)));
                atomicMin(&B->nan_first[16 * c + b], kbase + row);
                atomicMax(&B->nan_last[16 * c + b], kbase + row);
              }
          }
          store(vt, i, x);
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&B->v_full[st]);
    }
  } else if (warp >= 8) {
    tc::regs_dec<kRegsMma>();
    if (warp < kMmaWarp) {
      // ---------------------------------------------------------- producers
      // Lane i (0..7) looks up page i of a tile (the next tile's ids are
      // requested before the current tile's copies are issued); lane 0 issues
      // the boxes.  A page that is not read uses a row past the end of the
      // tensor map, which the TMA engine reads as zeros.
      const int h = warp - 8;
      const CUtensorMap* tmap = h ? &p.tmap_v : &p.tmap_k;
      const int oob_row = p.num_blocks * Hkv * kPage;
      uint8_t* raw = smem + Smem<D>::raw + h * Smem<D>::kRaw;
      int next = table_ids(j_lo);
      int issued = 0;
      for (int jj = 0; jj < nt; ++jj) {
        int row = oob_row;
        if (reads_page(j_lo + jj)) {
          if (next >= 0 && next < p.num_blocks)
            row = (next * Hkv + g) * kPage;
          else if (h == 0)
            set_error(p.error_word, CB_DEVERR_BLOCK_RANGE);
        }
        next = table_ids(j_lo + jj + 1);
        if (jj >= 1) {
          const bool ok = __all_sync(0xffffffffu, mbar_wait(&B->raw_empty[h], (jj - 1) & 1, p.wait_ns));
          if (!ok) { abort_cta(B, p.error_word); break; }
        }
        if (*reinterpret_cast<volatile uint32_t*>(&B->abort)) break;
        if (lane == 0) mbar_arrive_expect_tx(&B->raw_full[h], Smem<D>::kRaw);
        // test hook: the withheld tile is announced but never copied, so the
        // bounded waits on it run out
        const bool withhold = h == 0 && blockIdx.x == 0 && jj == p.withhold_tile;
#pragma unroll
        for (int i = 0; i < kPages; ++i) {
          const int rr = __shfl_sync(0xffffffffu, row, i);
          if (lane == 0 && !withhold) tc::tma_load_2d(raw + i * (kPage * D), tmap, 0, rr, &B->raw_full[h]);
        }
        __syncwarp();
        issued = jj + 1;
      }
      // drain: every issued copy lands before the CTA may exit
      if (issued > 0) mbar_wait(&B->raw_full[h], (issued - 1) & 1, p.wait_ns);
    } else {
      // -------------------------------------------------------------- MMA
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
            const int jr = jj - 1, sp = jr % kStages;
            ok = wait_or_abort(&B->p_full[t], jr & 1, B, p.error_word, p.wait_ns) &&
                 wait_or_abort(&B->v_full[sp], (jr / kStages) & 1, B, p.error_word, p.wait_ns);
            if (!ok) break;
            tc::fence_after_sync();
            const uint64_t bv = dv0 + sp * kTileDesc;
#pragma unroll
            for (int piece = 0; piece < (kF32 ? 2 : 1); ++piece)
#pragma unroll
              for (int kk = 0; kk < kBN / 16; ++kk)
                tc::mma_f16_ts(tmem + col_o(t), tmem + col_s(t) + piece * 64 + kk * 8, bv + (kk * 2048 >> 4),
                               idesc_pv, ((!kF32 && jr > 0) || kk > 0 || piece > 0) ? 1u : 0u);
            tc::mma_commit(&B->v_empty[sp]);
            if (jj == nt) tc::mma_commit(&B->o_done[t]);
          }
          if (jj < nt) {
            const int s = jj % kStages;
            ok = wait_or_abort(&B->k_full[s], (jj / kStages) & 1, B, p.error_word, p.wait_ns);
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
    const bool valid = t < kTiles && tl < tpt && tok < q_len;
    const int pos = start + (valid ? tok : q_len - 1);
    // A warp copies its 32 rows of q and out kRowsAtOnce at a time, a row's
    // 16-byte chunks in neighbouring lanes, and turns them in shared memory: a
    // thread that reads or writes a row of its own touches a line for every
    // chunk (Q took 6 us of a CTA and O 8, now 3.5 and 3).
    constexpr int N = rope::Vec<T>::kN;
    constexpr int kChunks = D / N;
    constexpr int kRowsAtOnce = 32 / kChunks;
    const int chunk = lane % kChunks, sub = lane / kChunks;
    const uint32_t by_g = (65536u + G - 1) / G;   // x / G = x by_g / 2^16 for x < 128
    const int64_t first = ((int64_t)(q0 + tok0 + t * tpt) * p.num_q_heads + g * G) * D + chunk * N;
    // elements of q (and out) before the lane's chunk of row rr of the tile, or -1
    auto row_at = [&](int rr) -> int64_t {
      const int rt = (int)((uint32_t)rr * by_g >> 16);
      if (rt >= tpt || tok0 + t * tpt + rt >= q_len) return -1;
      return first + (int64_t)(rt * p.num_q_heads + rr - rt * G) * D;
    };
    float hs = 1.f;                               // score factor of the row
    if (t < kTiles) {
      // Q rows -> halves in shared memory, the largest magnitude at [2^14,
      // 2^15); the scale's sign goes with Q, and a scale of 0 makes Q zero.
      // First as they are: chunk c of a row where its halves will be (float32:
      // chunks from 16 on in the place of the low halves).
      uint8_t* qs = smem + Smem<D>::q + t * kTile;
      auto raw_at = [&](int rr, int c) {
        constexpr int kPer = D / 8;
        return qs + (c >= kPer ? kTile : 0u) + ((c % kPer) >> 3) * kHalf + swz(rr, c & 7);
      };
#pragma unroll 4
      for (int i = 0; i < kChunks; ++i) {
        const int rr = (warp & 3) * 32 + i * kRowsAtOnce + sub;
        const int64_t at = row_at(rr);
        // (0 bytes: zeros)
        cp_async16(smem_addr(raw_at(rr, chunk)), static_cast<const T*>(p.q) + max(at, (int64_t)0), at >= 0 ? 16 : 0);
      }
      asm volatile("cp.async.wait_all;" ::: "memory");
      __syncwarp();
      uint4 raw[kChunks];
#pragma unroll
      for (int i = 0; i < kChunks; ++i) raw[i] = *reinterpret_cast<const uint4*>(raw_at(row, i));
      auto load8 = [&](int i, float* x) {
        rope::Vec<T>::load(raw[i * (8 / N)], x);
        if constexpr (N == 4) rope::Vec<T>::load(raw[2 * i + 1], x + 4);
      };
      float amax = 0.f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float x[8];
        load8(i, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fabsf(x[e]));
      }
      // zeros, or a row that is not finite (nor are its scores): factor 1
      const int k = amax > 0.f && amax <= 3.402823466e38f ? max((int)(__float_as_uint(amax) >> 23) - 127, -110) : 14;
      // The row's factor is never so small that times a block's scale it is 0
      // (a masked score is -inf): below 2^-80 it stays there and what is
      // missing goes into Q, whose halves then lose bits of scores that are
      // under 2^-9 at any scale of the blocks.
      const float mag = fabsf(p.scale_log2), factor = mag * q8::exp2i(k - 14);
      const bool tiny = factor < q8::exp2i(-80);
      hs = mag == 0.f ? 1.f : tiny ? q8::exp2i(-80) : factor;
      const float up = copysignf(mag == 0.f ? 0.f : tiny ? mag * q8::exp2i(80) : q8::exp2i(14 - k), p.scale_log2);
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        float x[8];
        load8(i, x);
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
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = active;
    // keys before key_row are outside this row's window
    const int key_row = p.window > 0 ? pos - p.window + 1 : -(1 << 30);
    for (int jj = 0; jj < nt && ok; ++jj) {
      // Warps w and 4 + w, which share a quarter of the SM, take turns on its
      // exponential and FMA units while the tensor core works for the other.
      if (has_t1 && (t == 1 || jj >= 1)) {
        const bool tw = __all_sync(0xffffffffu, mbar_wait(&B->turn[t ^ 1][warp & 3], (t == 0 ? jj - 1 : jj) & 1, p.wait_ns));
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
      // scales of block b of the tile (read where they are used: the scores
      // take most of the registers)
      const uint32_t sc = smem_addr(B->scales[jj % kScaleSlots]);
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
          const float4 k = lds_float4(sc + 16 * (b + u));
          z2[u] = fmaf(fmaxf(a, c), k.x * hs, k.y);
        }
        top = fmax3(top, z2[0], z2[1]);
      }
      top -= kTop<T>;
      if constexpr (kF32) top = rintf(top);
      const bool resc = top - m_run > kLag<T>;    // also on a row's first visible key
      const float alpha = resc ? ex2_approx(m_run - top) : 1.f;
      m_run = resc ? top : m_run;
      // a row with every key so far masked has m = -inf: subtract 0 instead,
      // so that its masked scores give 2^-inf = 0 rather than NaN
      const float m_sub = m_run == -INFINITY ? 0.f : m_run;
      float lsum = 0.f;
      if constexpr (kF32) {
#pragma unroll
        for (int b = 0; b < kPages; ++b) {
          const float4 k = lds_float4(sc + 16 * b);
          const float f = k.x * hs, fl = f * p.scale_log2_low, base = k.y - m_sub;
          float bs = 0.f;
          uint32_t hi[8], lw[8];
#pragma unroll
          for (int i = 0; i < 16; i += 2) {
            const float p0 = ex2_approx(exponent(sv[16 * b + i], f, fl, base));
            const float p1 = ex2_approx(exponent(sv[16 * b + i + 1], f, fl, base));
            bs += p0 + p1;
            hi[i / 2] = halves(p0, p1);
            const float2 h = floats(hi[i / 2]);
            lw[i / 2] = halves(p0 - h.x, p1 - h.y);
          }
          lsum = fmaf(bs, k.z, lsum);
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
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          uint32_t pk[16];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int b = 2 * h + u;
            const float4 k = lds_float4(sc + 16 * b);
            const float f = k.x * hs, base = k.y - m_sub;
            const float2 f2 = make_float2(f, f), b2 = make_float2(base, base);
            float2 sum[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              float2 z = __ffma2_rn(make_float2(sv[16 * b + i], sv[16 * b + i + 1]), f2, b2);
              z.x = ex2_approx(z.x);
              z.y = ex2_approx(z.y);
              sum[i / 2 & 1] = __fadd2_rn(sum[i / 2 & 1], z);
              pk[8 * u + i / 2] = halves(z.x, z.y);
            }
            lsum = fmaf((sum[0].x + sum[1].x) + (sum[0].y + sum[1].y), k.z, lsum);
          }
          tc::tmem_st16(trow + colS + 16 * h, pk);
          if (h == 3 && lane == 0) mbar_arrive(&B->turn[t][warp & 3]);
        }
      }
      l_run = fmaf(l_run, alpha, lsum);
      // S_t(j) ready implies P_t.V(j-1) completed (same issuing thread, in
      // order), so O_t is stable here and may be rescaled.
      if (kF32 && jj >= 1) {
        // the sum of the tiles before, in the place of the second tile's O
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          float o[16], a[16];
          tc::tmem_ld16(trow + colO + 16 * c, o);
          if (jj > 1) tc::tmem_ld16(trow + col_o(1) + 16 * c, a);
          tc::tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; ++e) o[e] = (jj > 1 ? a[e] + o[e] : o[e]) * alpha;
          tc::tmem_st16(trow + col_o(1) + 16 * c, reinterpret_cast<const uint32_t*>(o));
        }
      } else if (jj >= 1 && __any_sync(0xffffffffu, resc)) {
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
        const int part = VB->split;                 // -1: the row's only one
        const bool parted = part >= 0;
        const float inv = parted ? 1.f : 1.f / l_run;
        // The rows are turned in shared memory, so that a warp stores whole
        // ones: Q's place is free (its last product preceded O's).
        uint8_t* turn = smem + Smem<D>::q + t * kTile + (warp & 3) * (32 * kChunks * 16);
        auto slot_of = [&](int rr) -> int64_t {
          const int rt = (int)((uint32_t)rr * by_g >> 16);
          if (rt >= tpt || tok0 + t * tpt + rt >= q_len) return -1;
          return (int64_t)(q0 - p.cu_seqlens_q[p.row_begin] + tok0 + t * tpt + rt) * p.splits + part;
        };
        auto head_of = [&](int rr) { return g * G + rr - (int)((uint32_t)rr * by_g >> 16) * G; };
        auto store_part = [&](uint8_t* turn, int c, const float* o) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<float4*>(turn + (lane * 8 + (e ^ (lane & 7))) * 16) =
                make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          __syncwarp();
#pragma unroll 2
          for (int i = 0; i < 8; ++i) {
            const int rr = i * 4 + lane / 8;          // of the warp's rows
            const float4 v = *reinterpret_cast<const float4*>(turn + (rr * 8 + (lane % 8 ^ (rr & 7))) * 16);
            const int64_t slot = slot_of((warp & 3) * 32 + rr);
            if (slot >= 0)
              reinterpret_cast<float4*>(p.part_acc + (slot * p.num_q_heads + head_of((warp & 3) * 32 + rr)) * D + 32 * c)[lane % 8] = v;
          }
          __syncwarp();  // before the next dims take its place
        };
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tc::tmem_ld32_sync(trow + colO + 32 * c, o);
          if (kF32 && nt > 1) {
            float a[32];
            tc::tmem_ld32_sync(trow + col_o(1) + 32 * c, a);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] += a[e];
          }
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= inv;
          if (parted) {
            // 32 dims of this split's part, in float32, row by row
            store_part(turn, c, o);
            continue;
          }
#pragma unroll
          for (int e = 0; e < 32; e += N) {
            const int at = (32 * c + e) / N;
            *reinterpret_cast<uint4*>(turn + (lane * kChunks + (at ^ (lane & 7))) * 16) = rope::Vec<T>::store(o + e);
          }
        }
        __syncwarp();
        if (parted) {
          const int64_t slot = slot_of(row);
          if (slot >= 0) *reinterpret_cast<float2*>(p.part_ml + (slot * p.num_q_heads + head_of(row)) * 2) = make_float2(m_run, l_run);
        }
#pragma unroll 4
        for (int i = 0; i < kChunks && !parted; ++i) {
          const int rr = i * kRowsAtOnce + sub;       // of the warp's rows
          const uint4 v = *reinterpret_cast<const uint4*>(turn + (rr * kChunks + (chunk ^ (rr & 7))) * 16);
          const int64_t at = row_at((warp & 3) * 32 + rr);
          if (at >= 0) *reinterpret_cast<uint4*>(static_cast<T*>(p.out) + at) = v;
        }
        // NaN over the rows' outputs where it belongs (apart from the rest, which
        // every call runs)
        if (*reinterpret_cast<volatile int32_t*>(&B->nan_any) != 0) {
          __syncwarp();                             // the rows are written
          const int64_t at = valid ? (parted ? slot_of(row) : (int64_t)(q0 + tok)) * p.num_q_heads + head_of(row) : -1;
#pragma unroll 1
          for (int c = 0; c < D / 32 && valid; ++c) {
            uint32_t nan = nan_dims<D>(p, VB, g, 32 * c, pos, key_row);
            for (; nan != 0; nan &= nan - 1) {
              const int64_t d = at * D + 32 * c + __ffs(nan) - 1;
              if (parted) p.part_acc[d] = __int_as_float(0x7fffffff);
              else rope::from_float(static_cast<T*>(p.out) + d, __int_as_float(0x7fffffff));
            }
          }
        }
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == kMmaWarp) tc::tmem_dealloc(tmem, kTmemCols);
}

// Joins the splits' parts of the prefill rows' outputs: one warp for each
// (token, head); sum_s 2^(m_s - M) acc_s / sum_s 2^(m_s - M) l_s, in the
// splits' order.  Bound by its latency (a search for the token's row, then
// all parts at once).
template <typename T, int D>
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ Params p) {
  constexpr bool kF32 = std::is_same<T, float>::value;
  constexpr int kE = D / 32;                      // elements of a lane
  const int lane = threadIdx.x & 31;
  const int64_t w = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  const int i = (int)(w / p.num_q_heads), head = (int)(w - (int64_t)i * p.num_q_heads);
  const int32_t* cu = p.cu_seqlens_q + p.row_begin;
  const int token = cu[0] + i;
  if (cu[0] < 0 || token >= cu[p.num_rows] || token >= p.num_tokens) return;
  int lo = 0, hi = p.num_rows - 1;                // the row with cu[row] <= token < cu[row + 1]
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= token) lo = mid; else hi = mid - 1;
  }
  const int q_len = cu[lo + 1] - cu[lo], L = p.seq_lens[p.row_begin + lo];
  if (token < cu[lo] || token >= cu[lo + 1] || !row_fits(p, cu[lo], q_len, L)) return;
  const int tpp = (kF32 ? 1 : 2) * (kBM / p.group);
  const int tok0 = (token - cu[lo]) / tpp * tpp;
  const Tiles t = tiles_of(p, L - q_len, q_len, tok0, tpp);
  if (t.splits <= 1) return;                      // the CTA has written its rows
  const int64_t first = (int64_t)i * p.splits;
  float2 ml = make_float2(-INFINITY, 0.f);
  if (lane < t.splits) ml = reinterpret_cast<const float2*>(p.part_ml)[(first + lane) * p.num_q_heads + head];
  float acc[kMaxSplits][kE];
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) {
    const float* part = p.part_acc + ((first + s) * p.num_q_heads + head) * D + kE * lane;
#pragma unroll
    for (int e = 0; e < kE; e += 2) {
      const float2 v = s < t.splits ? *reinterpret_cast<const float2*>(part + e) : make_float2(0.f, 0.f);
      acc[s][e] = v.x;
      acc[s][e + 1] = v.y;
    }
  }
  float M = ml.x;
#pragma unroll
  for (int o = kMaxSplits / 2; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
  M = __shfl_sync(0xffffffffu, M, 0);
  const float weight = lane < t.splits ? exp2f(ml.x - M) : 0.f;
  float l = weight * ml.y, out[kE] = {};
#pragma unroll
  for (int o = kMaxSplits / 2; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  l = __shfl_sync(0xffffffffu, l, 0);
#pragma unroll
  for (int s = 0; s < kMaxSplits; ++s) {
    const float f = __shfl_sync(0xffffffffu, weight, s);
    if (s < t.splits) {
#pragma unroll
      for (int e = 0; e < kE; ++e) out[e] = fmaf(f, acc[s][e], out[e]);
    }
  }
  T* dst = static_cast<T*>(p.out) + ((int64_t)token * p.num_q_heads + head) * D + kE * lane;
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < kE; e += 2) decode::store2(dst + e, out[e] * inv, out[e + 1] * inv);
}

namespace {

// What the prefill kernel and the joining one both read.
void set_call(const cb_attention_args& a, const Parts& parts, Params* out) {
  Params& p = *out;
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
  const double scale_log2 = (double)a.scale * 1.4426950408889634;
  p.scale_log2 = (float)scale_log2;
  p.scale_log2_low = p.scale_log2 != 0.f ? (float)((scale_log2 - p.scale_log2) / p.scale_log2) : 0.f;
  p.window = a.sliding_window;
  p.splits = parts.splits;
  p.part_ml = parts.ml;
  p.part_acc = parts.acc;
}

template <typename T, int D>
cb_status launch_kernel(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                        int64_t scale_stride, const Parts& parts, uint32_t* error_word,
                        cudaStream_t stream) {
  auto kern = prefill_kernel<T, D>;
  static std::atomic<uint8_t> attr_set[kMaxDevices];
  cb_status st = ensure_smem_attr(reinterpret_cast<const void*>(kern), Smem<D>::total, attr_set);
  if (st != CB_OK) return st;
  const int64_t n = ctas(a) * parts.splits;
  if (n <= 0) return CB_OK;
  if (n >= ((int64_t)1 << 31)) return CB_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)a.num_blocks * a.num_kv_heads * kPage;
  if (rows >= ((int64_t)1 << 31) - kPage) return CB_ERR_UNSUPPORTED;
  Params p{};
  st = cached_cache_map(&p.tmap_k, a.k_cache, rows, D, 1);
  if (st != CB_OK) return st;
  st = cached_cache_map(&p.tmap_v, a.v_cache, rows, D, 1);
  if (st != CB_OK) return st;
  p.v_cache = static_cast<const uint8_t*>(a.v_cache);
  p.k_scales = k_scales;
  p.v_scales = v_scales;
  p.scale_stride = scale_stride;
  set_call(a, parts, &p);
  p.error_word = error_word;
  p.wait_ns = wait_limit_ns();
  p.withhold_tile = withheld_prefill_tile();
  kern<<<(unsigned)n, kThreads, Smem<D>::total, stream>>>(p);
  const cudaError_t e = cudaGetLastError();
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

int splits(const cb_attention_args& a, int64_t slots) {
  const int64_t n = ctas(a);
  if (n <= 0) return 1;
  // keys that a pair of query tiles may see
  int64_t keys = a.max_seq_len;
  if (a.sliding_window > 0) keys = std::min<int64_t>(keys, (int64_t)a.sliding_window + 2 * kBM);
  int64_t s = sm_count_current_device() / n;
  s = std::min<int64_t>(s, kMaxSplits);
  s = std::min<int64_t>(s, keys / (kBN * kLeastTiles));
  s = std::min<int64_t>(s, slots / a.num_tokens);
  return s < 2 ? 1 : (int)s;
}

cb_status launch(const cb_attention_args& a, const uint8_t* k_scales, const uint8_t* v_scales,
                 int64_t scale_stride, const Parts& parts, uint32_t* error_word, cudaStream_t stream) {
  if (a.num_q_heads / a.num_kv_heads > kBM) return CB_ERR_UNSUPPORTED;
#define CB_PRE(T, DD) \
  return launch_kernel<T, DD>(a, k_scales, v_scales, scale_stride, parts, error_word, stream)
  if (a.dtype == CB_DTYPE_F32) {
    if (a.head_dim == 64) CB_PRE(float, 64);
    CB_PRE(float, 128);
  }
  if (a.head_dim == 64) CB_PRE(__nv_bfloat16, 64);
  CB_PRE(__nv_bfloat16, 128);
#undef CB_PRE
}

cb_status join(const cb_attention_args& a, const Parts& parts, cudaStream_t stream) {
  Params p{};
  set_call(a, parts, &p);
  const unsigned n = (unsigned)(((int64_t)a.num_tokens * a.num_q_heads + 7) / 8);
  if (a.dtype == CB_DTYPE_F32) {
    if (a.head_dim == 64) join_kernel<float, 64><<<n, 256, 0, stream>>>(p);
    else join_kernel<float, 128><<<n, 256, 0, stream>>>(p);
  } else {
    if (a.head_dim == 64) join_kernel<__nv_bfloat16, 64><<<n, 256, 0, stream>>>(p);
    else join_kernel<__nv_bfloat16, 128><<<n, 256, 0, stream>>>(p);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "prefill join launch: %s", cudaGetErrorString(e));
  return CB_OK;
}

}  // namespace prefill_q8
}  // namespace cb
