// cb_step_tables / cb_trim_tables: block tables, slot maps and positions
// built on the GPU from the rows' lengths.
//
// "vLLM serving internals", PagedAttention as a virtual memory system: a
// sequence's block table maps positions to physical blocks, which come from
// a free list and go back to it.  A row with n cached tokens and q new ones
// takes need = pages(n + q) - pages(n) blocks.  With exclusive prefix sums
// over the rows of q (tok) and of need (blk), row r's new page j is
// ring[(head + blk[r] + j) % N], token t of row r has position n + t -
// tok[r], and its slot follows from the table entry of its page -- so after
// one scan over the rows every token and page is written independently.
//
// Nothing here is bound by bytes (a few words per row, token and page): a
// call costs its launch, two rounds of dependent loads (lengths, then ring)
// and a scan.  So it is ONE launch: every CTA of a thread-block cluster
// scans all rows for itself in shared memory, one cluster barrier separates
// the reads of the state from its writes, and the CTAs share the tokens and
// pages.  No atomics and no scratch: the order of the blocks is the rows'.
// Measured on the GPU alone, a step and the trim that takes it back: 64 rows
// of one token 9.5 us, 1000 rows of 37k tokens in all 14.9 us (the bytes of
// the latter take 0.06 us).
#include <cuda_runtime.h>

#include "cb_error.h"
#include "device_utils.cuh"
#include "launch_common.h"

namespace cb {
namespace tables {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxRows = CB_TABLES_MAX_ROWS;

struct Params {
  cb_tables t;
  int32_t shift;                // log2 of the block size
  const int32_t* lens;          // q_lens, or keep_lens
  int32_t max_tokens;
  int32_t* cu_seqlens_q;
  int32_t* seq_lens;
  int32_t* slot_mapping;
  int32_t* positions;
  int32_t vec;                  // slot_mapping and positions are 16-byte aligned
};

// Per-row arrays in shared memory (R rows): 5 R + 2 words.
struct Rows {
  int32_t* tok;     // [R + 1] tokens of the rows before
  int32_t* blk;     // [R + 1] pages of the rows before
  int32_t* take;    // [R] tokens appended (trim: unused)
  int32_t* need;    // [R] pages taken or given back
  int32_t* cached;  // [R]
};
__device__ __forceinline__ Rows rows_of(int32_t* smem, int R) {
  return Rows{smem, smem + R + 1, smem + 2 * R + 2, smem + 3 * R + 2, smem + 4 * R + 2};
}
constexpr size_t rows_bytes(int64_t R) { return (size_t)(5 * R + 2) * 4; }

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ int32_t clamp31(int64_t x) {
  return (int32_t)(x < 0x7fffffff ? x : 0x7fffffff);
}

// tok and blk from take and need, over all rows; thread i writes the entries
// of its own rows [b, e).  Sums are 64-bit; entries saturate at 2^31 - 1
// (then the totals pass every limit and the rows behind are dropped).
__device__ __forceinline__ void scan_rows(const Rows& s, int R, int b, int e, int64_t& total_tok,
                                          int64_t& total_blk, int64_t (*red)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t a = 0, c = 0;
  for (int r = b; r < e; ++r) {
    a += s.take[r];
    c += s.need[r];
  }
  int64_t ia = a, ic = c;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t va = __shfl_up_sync(0xffffffffu, ia, o);
    const int64_t vc = __shfl_up_sync(0xffffffffu, ic, o);
    if (lane >= o) {
      ia += va;
      ic += vc;
    }
  }
  if (lane == 31) {
    red[warp][0] = ia;
    red[warp][1] = ic;
  }
  __syncthreads();
  int64_t run_a = ia - a, run_c = ic - c;
  total_tok = total_blk = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const int64_t ra = red[w][0], rc = red[w][1];
    if (w < warp) {
      run_a += ra;
      run_c += rc;
    }
    total_tok += ra;
    total_blk += rc;
  }
  for (int r = b; r < e; ++r) {
    s.tok[r] = clamp31(run_a);
    s.blk[r] = clamp31(run_c);
    run_a += s.take[r];
    run_c += s.need[r];
  }
  if (threadIdx.x == 0) {
    s.tok[R] = clamp31(total_tok);
    s.blk[R] = clamp31(total_blk);
  }
  __syncthreads();  // the prefixes are complete, and red may be rewritten
}

// Largest row r with prefix[r] <= i (prefix[0] = 0 <= i < prefix[R]).
__device__ __forceinline__ int find_row(const int32_t* prefix, int rows, int i) {
  int lo = 0, hi = rows - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (prefix[mid] <= i) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int ring_at(int head, int i, int n) {
  const int64_t x = (int64_t)head + i;
  return (int)(x < n ? x : x - n);
}

// head and count of the ring; a state that is no ring counts as empty
__device__ __forceinline__ void load_ring(const Params& p, int& head, int& count, bool& bad) {
  head = p.t.free_state[0];
  count = p.t.free_state[1];
  bad = head < 0 || head >= p.t.num_blocks || count < 0 || count > p.t.num_blocks;
  if (bad) head = count = 0;
}

__device__ __forceinline__ int pages_of(int64_t n, int shift) {
  return (int)((n + (1 << shift) - 1) >> shift);
}

__global__ void __launch_bounds__(kThreads) step_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t red[kWarps][2];
  const int R = p.t.num_rows, W = p.t.max_blocks_per_seq, N = p.t.num_blocks;
  const Rows s = rows_of(smem, R);
  const uint32_t rank = cluster_rank();
  const int64_t most = (int64_t)W << p.shift;
  const int in_block = (1 << p.shift) - 1;
  int head, count;
  bool bad_ring;
  load_ring(p, head, count, bad_ring);
  uint32_t errors = bad_ring ? CB_DEVERR_NO_BLOCKS : 0u;
  const int seg = (R + kThreads - 1) / kThreads;
  const int b = min((int)threadIdx.x * seg, R), e = min(b + seg, R);
  for (int r = b; r < e; ++r) {
    const int q = p.lens[r], n = p.t.cached_lens[r];
    const bool ok = q >= 0 && n >= 0 && (int64_t)n + q <= most;
    if (!ok) errors |= CB_DEVERR_SEQ_RANGE;
    s.cached[r] = n;
    s.take[r] = ok ? q : 0;
    s.need[r] = ok ? pages_of((int64_t)n + q, p.shift) - pages_of(n, p.shift) : 0;
  }
  int64_t total_tok, total_blk;
  scan_rows(s, R, b, e, total_tok, total_blk, red);
  // rows past the token capacity, then rows past the free blocks, are
  // dropped (a row's own prefixes tell, and they grow with the row)
  if (total_tok > p.max_tokens) {
    for (int r = b; r < e; ++r)
      if (s.take[r] > 0 && (int64_t)s.tok[r] + s.take[r] > p.max_tokens) {
        s.take[r] = s.need[r] = 0;
        errors |= CB_DEVERR_SEQ_RANGE;
      }
    scan_rows(s, R, b, e, total_tok, total_blk, red);
  }
  if (total_blk > count) {
    for (int r = b; r < e; ++r)
      if (s.need[r] > 0 && (int64_t)s.blk[r] + s.need[r] > count) {
        s.take[r] = s.need[r] = 0;
        errors |= CB_DEVERR_NO_BLOCKS;
      }
    scan_rows(s, R, b, e, total_tok, total_blk, red);
  }
  // every CTA of the cluster has read the lengths and the ring's state
  cluster_sync();

  if (rank == 0) {
    if (errors) set_error(p.t.error_word, errors);
    for (int r = threadIdx.x; r < R; r += kThreads) {
      const int q = s.take[r];
      p.cu_seqlens_q[r] = s.tok[r];
      p.seq_lens[r] = q > 0 ? s.cached[r] + q : 0;
      if (q > 0) p.t.cached_lens[r] = s.cached[r] + q;
    }
    if (threadIdx.x == 0) {
      p.cu_seqlens_q[R] = (int32_t)total_tok;
      if (total_blk > 0) {
        p.t.free_state[0] = ring_at(head, (int)total_blk, N);
        p.t.free_state[1] = count - (int)total_blk;
      }
    }
  }
  const int workers = (int)cluster_size() * kThreads;
  const int me = (int)rank * kThreads + threadIdx.x;
  const int tokens = (int)total_tok, pages = (int)total_blk;
  // pages: the new table entries
  for (int i = me; i < pages; i += workers) {
    const int r = find_row(s.blk, R, i);
    const int page = pages_of(s.cached[r], p.shift) + i - s.blk[r];
    const int id = p.t.free_ring[ring_at(head, i, N)];
    if (id < 0 || id >= N) set_error(p.t.error_word, CB_DEVERR_BLOCK_RANGE);
    p.t.block_tables[(int64_t)r * W + page] = id;
  }
  // tokens, four neighbours to a thread
  for (int t0 = me * 4; t0 < p.max_tokens; t0 += workers * 4) {
    int slot[4], pos[4];
    int r = t0 < tokens ? find_row(s.tok, R, t0) : 0;
    int page_of = -1, base = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = t0 + i;
      slot[i] = -1;
      pos[i] = 0;
      if (t < tokens) {
        while (t >= s.tok[r + 1]) {
          ++r;
          page_of = -1;
        }
        const int n = s.cached[r];
        pos[i] = n + t - s.tok[r];
        const int page = pos[i] >> p.shift;
        if (page != page_of) {
          // the row's last page may be part filled; later ones come from the ring
          const int kept = pages_of(n, p.shift);
          const int id = page < kept ? p.t.block_tables[(int64_t)r * W + page]
                                     : p.t.free_ring[ring_at(head, s.blk[r] + page - kept, N)];
          page_of = page;
          base = id;
          if (id < 0 || id >= N) {
            base = -1;
            set_error(p.t.error_word, CB_DEVERR_BLOCK_RANGE);
          }
        }
        if (base >= 0) slot[i] = (base << p.shift) + (pos[i] & in_block);
      }
    }
    if (p.vec && t0 + 4 <= p.max_tokens) {
      *reinterpret_cast<int4*>(p.slot_mapping + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(p.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (t0 + i < p.max_tokens) {
          p.slot_mapping[t0 + i] = slot[i];
          p.positions[t0 + i] = pos[i];
        }
    }
  }
}

__global__ void __launch_bounds__(kThreads) trim_kernel(const __grid_constant__ Params p) {
  extern __shared__ int32_t smem[];
  __shared__ int64_t red[kWarps][2];
  const int R = p.t.num_rows, W = p.t.max_blocks_per_seq, N = p.t.num_blocks;
  const Rows s = rows_of(smem, R);
  const uint32_t rank = cluster_rank();
  int head, count;
  bool bad_ring;
  load_ring(p, head, count, bad_ring);
  uint32_t errors = bad_ring ? CB_DEVERR_NO_BLOCKS : 0u;
  const int room = bad_ring ? 0 : N - count;
  const int seg = (R + kThreads - 1) / kThreads;
  const int b = min((int)threadIdx.x * seg, R), e = min(b + seg, R);
  // take[r]: 1 for a row that is shortened
  for (int r = b; r < e; ++r) {
    const int keep = p.lens[r], n = p.t.cached_lens[r];
    const bool ok = keep <= n && n >= 0 && pages_of(n, p.shift) <= W;
    const bool cut = ok && keep >= 0 && keep < n;
    if (!ok && keep >= 0) errors |= CB_DEVERR_SEQ_RANGE;
    s.cached[r] = n;
    s.take[r] = cut ? 1 : 0;
    s.need[r] = cut ? pages_of(n, p.shift) - pages_of(keep, p.shift) : 0;
  }
  int64_t total_tok, total_blk;
  scan_rows(s, R, b, e, total_tok, total_blk, red);
  if (total_blk > room) {
    for (int r = b; r < e; ++r)
      if (s.need[r] > 0 && (int64_t)s.blk[r] + s.need[r] > room) {
        s.take[r] = s.need[r] = 0;
        errors |= CB_DEVERR_NO_BLOCKS;
      }
    scan_rows(s, R, b, e, total_tok, total_blk, red);
  }
  // every CTA of the cluster has read the lengths and the ring's state
  cluster_sync();

  if (rank == 0) {
    if (errors) set_error(p.t.error_word, errors);
    for (int r = threadIdx.x; r < R; r += kThreads)
      if (s.take[r]) p.t.cached_lens[r] = p.lens[r];
    if (threadIdx.x == 0 && total_blk > 0) p.t.free_state[1] = count + (int)total_blk;
  }
  const int tail = ring_at(head, count, N);
  const int pages = (int)total_blk;
  for (int i = (int)rank * kThreads + threadIdx.x; i < pages; i += (int)cluster_size() * kThreads) {
    const int r = find_row(s.blk, R, i);
    int32_t* entry = p.t.block_tables + (int64_t)r * W +
                     (pages_of(s.cached[r], p.shift) - s.need[r] + i - s.blk[r]);
    const int id = *entry;
    if (id < 0 || id >= N) set_error(p.t.error_word, CB_DEVERR_BLOCK_RANGE);
    p.t.free_ring[ring_at(tail, i, N)] = id;
    *entry = -1;
  }
}

namespace {

cb_status check(const cb_tables* t, const int32_t* lens, const char* what) {
  if (!t) return fail(CB_ERR_INVALID_ARG, "%s: tables is NULL", what);
  if (t->num_rows <= 0 || t->max_blocks_per_seq <= 0 || t->num_blocks <= 0 || t->block_size <= 0)
    return fail(CB_ERR_INVALID_ARG, "%s: sizes must be positive", what);
  if (!t->cached_lens || !t->block_tables || !t->free_ring || !t->free_state || !lens)
    return fail(CB_ERR_INVALID_ARG, "%s: NULL pointer", what);
  if ((t->block_size & (t->block_size - 1)) != 0)
    return fail(CB_ERR_UNSUPPORTED, "%s: block_size must be a power of two", what);
  if (t->num_rows > kMaxRows)
    return fail(CB_ERR_UNSUPPORTED, "%s: more than %d rows", what, kMaxRows);
  if ((int64_t)t->num_blocks * t->block_size > ((int64_t)1 << 31) ||
      (int64_t)t->max_blocks_per_seq * t->block_size > ((int64_t)1 << 31) - 1)
    return fail(CB_ERR_UNSUPPORTED, "%s: slots or positions pass 2^31", what);
  return CB_OK;
}

using Kernel = void (*)(Params);

cb_status launch(Kernel kernel, const Params& p, int64_t items, std::atomic<uint8_t>* attr_set,
                 cudaStream_t stream, const char* what) {
  cb_status st = ensure_smem_attr(reinterpret_cast<const void*>(kernel), rows_bytes(kMaxRows), attr_set);
  if (st != CB_OK) return st;
  cudaLaunchConfig_t cfg{};
  // one CTA while its threads hold every token and row at once (and every page
  // that a trim may give back, at one to a thread), else the portable cluster
  // size (step and trim of 64 rows, 64 tokens: 9.6 us, 9.8 with a cluster for
  // both; 80 rows, 10k tokens: 10.5 us with eight, 16.1 with one; a trim alone
  // that gives back 64 pages 9.3 us either way, 4096 9.3 and 13.5, 131k 25.7
  // and 148.6)
  const unsigned ctas = items <= kThreads * 4 ? 1 : 8;
  cfg.gridDim = dim3(ctas, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.dynamicSmemBytes = rows_bytes(p.t.num_rows);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess) return fail(CB_ERR_CUDA, "%s launch: %s", what, cudaGetErrorString(e));
  return CB_OK;
}

Params params_of(const cb_tables& t, const int32_t* lens) {
  Params p{};
  p.t = t;
  p.lens = lens;
  while ((1 << p.shift) < t.block_size) ++p.shift;
  return p;
}

}  // namespace
}  // namespace tables
}  // namespace cb

extern "C" cb_status cb_step_tables(const cb_tables* tables, const int32_t* q_lens, int32_t max_tokens,
                                    int32_t* cu_seqlens_q, int32_t* seq_lens, int32_t* slot_mapping,
                                    int32_t* positions, cb_stream_t stream) {
  using namespace cb::tables;
  cb_status st = check(tables, q_lens, "cb_step_tables");
  if (st != CB_OK) return st;
  if (max_tokens < 0) return cb::fail(CB_ERR_INVALID_ARG, "cb_step_tables: max_tokens < 0");
  if (!cu_seqlens_q || !seq_lens || (max_tokens > 0 && (!slot_mapping || !positions)))
    return cb::fail(CB_ERR_INVALID_ARG, "cb_step_tables: NULL pointer");
  Params p = params_of(*tables, q_lens);
  p.max_tokens = max_tokens;
  p.cu_seqlens_q = cu_seqlens_q;
  p.seq_lens = seq_lens;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.vec = (((uintptr_t)slot_mapping | (uintptr_t)positions) & 15u) == 0;
  static std::atomic<uint8_t> attr_set[cb::kMaxDevices];
  const int64_t items = max_tokens > tables->num_rows * 4ll ? max_tokens : tables->num_rows * 4ll;
  return launch(step_kernel, p, items, attr_set, (cudaStream_t)stream, "cb_step_tables");
}

extern "C" cb_status cb_trim_tables(const cb_tables* tables, const int32_t* keep_lens,
                                    cb_stream_t stream) {
  using namespace cb::tables;
  cb_status st = check(tables, keep_lens, "cb_trim_tables");
  if (st != CB_OK) return st;
  const Params p = params_of(*tables, keep_lens);
  static std::atomic<uint8_t> attr_set[cb::kMaxDevices];
  const int64_t entries = (int64_t)tables->num_rows * tables->max_blocks_per_seq;
  const int64_t pages = entries < tables->num_blocks ? entries : tables->num_blocks;
  const int64_t items = (pages > tables->num_rows ? pages : tables->num_rows) * 4;
  return launch(trim_kernel, p, items, attr_set, (cudaStream_t)stream, "cb_trim_tables");
}
