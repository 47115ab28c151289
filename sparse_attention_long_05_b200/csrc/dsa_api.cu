// libdsa.so: C ABI of the DSA forward path on B200 (declarations and contracts in include/dsa.h).
//
// Host side only: argument checks, TMA tensor-map construction, launch configuration and the order of the
// kernels of the prefill and decode drivers.  Every step of the computation runs in the kernels included
// below.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <algorithm>
#include <atomic>
#include <mutex>
#include <vector>

#include "common.cuh"
#include "indexer.cuh"
#include "indexer_bwd.cuh"
#include "rope.cuh"
#include "scatter.cuh"
#include "sparse_mla.cuh"
#include "sparse_mla_bwd.cuh"
#include "topk.cuh"
#include "topk_cluster.cuh"

namespace dsa {

// ------------------------------------------------------------------------------------------ decode append
// Writes the new token's indexer key (+ scale) and latent entry at position ctx_len[b] of sequence b, n_b + 1
// into len1[b] (the number of keys the new token attends to) and the start of the sequence's score row into
// score_off[b].  Score rows are packed in sequence order, each padded to a multiple of 4 floats, so that every
// row starts on a 16-byte boundary (the top-k reads rows with 16-byte loads); they do not follow the cache
// layout.  A sequence whose cache range is invalid (cache_off < 0, ctx_len < 0, or the new row outside the
// cache) or whose score row would not fit in score_cap floats raises DSA_ERR_BAD_INDEX and gets len1 = 0: no
// kernel after this one reads or writes anything of it.

__device__ __forceinline__ bool decode_seq_valid(const long long* cache_off, const int* ctx_len,
                                                 long long cache_rows, int b) {
  const long long off = cache_off[b];
  const int n = ctx_len[b];
  return off >= 0 && n >= 0 && off + n < cache_rows;
}

// Paged caches: the caches are pools of pages of page_rows rows; row (page_table[b][pos / page_rows] * page_rows +
// pos % page_rows) holds position pos of sequence b.  A sequence is valid when its new position ctx_len[b] falls
// inside its table and every page up to it is in [0, num_pages).  Every thread of the CTA calls this.
__device__ __forceinline__ bool decode_seq_valid_paged(const int* page_table, int max_pages, int page_rows,
                                                       long long num_pages, const int* ctx_len, int b) {
  __shared__ int bad;
  const int n = ctx_len[b];
  if (threadIdx.x == 0) bad = (n < 0 || n / page_rows >= max_pages) ? 1 : 0;
  __syncthreads();
  if (!bad) {
    const int* row = page_table + static_cast<long long>(b) * max_pages;
    for (int j = threadIdx.x; j <= n / page_rows; j += blockDim.x)
      if (row[j] < 0 || row[j] >= num_pages) bad = 1;
  }
  __syncthreads();
  return bad == 0;
}

__device__ __forceinline__ long long padded4(long long n) { return (n + 3) & ~3ll; }

constexpr int kAppendThreads = 128;

// Cache layout of a decode step: flat (sequence b owns rows cache_off[b] ..) or paged (page_table non-null).
struct DecodeLayout {
  const long long* cache_off;   // flat: [B]
  long long cache_rows;         // flat: rows of the caches
  const int* page_table;        // paged: [B, max_pages], or null
  int max_pages, page_rows;
  long long num_pages;
};

__global__ void __launch_bounds__(kAppendThreads)
    decode_append_kernel(int B, DecodeLayout lay, const int* ctx_len, const uint8_t* k_new,
                         const float* k_scale_new, const uint16_t* c_new, uint8_t* k_cache, float* k_scale_cache,
                         uint16_t* c_cache, int d_I, int* len1, long long* score_off, long long score_cap,
                         unsigned* hist) {
  pdl_allow_next();
  pdl_wait();
  const int b = blockIdx.x;
  if (b >= B) return;
  // the sequence's score histogram, accumulated by the indexer (when the step uses one)
  if (hist)
    for (int i = threadIdx.x; i < kTopkBins; i += blockDim.x) hist[static_cast<long long>(b) * kTopkBins + i] = 0;
  // start of this sequence's score row: the padded lengths of the sequences before it that pass the cheap part
  // of their check (paged: the page-table entries of another sequence are not read here; a sequence that fails
  // only on those keeps its reserved row unused)
  __shared__ long long part[kAppendThreads / 32];
  long long acc = 0;
  for (int j = threadIdx.x; j < b; j += blockDim.x) {
    const int nj = ctx_len[j];
    if (lay.page_table ? (nj >= 0 && nj / lay.page_rows < lay.max_pages)
                       : decode_seq_valid(lay.cache_off, ctx_len, lay.cache_rows, j))
      acc += padded4(static_cast<long long>(nj) + 1);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
  __syncthreads();
  long long s0 = 0;
#pragma unroll
  for (int w = 0; w < kAppendThreads / 32; ++w) s0 += part[w];
  const bool fits = s0 + padded4(static_cast<long long>(ctx_len[b]) + 1) <= score_cap;
  const bool valid = (lay.page_table ? decode_seq_valid_paged(lay.page_table, lay.max_pages, lay.page_rows,
                                                              lay.num_pages, ctx_len, b)
                                     : decode_seq_valid(lay.cache_off, ctx_len, lay.cache_rows, b)) && fits;
  if (!valid) {
    if (threadIdx.x == 0) { raise_status(DSA_ERR_BAD_INDEX); len1[b] = 0; score_off[b] = 0; }
    return;
  }
  const int n = ctx_len[b];
  const long long row = lay.page_table
      ? static_cast<long long>(lay.page_table[static_cast<long long>(b) * lay.max_pages + n / lay.page_rows]) *
            lay.page_rows + n % lay.page_rows
      : lay.cache_off[b] + n;
  const uint4* ks = reinterpret_cast<const uint4*>(k_new + static_cast<long long>(b) * d_I);
  uint4* kd = reinterpret_cast<uint4*>(k_cache + row * d_I);
  for (int i = threadIdx.x; i < d_I / 16; i += blockDim.x) kd[i] = ks[i];
  const uint4* cs = reinterpret_cast<const uint4*>(c_new + static_cast<long long>(b) * mla::D);
  uint4* cd = reinterpret_cast<uint4*>(c_cache + row * mla::D);
  for (int i = threadIdx.x; i < mla::D * 2 / 16; i += blockDim.x) cd[i] = cs[i];
  if (threadIdx.x == 0) {
    k_scale_cache[row] = k_scale_new[b];
    len1[b] = ctx_len[b] + 1;
    score_off[b] = s0;
  }
}

// ------------------------------------------------------------------------------------------ varlen prefill
// Row offset of every token of a packed batch of sequences: the first row of its own sequence (the largest b
// with cu[b] <= t, so an empty sequence never owns a token).
__global__ void varlen_row_off_kernel(const long long* cu, int nseq, long long total, long long* row_off) {
  const long long t = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (t >= total) return;
  int lo = 0, hi = nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  row_off[t] = cu[lo];
}

// Score-row offset and length of every row of a group of packed sequences for the top-k: row r of sequence b at
// position t reads the t + 1 scores at seq_off[b] + (t - k) * seq_ld[b] (rows t < k read nothing: every earlier key
// is selected).  cu: the group's sequence starts relative to its first row, nseq + 1 entries.
__global__ void varlen_score_rows_kernel(const long long* cu, int nseq, const long long* seq_off, const int* seq_ld,
                                         int k, long long* row_off, int* row_len) {
  pdl_allow_next();
  pdl_wait();
  const long long r = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (r >= cu[nseq]) return;
  int lo = 0, hi = nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= r) lo = mid; else hi = mid - 1;
  }
  const long long t = r - cu[lo];
  row_len[r] = static_cast<int>(t + 1);
  row_off[r] = (t >= k) ? seq_off[lo] + (t - k) * seq_ld[lo] : 0;
}

// ------------------------------------------------------------------------------------------ bounded-wait self-check
// One CTA of two warps exercises the bounded mbarrier wait every pipeline of the library uses, on barriers
// that nothing arrives on.  Warp 0 waits from the start and runs out of budget (g_wait_limit cycles, about a
// second): it records DSA_ERR_TIMEOUT and raises the CTA's abort flag.  Warp 1 starts its wait half a budget
// later and must leave on the abort flag, well before its own budget ends.  result[2w] = 1 if warp w's wait
// succeeded, result[2w + 1] = its wait in units of 2^20 cycles.
__global__ void __launch_bounds__(64) wait_selfcheck_kernel(int* result) {
  __shared__ __align__(8) uint64_t bars[2];
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&bars[0]), 1);
    mbar_init(smem_u32(&bars[1]), 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  if (lane != 0) return;
  if (warp == 1) {
    const long long t0 = clock64();
    while (clock64() - t0 < (g_wait_limit >> 1)) {
    }
  }
  const long long t0 = clock64();
  const bool ok = mbar_wait(smem_u32(&bars[warp]), 0, &abort_flag);
  result[2 * warp] = ok ? 1 : 0;
  result[2 * warp + 1] = static_cast<int>((clock64() - t0) >> 20);
}

// ------------------------------------------------------------------------------------------ host helpers
namespace {

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// rank-2/3 tensor map; dims / strides innermost first (strides in bytes, rank-1 entries)
bool make_map(CUtensorMap* m, CUtensorMapDataType dt, int rank, const void* base, const cuuint64_t* dims,
              const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle sw) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, dt, rank, const_cast<void*>(base), dims, strides, box, es, CU_TENSOR_MAP_INTERLEAVE_NONE, sw,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int num_sms() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 148;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  return n;
}

template <typename K>
cudaError_t set_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

std::atomic<unsigned long long> g_launches{0};

// Launch with programmatic stream serialisation (see pdl_wait): the kernel may be scheduled while its predecessor
// on the stream finishes, and waits for it on the device.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                       Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
}

// launch_pdl of a kernel with more dynamic shared memory than the default: the attribute that allows it is set at the
// kernel's first launch on a device (`seen`: one bit a device), and once more where a launch is refused without it
// (after a cudaDeviceReset); setting it on every call costs about as much as a third of a launch.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl_large(std::atomic<unsigned long long>& seen, void (*kernel)(KArgs...), dim3 grid, dim3 block,
                             size_t smem, cudaStream_t st, Args... args) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = 1ull << (dev & 63);
  const bool known = dev < 64 && (seen.load(std::memory_order_relaxed) & bit);
  if (known) {
    e = launch_pdl(kernel, grid, block, smem, st, args...);
    if (e != cudaErrorInvalidValue) return e;
    cudaGetLastError();
  }
  if ((e = set_smem(kernel, static_cast<int>(smem))) != cudaSuccess) return e;
  if (dev < 64) seen.fetch_or(bit, std::memory_order_relaxed);
  return launch_pdl(kernel, grid, block, smem, st, args...);
}

dsa_status_t last_launch_status() {
  g_launches.fetch_add(1, std::memory_order_relaxed);
  return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// floats of the decode score rows: every valid sequence's n_b + 1 keys, padded to a multiple of 4; sequences
// own disjoint cache ranges, so the rows need at most cache_rows + 3 B floats
size_t decode_score_cap(int B, int64_t cache_rows) { return size_t(cache_rows) + 4 * size_t(B); }

// ------------------------------------------------------------------------------------------ launchers
// A configuration that allocates all 512 TMEM columns runs one CTA per SM: at least 120 KB of shared memory is
// requested to keep a second CTA off the SM (its allocation would wait for the first CTA to finish).
constexpr int kMinIndexerSmem = 120 * 1024;

template <int H_I, int D_I, int NT, int NG, int QBUF, int KST, int EPI, int MODE>
dsa_status_t launch_indexer(const uint8_t* q_idx, int q_rows, const uint8_t* k_idx, long long k_rows,
                            const IndexerParams& p, int grid, cudaStream_t st) {
  using C = IndexerCfg<H_I, D_I, NT, NG, QBUF, KST, EPI, MODE>;
  CUtensorMap tq, tk;
  const cuuint64_t qd[2] = {static_cast<cuuint64_t>(D_I), static_cast<cuuint64_t>(q_rows) * H_I};
  const cuuint64_t qs[1] = {static_cast<cuuint64_t>(D_I)};
  const cuuint32_t qb[2] = {static_cast<cuuint32_t>(D_I), static_cast<cuuint32_t>(C::N)};
  const cuuint64_t kd[2] = {static_cast<cuuint64_t>(D_I), static_cast<cuuint64_t>(k_rows)};
  const cuuint32_t kb[2] = {static_cast<cuuint32_t>(D_I), 128u};
  const CUtensorMapSwizzle sw = (D_I == 128) ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  if (!make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, q_idx, qd, qs, qb, sw)) return DSA_ERR_CUDA;
  if (!make_map(&tk, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, k_idx, kd, qs, kb, sw)) return DSA_ERR_CUDA;
  auto kern = indexer_kernel<H_I, D_I, NT, NG, QBUF, KST, EPI, MODE>;
  IndexerParams pk = p;
  pk.k_rows = k_rows;
  pk.q_rows = q_rows;
  const int smem = (C::TMEM_COLS == 512 && C::SMEM < kMinIndexerSmem) ? kMinIndexerSmem : C::SMEM;
  if (set_smem(kern, smem) != cudaSuccess) return DSA_ERR_CUDA;
  if (launch_pdl(kern, dim3(grid), dim3(C::NUM_THREADS), smem, st, tq, tk, pk) != cudaSuccess) return DSA_ERR_CUDA;
  return last_launch_status();
}

// scores [T, S] of query rows at positions pos0.. against keys 0..S-1 (materialised)
dsa_status_t run_indexer_scores(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                const float* k_scale, const float* w, int T, int S, int H_I, int d_I, int pos0,
                                float* scores, long long ld, cudaStream_t st) {
  IndexerParams p{};
  p.w = w;
  p.q_scale = q_scale;
  p.k_scale = k_scale;
  p.scores = scores;
  p.ld = ld;
  p.T = T;
  p.S = S;
  p.pos0 = pos0;
  const int tok = (H_I == 64) ? 16 : 256;
  const int nqb = (T + tok - 1) / tok;
  const int ntiles = (S + 127) / 128;
  // Work items (query block x key-tile range) go round-robin to one persistent CTA per SM.  The key range is
  // split so that the items divide evenly over the SMs: cost = rounds x (tiles per item + ~2 tiles of per-item
  // setup: query block load, pipeline fill), the fewest splits winning ties.
  const int sms = num_sms();
  int best_split = 1;
  double best_cost = 1e300;
  for (int ns = 1; ns <= (ntiles < 64 ? ntiles : 64); ++ns) {
    const int per = (ntiles + ns - 1) / ns;
    const long long items = static_cast<long long>(nqb) * ((ntiles + per - 1) / per);
    const double cost = static_cast<double>((items + sms - 1) / sms) * (per + 2.0);
    if (cost < best_cost - 1e-9) { best_cost = cost; best_split = per; }
  }
  p.split_tiles = best_split;
  p.nsplit = (ntiles + p.split_tiles - 1) / p.split_tiles;
  p.n_items = nqb * p.nsplit;
  const int grid = p.n_items < sms ? p.n_items : sms;
  if (H_I == 64)
    return launch_indexer<64, 128, 4, 4, 1, 4, 2, kModeScores>(q_idx, T, k_idx, S, p, grid, st);
  return launch_indexer<4, 64, 64, 4, 1, 4, 2, kModeScores>(q_idx, T, k_idx, S, p, grid, st);
}

// Indexer scores of the runs of query rows in segs_host (one launch; segs_dev: a device copy of the table, written
// by the caller), into `scores`.  Chooses the key split and fills each run's nsplit and item0 in segs_host before
// the caller copies it.  Returns the number of items through *n_items.
void plan_segments(IndexerSeg* segs, int n_segs, int tok, int* split_tiles, int* n_items) {
  const int sms = num_sms();
  int best = 1;
  double best_cost = 1e300;
  for (int split = 1; split <= 64; ++split) {
    long long items = 0;
    for (int i = 0; i < n_segs; ++i) {
      const int nqb = (segs[i].n_rows + tok - 1) / tok, ntiles = (segs[i].S + 127) / 128;
      items += static_cast<long long>(nqb) * ((ntiles + split - 1) / split);
    }
    const double cost = static_cast<double>((items + sms - 1) / sms) * (split + 2.0);
    if (cost < best_cost - 1e-9) { best_cost = cost; best = split; }
  }
  int item = 0;
  for (int i = 0; i < n_segs; ++i) {
    const int nqb = (segs[i].n_rows + tok - 1) / tok, ntiles = (segs[i].S + 127) / 128;
    segs[i].nsplit = (ntiles + best - 1) / best;
    segs[i].item0 = item;
    item += nqb * segs[i].nsplit;
  }
  *split_tiles = best;
  *n_items = item;
}

dsa_status_t run_indexer_segments(const uint8_t* q_idx, long long q_rows, const float* q_scale, const uint8_t* k_idx,
                                  long long k_rows, const float* k_scale, const float* w, int H_I, int d_I,
                                  const IndexerSeg* segs_dev, int n_segs, int split_tiles, int n_items,
                                  float* scores, cudaStream_t st) {
  if (n_items <= 0) return DSA_OK;
  IndexerParams p{};
  p.w = w;
  p.q_scale = q_scale;
  p.k_scale = k_scale;
  p.scores = scores;
  p.segs = segs_dev;
  p.n_segs = n_segs;
  p.split_tiles = split_tiles;
  p.n_items = n_items;
  const int sms = num_sms();
  const int grid = n_items < sms ? n_items : sms;
  if (H_I == 64)
    return launch_indexer<64, 128, 4, 4, 1, 4, 2, kModeSegments>(q_idx, static_cast<int>(q_rows), k_idx, k_rows, p,
                                                                 grid, st);
  return launch_indexer<4, 64, 64, 4, 1, 4, 2, kModeSegments>(q_idx, static_cast<int>(q_rows), k_idx, k_rows, p, grid,
                                                             st);
}

#ifdef DSA_CHECKS
// DSA_CHECKS builds: every output row of a top-k launch holds min(k, n) entries, strictly ascending and in [0, n)
// for the row's n keys, then -1 padding.  One CTA per row; launched without the dependent-launch attribute, so
// it starts once the top-k has finished.
__global__ void __launch_bounds__(256) topk_check_kernel(const TopkParams p) {
  const int r = blockIdx.x;
  const long long n = p.row_len ? p.row_len[r] : (p.ld < p.pos0 + r + 1 ? p.ld : p.pos0 + r + 1);
  const int m = static_cast<int>(n < p.k ? (n > 0 ? n : 0) : p.k);
  const int* row = p.idx + static_cast<long long>(r) * p.idx_ld;
  bool good = true;
  for (int i = threadIdx.x; i < p.k; i += blockDim.x) {
    const int v = row[i];
    if (i < m) good &= v >= 0 && v < n && (i == 0 || v > row[i - 1]);
    else good &= v == -1;
  }
  if (!good) raise_status(DSA_ERR_CHECK);
}
#endif

dsa_status_t run_topk(const float* scores, long long ld, const long long* row_off, const int* row_len, int pos0,
                      int rows, int k, int* idx, long long idx_ld, cudaStream_t st, float* sel_scores = nullptr,
                      const unsigned* hist = nullptr) {
  if (rows <= 0) return DSA_OK;
  TopkParams p{scores, ld, row_off, row_len, pos0, rows, k, idx, idx_ld, sel_scores, hist};
  if (rows < num_sms()) {
    // fewer rows than SMs (decode): one cluster of kTkcCluster CTAs per row
    if (set_smem(topk_cluster_kernel, static_cast<int>(sizeof(TkcSmem))) != cudaSuccess) return DSA_ERR_CUDA;
    if (launch_pdl(topk_cluster_kernel, dim3(rows * kTkcCluster), dim3(kTkcThreads), sizeof(TkcSmem), st, p) !=
        cudaSuccess)
      return DSA_ERR_CUDA;
  } else {
    if (set_smem(topk_rows_kernel<kTopkThreads>, static_cast<int>(sizeof(TopkSmem<kTopkThreads>))) != cudaSuccess)
      return DSA_ERR_CUDA;
    if (launch_pdl(topk_rows_kernel<kTopkThreads>, dim3(rows), dim3(kTopkThreads), sizeof(TopkSmem<kTopkThreads>), st,
                   p) != cudaSuccess)
      return DSA_ERR_CUDA;
  }
#ifdef DSA_CHECKS
  {
    const dsa_status_t e = last_launch_status();
    if (e != DSA_OK) return e;
    topk_check_kernel<<<rows, 256, 0, st>>>(p);
  }
#endif
  return last_launch_status();
}

// Attention launch.  dense: kMlaSparse (every token gathers its index row), kMlaCausal (token t has the
// t - row_off[t] + 1 keys of its sequence) or kMlaCounts (token t has n_keys[t] keys); in the dense modes a
// token with at most k keys attends to all of them, read as contiguous tiles.
dsa_status_t run_mla(const uint16_t* q, const uint16_t* c, long long S, const int* idx, const long long* row_off,
                     int T, int H, int k, float scale, uint16_t* out, float* lse, cudaStream_t st,
                     int dense = kMlaSparse, const int* n_keys = nullptr, const int* page_table = nullptr,
                     int pt_stride = 0, int page_rows = 0, int pos0 = 0, const float* kl_lse = nullptr,
                     const float* kl_scores = nullptr, float* kl_out = nullptr) {
  if (T <= 0) return DSA_OK;
  CUtensorMap tq;
  const cuuint64_t qd[3] = {576, static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t qs[2] = {576 * 2, static_cast<cuuint64_t>(H) * 576 * 2};
  const cuuint32_t qb[3] = {64, 128, 1};
  if (!make_map(&tq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, qd, qs, qb, CU_TENSOR_MAP_SWIZZLE_128B)) return DSA_ERR_CUDA;
  CUtensorMap tc;   // rows of c, one 64-column box high 1 row (the form tile::gather4 takes)
  const cuuint64_t cd[2] = {576, static_cast<cuuint64_t>(S)};
  const cuuint64_t cs[1] = {576 * 2};
  const cuuint32_t cb[2] = {64, 1};
  if (!make_map(&tc, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c, cd, cs, cb, CU_TENSOR_MAP_SWIZZLE_128B)) return DSA_ERR_CUDA;
  CUtensorMap tcd;  // contiguous tiles of c: one 64-column box one key tile high (dense tokens)
  const cuuint32_t cbd[2] = {64, static_cast<cuuint32_t>(mla::NK)};
  if (!make_map(&tcd, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, c, cd, cs, cbd, CU_TENSOR_MAP_SWIZZLE_128B))
    return DSA_ERR_CUDA;
  MlaParams p{};
  p.dense = dense;
  p.pos0 = pos0;
  p.n_keys = n_keys;
  p.page_table = page_table;
  p.pt_stride = pt_stride;
  p.page_rows = page_rows;
  p.kl_lse = kl_lse;
  p.kl_scores = kl_scores;
  p.kl_out = kl_out;
  p.idx = idx;
  p.row_off = row_off;
  p.out = out;
  p.lse = lse;
  p.T = T;
  p.H = H;
  p.k = k;
  p.S = S;
  p.scale_log2 = scale * 1.4426950408889634f;
  // the instantiation with exactly the features this launch uses
  const bool dn = dense != kMlaSparse, pg = page_table != nullptr;
  auto kern = kl_out ? (dn ? sparse_mla_kernel<true, true, false> : sparse_mla_kernel<true, false, false>)
            : pg     ? sparse_mla_kernel<false, true, true>
            : dn     ? sparse_mla_kernel<false, true, false>
                     : sparse_mla_kernel<false, false, false>;
  if (pg && !dn) return DSA_ERR_INVALID_ARG;      // paged caches only come with per-token key counts
  if (set_smem(kern, mla::SMEM) != cudaSuccess) return DSA_ERR_CUDA;
  // KL mode: every CTA takes tokens of its own (the grid still comes in pairs, the kernel's cluster shape)
  const int per_cluster = kl_out ? 2 : 1;
  int clusters = num_sms() / 2;
  if (clusters > (T + per_cluster - 1) / per_cluster) clusters = (T + per_cluster - 1) / per_cluster;
  if (launch_pdl(kern, dim3(2 * clusters), dim3(mla::THREADS), mla::SMEM, st, tq, tc, tcd, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  return last_launch_status();
}

// Causal rows [pos0, pos0 + T) of one sequence (row r at position pos0 + r, its keys from row 0 of c): the rows at
// positions below k (every earlier key selected) run on the dense instantiation, the others on the gathered one.
dsa_status_t run_mla_causal(const uint16_t* q, const uint16_t* c, long long S, const int* idx, int T, int H, int k,
                            float scale, uint16_t* out, float* lse, cudaStream_t st, int pos0,
                            const float* kl_lse = nullptr, const float* kl_scores = nullptr,
                            float* kl_out = nullptr) {
  const int nd = std::max(0, std::min(T, k - pos0));
  dsa_status_t e = DSA_OK;
  if (nd > 0)
    e = run_mla(q, c, S, idx, nullptr, nd, H, k, scale, out, lse, st, kMlaCausal, nullptr, nullptr, 0, 0, pos0,
                kl_lse, kl_scores, kl_out);
  if (e != DSA_OK || nd == T) return e;
  const size_t n = static_cast<size_t>(nd);
  return run_mla(q + n * H * 576, c, S, idx + n * k, nullptr, T - nd, H, k, scale, out ? out + n * H * 512 : nullptr,
                 lse ? lse + n * H : nullptr, st, kMlaSparse, nullptr, nullptr, 0, 0, 0,
                 kl_lse ? kl_lse + n * H : nullptr, kl_scores ? kl_scores + n * k : nullptr,
                 kl_out ? kl_out + n : nullptr);
}

// k: at least 128 and a multiple of 64 (slots of a last, half-filled 128-key tile are masked), at most KMAX
bool mla_k_ok(int k) { return k >= 128 && k % 64 == 0 && k <= mla::KMAX; }

bool indexer_shape_ok(int H_I, int d_I) { return (H_I == 64 && d_I == 128) || (H_I == 4 && d_I == 64); }

size_t prefill_chunk_rows(int L) {
  // rows of scores materialised per chunk: about 1 GiB of fp32 scores, at least 256 rows
  size_t r = (size_t(1) << 30) / (4 * size_t(L > 0 ? L : 1));
  if (r < 256) r = 256;
  if (r > size_t(L)) r = size_t(L);
  return r;
}

int round4(int n) { return (n + 3) & ~3; }

// Scores the varlen select holds at once: at least one sequence's blocked select (the longest), and up to 1 GiB
// for groups of sequences scored together.
size_t varlen_score_floats(int64_t total, int max_len) {
  const size_t one = prefill_chunk_rows(max_len) * size_t(max_len);
  const size_t all = size_t(total) * size_t(round4(max_len));
  const size_t cap = size_t(1) << 28;
  return std::max(one, std::min(all, cap));
}

// Group metadata of the varlen select: runs of query rows, relative sequence starts, score offsets and strides.
size_t varlen_meta_bytes(int nseq) {
  return align_up(size_t(nseq) * sizeof(IndexerSeg), 256) + align_up(size_t(nseq + 1) * 8 + size_t(nseq) * 12, 256);
}

// Steps 1-2 for rows [pos_begin, pos_end) of one causal sequence (row r attends to keys 0..r): q_idx, q_scale, w and
// idx_out point at row pos_begin; k_idx, k_scale hold keys 0..pos_end-1.  Rows t < k form one block whose
// selection needs no scores; later rows go in blocks of chunk_rows, each an indexer launch into `sc` (room for
// chunk_rows x pos_end scores) and a top-k launch.  With sel_scores (pointing at row pos_begin), the index score of
// every selected position is written too, and the indexer then also scores the rows t < k.
dsa_status_t select_rows(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx, const float* k_scale,
                         const float* w, int H_I, int d_I, int k, int pos_begin, int pos_end, int32_t* idx_out,
                         float* sc, size_t chunk_rows, cudaStream_t st, float* sel_scores = nullptr) {
  for (int r0 = pos_begin, rows = 0; r0 < pos_end; r0 += rows) {
    rows = (r0 < k) ? std::min(k, pos_end) - r0 : static_cast<int>(std::min<size_t>(chunk_rows, pos_end - r0));
    const int s_eff = r0 + rows;   // keys beyond the block's last row are never selected (causal)
    const size_t i = static_cast<size_t>(r0 - pos_begin);
    // a block whose every row t has t + 1 <= k selects all of 0..t whatever the scores: no indexer launch (the
    // top-k kernel writes 0..t and the -1 padding of such rows without reading them)
    dsa_status_t e = DSA_OK;
    if (s_eff > k || sel_scores) {
      e = run_indexer_scores(q_idx + i * H_I * d_I, q_scale ? q_scale + i : nullptr, k_idx, k_scale, w + i * H_I,
                             rows, s_eff, H_I, d_I, r0, sc, s_eff, st);
      if (e != DSA_OK) return e;
    }
    e = run_topk(sc, s_eff, nullptr, nullptr, r0, rows, k, idx_out + i * k, k, st,
                 sel_scores ? sel_scores + i * k : nullptr);
    if (e != DSA_OK) return e;
  }
  return DSA_OK;
}

// Rows of the score block of an L-row prefill that starts at row r0: rows t < k form a block of their own, whose
// selection needs no scores; later blocks take prefill_chunk_rows(L) rows (the workspace's capacity at the
// longest key range).  Blocks sized to fill the workspace at every key range (many more rows early on) were
// measured slower for the indexer at 128K (98.2 against 96.0 ms per step) and are not used.
int prefill_block_rows(int L, int k, int r0) {
  if (r0 < 0 || r0 >= L) return 0;
  if (r0 < k) return std::min(k, L) - r0;
  return static_cast<int>(std::min<size_t>(prefill_chunk_rows(L), static_cast<size_t>(L - r0)));
}

// Host checks of a decode step's arguments, shared by both decode entry points (everything but the scratch).
dsa_status_t decode_args_status(int B, const int64_t* cache_off, const int32_t* ctx_len, const uint8_t* q_idx,
                                const float* w, const uint16_t* q, const uint8_t* k_new, const float* k_scale_new,
                                const uint16_t* c_new, const uint8_t* k_cache, const float* k_scale_cache,
                                const uint16_t* c_cache, int64_t cache_rows, int H_I, int d_I, int H, int k,
                                const int32_t* idx_out, const uint16_t* out) {
  if (B <= 0 || cache_rows <= 0 || H <= 0 || k <= 0 || !cache_off || !ctx_len || !q_idx || !w || !q || !k_new ||
      !k_scale_new || !c_new || !k_cache || !k_scale_cache || !c_cache || !out)
    return DSA_ERR_INVALID_ARG;
  if (H_I != 64 || d_I != 128 || H > 128 || !mla_k_ok(k) || B > kMaxDecodeSeqs) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(q) || !aligned16(k_new) || !aligned16(c_new) || !aligned16(k_cache) ||
      !aligned16(c_cache) || !aligned16(out) || (idx_out && !aligned16(idx_out)))
    return DSA_ERR_ALIGNMENT;
  return DSA_OK;
}

size_t decode_ws_bytes(int B, size_t score_cap, int k) {
  return align_up(score_cap * 4, 256) + align_up(size_t(B) * 4, 256) + align_up(size_t(B) * 8, 256) +
         align_up(size_t(B) * k * 4, 256) + align_up(size_t(B) * kTopkBins * 4, 256);
}

// One decode step once the arguments are checked: append -> indexer over each sequence's keys -> top-k -> sparse
// MLA.  Workspace: score rows (packed, 16-byte aligned, score_cap floats), len1 [B], score_off [B], selected
// indices [B, k] (when idx_out is null), each sequence's score histogram [B, 2048] (top 11 order-key bits).
// With fewer sequences than SMs the indexer counts the histogram as it writes the scores, and the cluster top-k
// reads it instead of counting the row again and merging its CTAs' counts.
dsa_status_t run_decode(int B, const DecodeLayout& lay, const int32_t* ctx_len, const uint8_t* q_idx,
                        const float* q_scale, const float* w, const uint16_t* q, const uint8_t* k_new,
                        const float* k_scale_new, const uint16_t* c_new, uint8_t* k_cache, float* k_scale_cache,
                        uint16_t* c_cache, size_t score_cap, int H, int k, float scale, int32_t* idx_out,
                        uint16_t* out, float* lse, void* ws, cudaStream_t st) {
  constexpr int H_I = 64, d_I = 128;
  char* wsb = static_cast<char*>(ws);
  float* dscores = reinterpret_cast<float*>(wsb);
  size_t at = align_up(score_cap * 4, 256);
  int* len1 = reinterpret_cast<int*>(wsb + at);
  at += align_up(size_t(B) * 4, 256);
  long long* soff = reinterpret_cast<long long*>(wsb + at);
  at += align_up(size_t(B) * 8, 256);
  int32_t* idx = idx_out ? idx_out : reinterpret_cast<int32_t*>(wsb + at);
  at += align_up(size_t(B) * k * 4, 256);
  unsigned* hist = (B < num_sms()) ? reinterpret_cast<unsigned*>(wsb + at) : nullptr;
  if (launch_pdl(decode_append_kernel, dim3(B), dim3(kAppendThreads), 0, st, B, lay, ctx_len, k_new, k_scale_new,
                 c_new, k_cache, k_scale_cache, c_cache, d_I, len1, soff, static_cast<long long>(score_cap), hist) !=
      cudaSuccess)
    return DSA_ERR_CUDA;
  dsa_status_t e = last_launch_status();
  if (e != DSA_OK) return e;
  IndexerParams p{};
  p.w = w;
  p.q_scale = q_scale;
  p.k_scale = k_scale_cache;
  p.scores = dscores;
  p.T = B;
  p.cache_off = lay.cache_off;
  p.len1 = len1;
  p.score_off = soff;
  p.page_table = lay.page_table;
  p.max_pages = lay.max_pages;
  p.page_rows = lay.page_rows;
  p.hist = hist;
  using DecCfg = IndexerCfg<H_I, d_I, 1, 1, 2, 4, 1, kModeDecode>;
  e = launch_indexer<H_I, d_I, 1, 1, 2, 4, 1, kModeDecode>(q_idx, B, k_cache, lay.cache_rows, p,
                                                         DecCfg::CTAS_PER_SM * num_sms(), st);
  if (e != DSA_OK) return e;
  e = run_topk(dscores, 0, soff, len1, 0, B, k, idx, k, st, nullptr, hist);
  if (e != DSA_OK) return e;
  return run_mla(q, c_cache, lay.cache_rows, idx, lay.cache_off, B, H, k, scale, out, lse, st, kMlaCounts, len1,
                 lay.page_table, lay.max_pages, lay.page_rows);
}

// ------------------------------------------------------------------------------------------ backward passes
// Hands out 256-byte aligned pieces of a workspace that starts on 16 bytes (null base: only counts).  The 32-byte
// stores of P and dS need more than the 16 bytes a caller's workspace is asked for, so the first piece starts at its
// first 256-byte boundary; bytes() counts the most that skips, whatever the address.
struct Carve {
  char* base;
  size_t at = 0;
  explicit Carve(void* ws)
      : base(reinterpret_cast<char*>(align_up(reinterpret_cast<uintptr_t>(ws), 256))) {}
  size_t bytes() const { return at + 256 - 16; }
  template <typename X>
  X* take(size_t n) {
    X* r = base ? reinterpret_cast<X*>(base + at) : nullptr;
    at += align_up(n * sizeof(X), 256);
    return r;
  }
};

// Tokens that a backward pass handles at once: as many as keep the per-entry buffers (`per_entry` bytes for each of
// kp slots) and the scatter table (2 bytes for each of S rows) of a chunk within 4 GiB, at least 64, and equal chunks.
// The attention's pass over 2048 tokens of k = 2048 took 4910 us with chunks of 512 (2 GiB) and 4722 with 1024.
int bwd_chunk(int T, int64_t S, int kp, size_t per_entry) {
  const size_t each = size_t(kp) * per_entry + 2 * size_t(S);
  const size_t cap = std::min<size_t>(sct::MAX_T, std::max<size_t>(64, (size_t(4) << 30) / each));
  if (size_t(T) <= cap) return T > 0 ? T : 1;
  const size_t chunks = (size_t(T) + cap - 1) / cap;
  return static_cast<int>((size_t(T) + chunks - 1) / chunks);
}

int round_up(int n, int m) { return (n + m - 1) / m * m; }

// Scatter of a chunk's contributions: the table and what goes with it.
struct ScatterWs {
  int* n_end;
  uint16_t *table, *contrib;
  float* acc;
  int ld;
};
ScatterWs carve_scatter(Carve& w, int Tc, int64_t S, int kp, int width, bool many) {
  ScatterWs s{};
  s.ld = round_up(Tc, 8);
  s.n_end = w.take<int>(Tc);
  s.table = w.take<uint16_t>(size_t(S) * s.ld);
  s.contrib = w.take<uint16_t>(size_t(Tc) * kp * width);
  s.acc = many ? w.take<float>(size_t(S) * width) : nullptr;
  return s;
}

// 16-byte pieces of the table, and the blocks that clear them
long long table_pieces(const ScatterWs& w, int64_t S) { return static_cast<long long>(S) * w.ld / 8; }
long long table_blocks(const ScatterWs& w, int64_t S) {
  return std::min<long long>((table_pieces(w, S) + 255) / 256, 8ll * num_sms());
}

dsa_status_t scatter_build(const ScatterWs& w, const int* idx, int T, int64_t S, int k, cudaStream_t st) {
  if (launch_pdl(scatter_build_kernel, dim3(T), dim3(256), 0, st, idx, k, static_cast<long long>(S), w.n_end,
                 w.table, w.ld) != cudaSuccess)
    return DSA_ERR_CUDA;
  return last_launch_status();
}

constexpr long long kShortList = 16;

template <int W>
dsa_status_t scatter_end(const ScatterWs& w, const int* idx, int T, int64_t S, int k, int kp, bool first, bool last,
                         uint16_t* out, cudaStream_t st) {
  const ScatterParams p{w.contrib, w.table, idx, w.ld, k, kp, w.acc, first ? 1 : 0, last ? 1 : 0, out};
  // by the mean length of a row's list (T k / S at most): short ones a warp each
  const bool brief = static_cast<long long>(T) * k < kShortList * static_cast<long long>(S);
  const cudaError_t err =
      brief ? launch_pdl(scatter_sum_short_kernel<W>, dim3(static_cast<unsigned>((S + kSumWarps - 1) / kSumWarps)),
                         dim3(32 * kSumWarps), 0, st, p, static_cast<long long>(S))
            : launch_pdl(scatter_sum_kernel<W>, dim3(static_cast<unsigned>(S)), dim3(ScatterCfg<W>::THREADS), 0, st, p);
  if (err != cudaSuccess) return DSA_ERR_CUDA;
  return last_launch_status();
}

// rank-3 map of [T, H, width] bf16 with boxes of 64 dims x 64 heads
bool make_heads_map(CUtensorMap* m, const uint16_t* base, int T, int H, int width) {
  const cuuint64_t d[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(T)};
  const cuuint64_t s[2] = {static_cast<cuuint64_t>(width) * 2, static_cast<cuuint64_t>(H) * width * 2};
  const cuuint32_t b[3] = {64, 64, 1};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B);
}
// rank-2 map of [rows, width] bf16 with boxes of 64 columns x box_rows
bool make_rows_map(CUtensorMap* m, const uint16_t* base, long long rows, int width, int box_rows) {
  const cuuint64_t d[2] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(rows)};
  const cuuint64_t s[1] = {static_cast<cuuint64_t>(width) * 2};
  const cuuint32_t b[2] = {64, static_cast<cuuint32_t>(box_rows)};
  return make_map(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, d, s, b, CU_TENSOR_MAP_SWIZZLE_128B);
}

// Splits of each of n items' `tiles` tiles over `workers` CTAs (or pairs) that minimise the rounds' length: cost =
// rounds x (tiles of a split + `setup`, what an item costs beside its tiles, in tiles).
int choose_splits(long long n, int workers, int tiles, double setup) {
  int best = 1;
  double best_cost = 1e300;
  for (int s = 1; s <= tiles; ++s) {
    const double cost = static_cast<double>((n * s + workers - 1) / workers) * ((tiles + s - 1) / s + setup);
    if (cost < best_cost - 1e-9) { best_cost = cost; best = s; }
  }
  return best;
}
// The same where the splits' sums have to be joined: only for at most two rounds of items, so that the parts stay
// small.
int choose_joined_splits(long long n, int workers, int tiles, double setup) {
  return n > 2 * workers ? 1 : choose_splits(n, workers, tiles, setup);
}

dsa_status_t join_splits(const float* part, const int* n_end, int keys, int splits, int T, int width, int tail,
                         uint16_t* out, float* out_tail, cudaStream_t st) {
  if (launch_pdl(join_splits_kernel, dim3((width + tail + 1023) / 1024, T), dim3(256), 0, st, part, n_end, keys, splits,
                 width, tail, out, out_tail) != cudaSuccess)
    return DSA_ERR_CUDA;
  return last_launch_status();
}

// Workspace of the attention's backward pass.
struct AttnBwdWs {
  int Tc, HP, kp;
  ScatterWs sc;
  float* delta;
  uint16_t* pds;
  int dq_splits;              // of a chunk of all T tokens (the only chunk where there are few)
  float* dq_part;
  size_t bytes;
};
AttnBwdWs attn_bwd_ws(void* ws, int T, int64_t S, int H, int k) {
  AttnBwdWs a{};
  a.HP = round_up(H, 64);
  a.kp = round_up(k, 128);
  a.Tc = bwd_chunk(T, S, a.kp, mbw::D * 2 + 4 * size_t(a.HP));
  Carve w(ws);
  a.sc = carve_scatter(w, a.Tc, S, a.kp, mbw::D, a.Tc < T);
  a.delta = w.take<float>(size_t(a.Tc) * H);
  a.pds = w.take<uint16_t>(size_t(a.Tc) * a.kp * 2 * a.HP);
  // 3 stages of 64 keys are about what an item's start and end take
  a.dq_splits = a.Tc < T ? 1 : choose_joined_splits(3ll * T, num_sms(), a.kp / mbw::dq::KT, 6.0);
  a.dq_part = a.dq_splits > 1 ? w.take<float>(size_t(T) * a.dq_splits * H * mbw::D) : nullptr;
  a.bytes = w.bytes();
  return a;
}

dsa_status_t run_attn_bwd(const uint16_t* q, const uint16_t* c, int S, const int32_t* idx, const uint16_t* out,
                          const float* lse, const uint16_t* dout, int T, int H, int k, float scale, uint16_t* dq,
                          uint16_t* dc, const AttnBwdWs& w, cudaStream_t st) {
  CUtensorMap tq, tdo, tc, tp128, tp64, tout;
  const size_t rows = size_t(w.Tc) * w.kp;
  if (!make_heads_map(&tq, q, T, H, mbw::D) || !make_heads_map(&tdo, dout, T, H, mbw::DV) ||
      !make_rows_map(&tc, c, S, mbw::D, 1) || !make_rows_map(&tp128, w.pds, rows, 2 * w.HP, 128) ||
      !make_rows_map(&tp64, w.pds, rows, 2 * w.HP, 64) ||
      !make_rows_map(&tout, w.sc.contrib, rows, mbw::D, 32))
    return DSA_ERR_CUDA;
  static std::atomic<unsigned long long> seen[3];
  const int sms = num_sms();
  for (int t0 = 0; t0 < T; t0 += w.Tc) {
    const int n = std::min(w.Tc, T - t0);
    const size_t o = static_cast<size_t>(t0);
    MlaBwdParams p{};
    p.idx = idx + o * k;
    p.n_end = w.sc.n_end;
    p.c = c;
    p.lse = lse + o * H;
    p.delta = w.delta;
    p.pds = w.pds;
    p.dq = dq + o * H * mbw::D;
    p.T = n;
    p.t0 = t0;
    p.H = H;
    p.HP = w.HP;
    p.k = k;
    p.kp = w.kp;
    p.S = S;
    p.scale = scale;
    p.scale_log2 = scale * 1.4426950408889634f;
    const long long dr = static_cast<long long>(n) * H;
    if (launch_pdl(mla_bwd_begin_kernel, dim3(static_cast<unsigned>(std::max((dr + 7) / 8, table_blocks(w.sc, S)))),
                   dim3(256), 0, st, dout + o * H * mbw::DV, out + o * H * mbw::DV, dr, w.delta,
                   reinterpret_cast<uint4*>(w.sc.table), table_pieces(w.sc, S)) != cudaSuccess)
      return DSA_ERR_CUDA;
    dsa_status_t e = last_launch_status();
    if (e != DSA_OK) return e;
    if ((e = scatter_build(w.sc, p.idx, n, S, k, st)) != DSA_OK) return e;
    p.splits = choose_splits(n, sms / 2, (k + 255) / 256, 0.8);
    if (launch_pdl_large(seen[0], mla_bwd_p_kernel<false>, dim3(2 * std::min(sms / 2, n * p.splits)),
                         dim3(mbw::p::THREADS), mbw::p::Map<false>::SMEM, st, tq, tdo, tc, p) != cudaSuccess)
      return DSA_ERR_CUDA;
    if ((e = last_launch_status()) != DSA_OK) return e;
    p.splits = choose_splits(3ll * n, sms / 2, (k + 255) / 256, 1.0);
    if (launch_pdl_large(seen[1], mla_bwd_dc_kernel, dim3(2 * std::min(sms / 2, 3 * n * p.splits)),
                         dim3(mbw::dc::THREADS), mbw::dc::SMEM, st, tp128, tq, tdo, tout, p) != cudaSuccess)
      return DSA_ERR_CUDA;
    if ((e = last_launch_status()) != DSA_OK) return e;
    p.splits = w.dq_splits;
    p.dq_part = w.dq_part;
    if (launch_pdl_large(seen[2], mla_bwd_dq_kernel, dim3(std::min(sms, 3 * n * p.splits)), dim3(mbw::dq::THREADS),
                         mbw::dq::SMEM, st, tp64, p) != cudaSuccess)
      return DSA_ERR_CUDA;
    if ((e = last_launch_status()) != DSA_OK) return e;
    if (p.splits > 1 && (e = join_splits(w.dq_part, w.sc.n_end, mbw::dq::KT, p.splits, n, H * mbw::D, 0, p.dq, nullptr,
                                         st)) != DSA_OK)
      return e;
    e = scatter_end<mbw::D>(w.sc, p.idx, n, S, k, w.kp, t0 == 0, t0 + n >= T, dc, st);
    if (e != DSA_OK) return e;
  }
  return DSA_OK;
}

size_t kl_bwd_ws_bytes(int T) {
  Carve w(nullptr);
  w.take<int>(T);
  return w.bytes();
}

dsa_status_t run_kl_bwd(const uint16_t* q, const uint16_t* c, int S, const int32_t* idx, const float* sel,
                        const float* lse, const float* dkl, int T, int H, int k, float scale, float* dsel, void* ws,
                        cudaStream_t st) {
  CUtensorMap tq, tc;
  if (!make_heads_map(&tq, q, T, H, mbw::D) || !make_rows_map(&tc, c, S, mbw::D, 1)) return DSA_ERR_CUDA;
  Carve w(ws);
  MlaBwdParams p{};
  int* n_end = w.take<int>(T);
  p.idx = idx;
  p.n_end = n_end;
  p.c = c;
  p.lse = lse;
  p.T = T;
  p.H = H;
  p.HP = round_up(H, 64);
  p.k = k;
  p.kp = round_up(k, 128);
  p.S = S;
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.sel = sel;
  p.dkl = dkl;
  p.dsel = dsel;
  if (launch_pdl(scatter_build_kernel, dim3(T), dim3(256), 0, st, idx, k, static_cast<long long>(S), n_end,
                 nullptr, 0) != cudaSuccess)
    return DSA_ERR_CUDA;
  const dsa_status_t e = last_launch_status();
  if (e != DSA_OK) return e;
  static std::atomic<unsigned long long> seen;
  if (launch_pdl_large(seen, mla_bwd_p_kernel<true>, dim3(2 * std::min(num_sms() / 2, T)), dim3(mbw::p::THREADS),
                 mbw::p::Map<true>::SMEM, st, tq, tq, tc, p) != cudaSuccess)
    return DSA_ERR_CUDA;
  return last_launch_status();
}

// Workspace of the index scores' backward pass.
struct IndexBwdWs {
  int Tc, kp, splits;
  ScatterWs sc;
  float* part;
  size_t bytes;
};
IndexBwdWs index_bwd_ws(void* ws, int T, int64_t S, int H_I, int d_I, int k) {
  IndexBwdWs a{};
  a.kp = round_up(k, 128);
  a.Tc = bwd_chunk(T, S, a.kp, size_t(d_I) * 2);
  Carve w(ws);
  a.sc = carve_scatter(w, a.Tc, S, a.kp, d_I, a.Tc < T);
  a.splits = a.Tc < T ? 1 : choose_joined_splits(T, num_sms(), a.kp / ixb::NK, 2.0);
  a.part = a.splits > 1 ? w.take<float>(size_t(T) * a.splits * (size_t(H_I) * d_I + H_I)) : nullptr;
  a.bytes = w.bytes();
  return a;
}

template <int HI, int DI>
dsa_status_t run_index_bwd(IndexerBwdParams p, int T, uint16_t* dk, const IndexBwdWs& w, cudaStream_t st) {
  CUtensorMap tout;
  if (!make_rows_map(&tout, w.sc.contrib, static_cast<long long>(w.Tc) * w.kp, DI, 32)) return DSA_ERR_CUDA;
  static std::atomic<unsigned long long> seen;
  p.n_end = w.sc.n_end;
  p.kp = w.kp;
  p.splits = w.splits;
  p.part = w.part;
  const IndexerBwdParams all = p;
  for (int t0 = 0; t0 < T; t0 += w.Tc) {
    const size_t o = static_cast<size_t>(t0);
    p.T = std::min(w.Tc, T - t0);
    p.q_idx = all.q_idx + o * HI * DI;
    p.q_scale = all.q_scale ? all.q_scale + o : nullptr;
    p.w = all.w + o * HI;
    p.idx = all.idx + o * p.k;
    p.dsel = all.dsel + o * p.k;
    p.dq = all.dq + o * HI * DI;
    p.dw = all.dw + o * HI;
    if (launch_pdl(scatter_clear_kernel, dim3(static_cast<unsigned>(table_blocks(w.sc, p.S))), dim3(256), 0, st,
                   reinterpret_cast<uint4*>(w.sc.table), table_pieces(w.sc, p.S)) != cudaSuccess)
      return DSA_ERR_CUDA;
    dsa_status_t e = last_launch_status();
    if (e != DSA_OK) return e;
    if ((e = scatter_build(w.sc, p.idx, p.T, p.S, p.k, st)) != DSA_OK) return e;
    if (launch_pdl_large(seen, indexer_bwd_kernel<HI, DI>, dim3(std::min(num_sms(), p.T * p.splits)),
                         dim3(ixb::THREADS), ixb::SMEM, st, tout, p) != cudaSuccess)
      return DSA_ERR_CUDA;
    if ((e = last_launch_status()) != DSA_OK) return e;
    if (p.splits > 1 &&
        (e = join_splits(w.part, w.sc.n_end, ixb::NK, p.splits, p.T, HI * DI, HI, p.dq, p.dw, st)) != DSA_OK)
      return e;
    e = scatter_end<DI>(w.sc, p.idx, p.T, p.S, p.k, w.kp, t0 == 0, t0 + p.T >= T, dk, st);
    if (e != DSA_OK) return e;
  }
  return DSA_OK;
}

// ------------------------------------------------------------------------------------------ rotary positions
template <typename E>
dsa_status_t launch_rope(RopeParams p, bool vec, bool inter, cudaStream_t st) {
  constexpr int V = 16 / sizeof(E);
  const int n = vec ? V : 1;
  const bool in_place = p.x == p.out;
  p.rot_units = vec && inter ? p.R / V : p.R / 2 / n;
  p.copy_units = in_place ? 0 : (p.D - p.R) / n;
  // one head a thread until the GPU's resident threads are covered, then up to eight (their loads in flight together,
  // one set of angles); more tokens than that go round the same threads, in equal shares
  const long long one = static_cast<long long>(p.T) * (p.rot_units + p.copy_units) * p.H, resident = 2048ll * num_sms();
  p.heads_per = static_cast<int>(std::min<long long>(std::min(8, p.H), std::max<long long>(1, one / resident)));
  if (p.H > 65535 * p.heads_per) p.heads_per = 8;       // blockIdx.y counts the groups
  const int groups = (p.H + p.heads_per - 1) / p.heads_per;
  const int bx = std::min(256, p.rot_units), by = 256 / bx;
  const long long blocks = (static_cast<long long>(p.T) + by - 1) / by;
  const long long most = std::max<long long>(1, 2 * resident / 256 / groups);
  const long long rounds = (blocks + most - 1) / most, gx = (blocks + rounds - 1) / rounds;
  auto kern = !vec             ? (inter ? rope_kernel<E, 1, true, 1> : rope_kernel<E, 1, false, 1>)
            : p.heads_per == 1 ? (inter ? rope_kernel<E, V, true, 1> : rope_kernel<E, V, false, 1>)
                               : (inter ? rope_kernel<E, V, true, 4> : rope_kernel<E, V, false, 4>);
  if (launch_pdl(kern, dim3(static_cast<unsigned>(gx), groups, p.copy_units ? 2 : 1), dim3(bx, by), 0, st, p) !=
      cudaSuccess)
    return DSA_ERR_CUDA;
  return last_launch_status();
}

// Elements [0, D) of each of T x H rows at the given strides do not meet each other.
bool rope_rows_apart(int T, int H, int D, int64_t st, int64_t sh) {
  if (H == 1) return T == 1 || st >= D;
  if (T == 1) return sh >= D;
  return (sh >= D && st >= (H - 1) * sh + D) || (st >= D && sh >= (T - 1) * st + D);
}

// T x H rows of D elements at these strides, which lie apart (rope_rows_apart), meet the same rows moved by `delta`.
// The larger stride is longer than all rows along the smaller one together, so that only the two multiples of it next
// to delta can leave a difference that those bridge, and for each of them two multiples of the smaller.
bool rope_moved_rows_meet(int64_t delta, int T, int H, int D, int64_t st, int64_t sh) {
  const bool heads_inside = st >= sh;
  const int64_t so = heads_inside ? st : sh, si = heads_inside ? sh : st;
  const int64_t no = heads_inside ? T : H, ni = heads_inside ? H : T;
  auto floor_div = [](int64_t a, int64_t b) { return b ? a / b - (a % b < 0 ? 1 : 0) : 0; };
  for (int64_t q = floor_div(delta, so), q1 = q + 1; q <= q1; ++q) {
    if (q <= -no || q >= no) continue;
    const int64_t r = delta - q * so;
    for (int64_t p = floor_div(r, si), p1 = p + 1; p <= p1; ++p)
      if (p > -ni && p < ni && std::abs(r - p * si) < D) return true;
  }
  return false;
}

dsa_status_t run_rope(const void* x, int64_t x_st, int64_t x_sh, void* out, int64_t o_st, int64_t o_sh,
                      const int32_t* positions, int pos0, const double* inv_freq, int T, int H, int D, int rot_off,
                      int rot_dim, int interleaved, float mscale, int dtype, bool backward, void* stream) {
  if (T < 0 || H <= 0 || D <= 0 || rot_dim <= 0 || rot_dim % 2 || rot_off < 0 || rot_off > D - rot_dim ||
      (T > 0 && (!x || !out || !inv_freq)) || x_st < 0 || x_sh < 0 || (dtype != DSA_BF16 && dtype != DSA_FP32))
    return DSA_ERR_INVALID_ARG;
  if (T == 0) return DSA_OK;
  if (T > (1 << 30) || H > (1 << 18)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!positions && pos0 > INT32_MAX - (T - 1)) return DSA_ERR_INVALID_ARG;
  const int es = dtype == DSA_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(x) % es || reinterpret_cast<uintptr_t>(out) % es ||
      reinterpret_cast<uintptr_t>(inv_freq) % 8 || reinterpret_cast<uintptr_t>(positions) % 4)
    return DSA_ERR_ALIGNMENT;
  // a single token's or head's stride does not matter
  if (T == 1) x_st = o_st = 0;
  if (H == 1) x_sh = o_sh = 0;
  if (!rope_rows_apart(T, H, D, o_st, o_sh)) return DSA_ERR_INVALID_ARG;
  // the result replaces its input exactly, or shares no element with it: apart in memory, or (equal strides) lying
  // between the other's rows
  if (x == out) {
    if (x_st != o_st || x_sh != o_sh) return DSA_ERR_INVALID_ARG;
  } else {
    const char *xb = static_cast<const char*>(x), *ob = static_cast<const char*>(out);
    const int64_t xe = ((T - 1) * x_st + (H - 1) * x_sh + D) * es, oe = ((T - 1) * o_st + (H - 1) * o_sh + D) * es;
    if (xb < ob + oe && ob < xb + xe &&
        (x_st != o_st || x_sh != o_sh || rope_moved_rows_meet((ob - xb) / es, T, H, D, o_st, o_sh)))
      return DSA_ERR_INVALID_ARG;
  }
  RopeParams p{};
  p.x = x;
  p.out = out;
  p.x_st = x_st;
  p.x_sh = x_sh;
  p.o_st = o_st;
  p.o_sh = o_sh;
  p.positions = positions;
  p.freq = inv_freq;
  p.pos0 = pos0;
  p.T = T;
  p.H = H;
  p.D = D;
  p.off = rot_off;
  p.R = rot_dim;
  p.m = mscale;
  p.backward = backward ? 1 : 0;
  // 16-byte pieces where every row, the rotated part and its halves start on them
  const int64_t v = 16 / es;
  const bool vec = aligned16(x) && aligned16(out) && x_st % v == 0 && x_sh % v == 0 && o_st % v == 0 &&
                   o_sh % v == 0 && D % v == 0 && rot_off % v == 0 && (interleaved ? rot_dim : rot_dim / 2) % v == 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  return dtype == DSA_BF16 ? launch_rope<__nv_bfloat16>(p, vec, interleaved != 0, st)
                           : launch_rope<float>(p, vec, interleaved != 0, st);
}

}  // namespace
}  // namespace dsa

using namespace dsa;

extern "C" {

const char* dsa_status_string(dsa_status_t s) {
  switch (s) {
    case DSA_OK: return "DSA_OK";
    case DSA_ERR_INVALID_ARG: return "DSA_ERR_INVALID_ARG";
    case DSA_ERR_UNSUPPORTED_SHAPE: return "DSA_ERR_UNSUPPORTED_SHAPE";
    case DSA_ERR_ALIGNMENT: return "DSA_ERR_ALIGNMENT";
    case DSA_ERR_CUDA: return "DSA_ERR_CUDA";
    case DSA_ERR_TIMEOUT: return "DSA_ERR_TIMEOUT";
    case DSA_ERR_BAD_INDEX: return "DSA_ERR_BAD_INDEX";
    case DSA_ERR_WORKSPACE: return "DSA_ERR_WORKSPACE";
    case DSA_ERR_CHECK: return "DSA_ERR_CHECK";
  }
  return "DSA_UNKNOWN_STATUS";
}

dsa_status_t dsa_get_device_status(void* stream, int* device_status) {
  if (!device_status) return DSA_ERR_INVALID_ARG;
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return DSA_ERR_CUDA;
  int v = 0;
  if (cudaMemcpyFromSymbol(&v, g_dev_status, sizeof(int)) != cudaSuccess) return DSA_ERR_CUDA;
  const int zero = 0;
  if (cudaMemcpyToSymbol(g_dev_status, &zero, sizeof(int)) != cudaSuccess) return DSA_ERR_CUDA;
  *device_status = v;
  return DSA_OK;
}

int dsa_num_sms(void) { return num_sms(); }

int dsa_checks_enabled(void) { return kChecks ? 1 : 0; }

dsa_status_t dsa_indexer_scores(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                const float* k_scale, const float* w, int T, int S, int H_I, int d_I, int pos0,
                                float* scores, void* stream) {
  if (T < 0 || S < 0 || pos0 < 0 || (T > 0 && (!q_idx || !w || !scores)) || (S > 0 && !k_idx))
    return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(k_idx)) return DSA_ERR_ALIGNMENT;
  if (T == 0 || S == 0) return DSA_OK;
  return run_indexer_scores(q_idx, q_scale, k_idx, k_scale, w, T, S, H_I, d_I, pos0, scores, S,
                            static_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_topk(const float* scores, int rows, int64_t ld, const int32_t* row_len, int pos0, int k,
                      int32_t* idx, void* stream) {
  if (rows < 0 || ld < 0 || k <= 0 || pos0 < 0 || (rows > 0 && (!scores || !idx))) return DSA_ERR_INVALID_ARG;
  return run_topk(scores, ld, nullptr, row_len, pos0, rows, k, idx, k, static_cast<cudaStream_t>(stream));
}

dsa_status_t dsa_indexer_kl(const uint16_t* q, const uint16_t* c, int S, const int32_t* idx, const float* sel_scores,
                            const float* lse, int T, int H, int k, float scale, float* kl, void* stream) {
  if (T < 0 || S <= 0 || H <= 0 || k <= 0 || (T > 0 && (!q || !c || !idx || !sel_scores || !lse || !kl)))
    return DSA_ERR_INVALID_ARG;
  if (H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q) || !aligned16(c) || !aligned16(idx)) return DSA_ERR_ALIGNMENT;
  return run_mla(q, c, S, idx, nullptr, T, H, k, scale, nullptr, nullptr, static_cast<cudaStream_t>(stream),
                 kMlaSparse, nullptr, nullptr, 0, 0, 0, lse, sel_scores, kl);
}

size_t dsa_prefill_kl_workspace_size(int L, int H_I, int d_I, int H, int k) {
  if (L <= 0 || k <= 0 || H <= 0) return 0;
  return dsa_prefill_workspace_size(L, H_I, d_I, H, k) + align_up(size_t(L) * size_t(k) * 4, 256) +
         align_up(size_t(L) * size_t(H) * 4, 256);
}

dsa_status_t dsa_forward_prefill_kl(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                    const float* k_scale, const float* w, const uint16_t* q, const uint16_t* c,
                                    int L, int H_I, int d_I, int H, int k, float scale, int32_t* idx_out,
                                    uint16_t* out, float* lse, float* kl, void* ws, size_t ws_bytes, void* stream) {
  if (L <= 0 || H <= 0 || k <= 0 || !q_idx || !k_idx || !w || !q || !c || !out || !kl) return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I) || H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(q) || !aligned16(c) || !aligned16(out) ||
      (idx_out && !aligned16(idx_out)))
    return DSA_ERR_ALIGNMENT;
  if (!ws || ws_bytes < dsa_prefill_kl_workspace_size(L, H_I, d_I, H, k)) return DSA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // workspace: the prefill's (score block, selected indices), then the selected index scores [L, k] and lse [L, H]
  char* wsb = static_cast<char*>(ws);
  const size_t score_bytes = align_up(prefill_chunk_rows(L) * size_t(L) * 4, 256);
  int32_t* idx = idx_out ? idx_out : reinterpret_cast<int32_t*>(wsb + score_bytes);
  size_t at = dsa_prefill_workspace_size(L, H_I, d_I, H, k);
  float* sel = reinterpret_cast<float*>(wsb + at);
  at += align_up(size_t(L) * size_t(k) * 4, 256);
  float* lse_buf = lse ? lse : reinterpret_cast<float*>(wsb + at);
  dsa_status_t e = select_rows(q_idx, q_scale, k_idx, k_scale, w, H_I, d_I, k, 0, L, idx, reinterpret_cast<float*>(wsb),
                               prefill_chunk_rows(L), st, sel);
  if (e != DSA_OK) return e;
  e = run_mla_causal(q, c, L, idx, L, H, k, scale, out, lse_buf, st, 0);
  if (e != DSA_OK) return e;
  return run_mla_causal(q, c, L, idx, L, H, k, scale, nullptr, nullptr, st, 0, lse_buf, sel, kl);
}

dsa_status_t dsa_sparse_mla_attn(const uint16_t* q, const uint16_t* c, int S, const int32_t* idx, int T, int H,
                                 int k, float scale, uint16_t* out, float* lse, void* stream) {
  if (T < 0 || S <= 0 || H <= 0 || k <= 0 || (T > 0 && (!q || !c || !idx || !out))) return DSA_ERR_INVALID_ARG;
  if (H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q) || !aligned16(c) || !aligned16(idx) || !aligned16(out)) return DSA_ERR_ALIGNMENT;
  return run_mla(q, c, S, idx, nullptr, T, H, k, scale, out, lse, static_cast<cudaStream_t>(stream));
}

size_t dsa_prefill_workspace_size(int L, int H_I, int d_I, int H, int k) {
  (void)H_I; (void)d_I; (void)H;
  if (L <= 0 || k <= 0) return 0;
  const size_t rows = prefill_chunk_rows(L);
  return align_up(rows * size_t(L) * 4, 256) + align_up(size_t(L) * size_t(k) * 4, 256);
}

dsa_status_t dsa_prefill_select(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                const float* k_scale, const float* w, int L, int H_I, int d_I, int k,
                                int32_t* idx_out, void* ws, size_t ws_bytes, void* stream) {
  if (L <= 0 || k <= 0 || !q_idx || !k_idx || !w || !idx_out) return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(k_idx)) return DSA_ERR_ALIGNMENT;
  if (!ws || ws_bytes < align_up(prefill_chunk_rows(L) * size_t(L) * 4, 256)) return DSA_ERR_WORKSPACE;
  return select_rows(q_idx, q_scale, k_idx, k_scale, w, H_I, d_I, k, 0, L, idx_out, static_cast<float*>(ws),
                     prefill_chunk_rows(L), static_cast<cudaStream_t>(stream));
}

size_t dsa_prefill_rows_workspace_size(int row0, int nrows, int H_I, int d_I, int H, int k) {
  (void)H_I; (void)d_I; (void)H;
  if (row0 < 0 || nrows <= 0 || k <= 0) return 0;
  const int S = row0 + nrows;
  return align_up(prefill_chunk_rows(S) * size_t(S) * 4, 256) + align_up(size_t(nrows) * size_t(k) * 4, 256);
}

dsa_status_t dsa_forward_prefill_rows(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                      const float* k_scale, const float* w, const uint16_t* q, const uint16_t* c,
                                      int row0, int nrows, int H_I, int d_I, int H, int k, float scale,
                                      int32_t* idx_out, uint16_t* out, float* lse, void* ws, size_t ws_bytes,
                                      void* stream) {
  if (row0 < 0 || nrows <= 0 || H <= 0 || k <= 0 || !q_idx || !k_idx || !w || !q || !c || !out)
    return DSA_ERR_INVALID_ARG;
  if (static_cast<long long>(row0) + nrows > INT32_MAX) return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I) || H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(q) || !aligned16(c) || !aligned16(out) ||
      (idx_out && !aligned16(idx_out)))
    return DSA_ERR_ALIGNMENT;
  if (!ws || ws_bytes < dsa_prefill_rows_workspace_size(row0, nrows, H_I, d_I, H, k)) return DSA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int S = row0 + nrows;
  const size_t score_bytes = align_up(prefill_chunk_rows(S) * size_t(S) * 4, 256);
  int32_t* idx = idx_out ? idx_out : reinterpret_cast<int32_t*>(static_cast<char*>(ws) + score_bytes);
  dsa_status_t e = select_rows(q_idx, q_scale, k_idx, k_scale, w, H_I, d_I, k, row0, S, idx, static_cast<float*>(ws),
                               prefill_chunk_rows(S), st);
  if (e != DSA_OK) return e;
  return run_mla_causal(q, c, S, idx, nrows, H, k, scale, out, lse, st, row0);
}

dsa_status_t dsa_forward_prefill(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                 const float* k_scale, const float* w, const uint16_t* q, const uint16_t* c,
                                 int L, int H_I, int d_I, int H, int k, float scale, int32_t* idx_out,
                                 uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (L <= 0 || H <= 0 || k <= 0 || !q_idx || !k_idx || !w || !q || !c || !out) return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I) || H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(q) || !aligned16(c) || !aligned16(out) ||
      (idx_out && !aligned16(idx_out)))
    return DSA_ERR_ALIGNMENT;
  if (!ws || ws_bytes < dsa_prefill_workspace_size(L, H_I, d_I, H, k)) return DSA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  int32_t* idx = idx_out ? idx_out
                         : reinterpret_cast<int32_t*>(static_cast<char*>(ws) +
                                                      align_up(prefill_chunk_rows(L) * size_t(L) * 4, 256));
  dsa_status_t e = dsa_prefill_select(q_idx, q_scale, k_idx, k_scale, w, L, H_I, d_I, k, idx, ws, ws_bytes, stream);
  if (e != DSA_OK) return e;
  return run_mla_causal(q, c, L, idx, L, H, k, scale, out, lse, st, 0);
}

// ------------------------------------------------------------------------------------------ host-buffer prefill
namespace {
constexpr int kHostChunks = 16;         // token chunks of the host-buffer prefill's pipeline

// The host-buffer prefill's device copies, laid out after the prefill workspace.
struct HostPrefillLayout {
  size_t ws, q_idx, q_scale, k_idx, k_scale, w, q, c, out, lse, total;
};
HostPrefillLayout host_prefill_layout(int L, int H_I, int d_I, int H, int k) {
  HostPrefillLayout lo{};
  size_t at = dsa_prefill_workspace_size(L, H_I, d_I, H, k);
  auto take = [&](size_t bytes) { const size_t o = at; at += align_up(bytes, 256); return o; };
  lo.ws = 0;
  lo.q_idx = take(size_t(L) * H_I * d_I);
  lo.q_scale = take(size_t(L) * 4);
  lo.k_idx = take(size_t(L) * d_I);
  lo.k_scale = take(size_t(L) * 4);
  lo.w = take(size_t(L) * H_I * 4);
  lo.q = take(size_t(L) * H * 576 * 2);
  lo.c = take(size_t(L) * 576 * 2);
  lo.out = take(size_t(L) * H * 512 * 2);
  lo.lse = take(size_t(L) * H * 4);
  lo.total = at;
  return lo;
}

// One copy stream per direction and device, created on first use (the call allocates no memory).
struct CopyStreams {
  cudaStream_t h2d = nullptr, d2h = nullptr;
};
CopyStreams g_copy_streams[64];
std::mutex g_copy_mutex;

dsa_status_t copy_streams(CopyStreams* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return DSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_copy_mutex);
  CopyStreams& cs = g_copy_streams[dev];
  if (!cs.h2d && cudaStreamCreateWithFlags(&cs.h2d, cudaStreamNonBlocking) != cudaSuccess) return DSA_ERR_CUDA;
  if (!cs.d2h && cudaStreamCreateWithFlags(&cs.d2h, cudaStreamNonBlocking) != cudaSuccess) return DSA_ERR_CUDA;
  *out = cs;
  return DSA_OK;
}
}  // namespace

size_t dsa_prefill_host_workspace_size(int L, int H_I, int d_I, int H, int k) {
  if (L <= 0 || k <= 0 || H <= 0 || !indexer_shape_ok(H_I, d_I)) return 0;
  return host_prefill_layout(L, H_I, d_I, H, k).total;
}

dsa_status_t dsa_forward_prefill_host(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                      const float* k_scale, const float* w, const uint16_t* q, const uint16_t* c,
                                      int L, int H_I, int d_I, int H, int k, float scale, int32_t* idx_out,
                                      uint16_t* out, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (L <= 0 || H <= 0 || k <= 0 || !q_idx || !k_idx || !w || !q || !c || !out) return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I) || H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!ws || ws_bytes < dsa_prefill_host_workspace_size(L, H_I, d_I, H, k)) return DSA_ERR_WORKSPACE;
  CopyStreams cs;
  dsa_status_t e = copy_streams(&cs);
  if (e != DSA_OK) return e;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const HostPrefillLayout lo = host_prefill_layout(L, H_I, d_I, H, k);
  char* d = static_cast<char*>(ws);
  uint8_t* dq_idx = reinterpret_cast<uint8_t*>(d + lo.q_idx);
  float* dq_scale = q_scale ? reinterpret_cast<float*>(d + lo.q_scale) : nullptr;
  uint8_t* dk_idx = reinterpret_cast<uint8_t*>(d + lo.k_idx);
  float* dk_scale = k_scale ? reinterpret_cast<float*>(d + lo.k_scale) : nullptr;
  float* dw = reinterpret_cast<float*>(d + lo.w);
  uint16_t* dq = reinterpret_cast<uint16_t*>(d + lo.q);
  uint16_t* dc = reinterpret_cast<uint16_t*>(d + lo.c);
  uint16_t* dout = reinterpret_cast<uint16_t*>(d + lo.out);
  float* dlse = reinterpret_cast<float*>(d + lo.lse);
  float* sc = reinterpret_cast<float*>(d);
  int32_t* didx = reinterpret_cast<int32_t*>(d + align_up(prefill_chunk_rows(L) * size_t(L) * 4, 256));
  // events: start, indexer inputs landed, per chunk its queries landed and its attention done, all copies back
  constexpr int NE = 2 + 2 * kHostChunks + 1;
  cudaEvent_t ev[NE] = {};
  for (int i = 0; i < NE; ++i)
    if (cudaEventCreateWithFlags(&ev[i], cudaEventDisableTiming) != cudaSuccess) {
      for (int j = 0; j < i; ++j) cudaEventDestroy(ev[j]);
      return DSA_ERR_CUDA;
    }
  cudaEvent_t& ev_start = ev[0];
  cudaEvent_t& ev_inputs = ev[1];
  cudaEvent_t* ev_q = ev + 2;
  cudaEvent_t* ev_att = ev + 2 + kHostChunks;
  cudaEvent_t& ev_done = ev[NE - 1];
  auto h2d = [&](void* dst, const void* src, size_t bytes) {
    return !src || cudaMemcpyAsync(dst, src, bytes, cudaMemcpyHostToDevice, cs.h2d) == cudaSuccess;
  };
  auto d2h = [&](void* dst, const void* src, size_t bytes) {
    return !dst || cudaMemcpyAsync(dst, src, bytes, cudaMemcpyDeviceToHost, cs.d2h) == cudaSuccess;
  };
  const size_t qrow = size_t(H) * 576 * 2, orow = size_t(H) * 512 * 2;
  bool ok = cudaEventRecord(ev_start, st) == cudaSuccess && cudaStreamWaitEvent(cs.h2d, ev_start, 0) == cudaSuccess &&
            cudaStreamWaitEvent(cs.d2h, ev_start, 0) == cudaSuccess;
  // host -> device: the indexer's inputs first, then c and the queries chunk by chunk
  ok = ok && h2d(dk_idx, k_idx, size_t(L) * d_I) && h2d(dk_scale, k_scale, size_t(L) * 4) &&
       h2d(dq_idx, q_idx, size_t(L) * H_I * d_I) && h2d(dq_scale, q_scale, size_t(L) * 4) &&
       h2d(dw, w, size_t(L) * H_I * 4) && cudaEventRecord(ev_inputs, cs.h2d) == cudaSuccess &&
       h2d(dc, c, size_t(L) * 576 * 2);
  int t0[kHostChunks + 1];
  for (int j = 0; j <= kHostChunks; ++j) t0[j] = static_cast<int>((static_cast<long long>(L) * j) / kHostChunks);
  for (int j = 0; j < kHostChunks && ok; ++j) {
    ok = h2d(reinterpret_cast<char*>(dq) + t0[j] * qrow, reinterpret_cast<const char*>(q) + t0[j] * qrow,
             size_t(t0[j + 1] - t0[j]) * qrow) &&
         cudaEventRecord(ev_q[j], cs.h2d) == cudaSuccess;
  }
  // compute, chunk by chunk: the chunk's rows' selection, then (once its queries landed) its attention
  ok = ok && cudaStreamWaitEvent(st, ev_inputs, 0) == cudaSuccess;
  for (int j = 0; j < kHostChunks && ok && e == DSA_OK; ++j) {
    const int n = t0[j + 1] - t0[j];
    if (n == 0) {
      ok = cudaEventRecord(ev_att[j], st) == cudaSuccess;
      continue;
    }
    e = select_rows(dq_idx + size_t(t0[j]) * H_I * d_I, dq_scale ? dq_scale + t0[j] : nullptr, dk_idx, dk_scale,
                    dw + size_t(t0[j]) * H_I, H_I, d_I, k, t0[j], t0[j + 1], didx + size_t(t0[j]) * k, sc,
                    prefill_chunk_rows(L), st);
    if (e != DSA_OK) break;
    ok = cudaStreamWaitEvent(st, ev_q[j], 0) == cudaSuccess;
    if (!ok) break;
    e = run_mla_causal(reinterpret_cast<const uint16_t*>(reinterpret_cast<const char*>(dq) + t0[j] * qrow), dc, L,
                       didx + size_t(t0[j]) * k, n, H, k, scale,
                       reinterpret_cast<uint16_t*>(reinterpret_cast<char*>(dout) + t0[j] * orow),
                       dlse + size_t(t0[j]) * H, st, t0[j]);
    if (e != DSA_OK) break;
    ok = cudaEventRecord(ev_att[j], st) == cudaSuccess;
    // device -> host of the chunk's results, on the other copy stream
    ok = ok && cudaStreamWaitEvent(cs.d2h, ev_att[j], 0) == cudaSuccess &&
         d2h(reinterpret_cast<char*>(out) + t0[j] * orow, reinterpret_cast<char*>(dout) + t0[j] * orow,
             size_t(n) * orow) &&
         d2h(lse ? lse + size_t(t0[j]) * H : nullptr, dlse + size_t(t0[j]) * H, size_t(n) * H * 4) &&
         d2h(idx_out ? idx_out + size_t(t0[j]) * k : nullptr, didx + size_t(t0[j]) * k, size_t(n) * k * 4);
  }
  // the caller's stream ends when every copy back has landed
  ok = ok && cudaEventRecord(ev_done, cs.d2h) == cudaSuccess && cudaStreamWaitEvent(st, ev_done, 0) == cudaSuccess;
  for (int i = 0; i < NE; ++i) cudaEventDestroy(ev[i]);     // released once the work that uses them completes
  if (e != DSA_OK) return e;
  return ok ? DSA_OK : DSA_ERR_CUDA;
}

size_t dsa_prefill_varlen_workspace_size(int nseq, int64_t total, int max_len, int H_I, int d_I, int H, int k) {
  (void)H_I; (void)d_I; (void)H;
  if (nseq <= 0 || total <= 0 || max_len <= 0 || k <= 0) return 0;
  return align_up(varlen_score_floats(total, max_len) * 4, 256) + align_up(size_t(total) * 8, 256) +
         align_up(size_t(nseq + 1) * 8, 256) + align_up(size_t(total) * size_t(k) * 4, 256) +
         align_up(size_t(total) * 8, 256) + align_up(size_t(total) * 4, 256) + varlen_meta_bytes(nseq);
}

dsa_status_t dsa_forward_prefill_varlen(int nseq, const int64_t* cu_seqlens, const uint8_t* q_idx,
                                        const float* q_scale, const uint8_t* k_idx, const float* k_scale,
                                        const float* w, const uint16_t* q, const uint16_t* c, int H_I, int d_I,
                                        int H, int k, float scale, int32_t* idx_out, uint16_t* out, float* lse,
                                        void* ws, size_t ws_bytes, void* stream) {
  if (nseq <= 0 || !cu_seqlens || H <= 0 || k <= 0 || !q_idx || !k_idx || !w || !q || !c || !out)
    return DSA_ERR_INVALID_ARG;
  if (cu_seqlens[0] != 0) return DSA_ERR_INVALID_ARG;
  int max_len = 0;
  for (int b = 0; b < nseq; ++b) {
    const int64_t len = cu_seqlens[b + 1] - cu_seqlens[b];
    if (len < 0 || cu_seqlens[b + 1] > INT32_MAX) return DSA_ERR_INVALID_ARG;
    if (len > max_len) max_len = static_cast<int>(len);
  }
  const int64_t total = cu_seqlens[nseq];
  if (total <= 0) return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I) || H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(q) || !aligned16(c) || !aligned16(out) ||
      (idx_out && !aligned16(idx_out)))
    return DSA_ERR_ALIGNMENT;
  if (!ws || ws_bytes < dsa_prefill_varlen_workspace_size(nseq, total, max_len, H_I, d_I, H, k))
    return DSA_ERR_WORKSPACE;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  // workspace: scores, per-token row offsets (attention), cu_seqlens, indices, per-row score offsets and lengths
  // (top-k), then the metadata of a group of sequences (runs of query rows, relative starts, score offsets, strides)
  char* wsb = static_cast<char*>(ws);
  const size_t budget = varlen_score_floats(total, max_len);
  float* sc = reinterpret_cast<float*>(wsb);
  size_t at = align_up(budget * 4, 256);
  long long* row_off = reinterpret_cast<long long*>(wsb + at);
  at += align_up(size_t(total) * 8, 256);
  long long* cu_dev = reinterpret_cast<long long*>(wsb + at);
  at += align_up(size_t(nseq + 1) * 8, 256);
  int32_t* idx = idx_out ? idx_out : reinterpret_cast<int32_t*>(wsb + at);
  at += align_up(size_t(total) * size_t(k) * 4, 256);
  long long* tk_off = reinterpret_cast<long long*>(wsb + at);
  at += align_up(size_t(total) * 8, 256);
  int* tk_len = reinterpret_cast<int*>(wsb + at);
  at += align_up(size_t(total) * 4, 256);
  char* meta = wsb + at;
  IndexerSeg* segs_dev = reinterpret_cast<IndexerSeg*>(meta);
  long long* gcu_dev = reinterpret_cast<long long*>(meta + align_up(size_t(nseq) * sizeof(IndexerSeg), 256));
  long long* soff_dev = gcu_dev + (nseq + 1);
  int* sld_dev = reinterpret_cast<int*>(soff_dev + nseq);
  if (cudaMemcpyAsync(cu_dev, cu_seqlens, size_t(nseq + 1) * 8, cudaMemcpyHostToDevice, st) != cudaSuccess)
    return DSA_ERR_CUDA;
  varlen_row_off_kernel<<<static_cast<unsigned>((total + 255) / 256), 256, 0, st>>>(cu_dev, nseq, total, row_off);
  dsa_status_t e = last_launch_status();
  if (e != DSA_OK) return e;
  // Steps 1-2.  Consecutive sequences are grouped while their scored rows (t >= k) fit the score buffer; a group
  // is one indexer launch over all of its sequences' scored rows and one top-k launch over all of its rows.  A
  // sequence whose scores alone exceed the buffer takes the blocked select of dsa_prefill_select.
  std::vector<IndexerSeg> segs;
  std::vector<long long> gcu, soff;
  std::vector<int> sld;
  const int tok = (H_I == 64) ? 16 : 256;
  for (int b = 0; b < nseq;) {
    const int64_t r0 = cu_seqlens[b];
    const int len = static_cast<int>(cu_seqlens[b + 1] - r0);
    const size_t need = (len > k) ? size_t(len - k) * size_t(round4(len)) : 0;
    if (need > budget) {
      e = select_rows(q_idx + r0 * H_I * d_I, q_scale ? q_scale + r0 : nullptr, k_idx + r0 * d_I,
                      k_scale ? k_scale + r0 : nullptr, w + r0 * H_I, H_I, d_I, k, 0, len, idx + r0 * k, sc,
                      prefill_chunk_rows(len), st);
      if (e != DSA_OK) return e;
      ++b;
      continue;
    }
    const int b0 = b;
    size_t used = 0;
    segs.clear();
    gcu.assign(1, 0);
    soff.clear();
    sld.clear();
    while (b < nseq && segs.size() < static_cast<size_t>(kMaxDecodeSeqs)) {
      const int64_t rb = cu_seqlens[b];
      const int lb = static_cast<int>(cu_seqlens[b + 1] - rb);
      const size_t nb = (lb > k) ? size_t(lb - k) * size_t(round4(lb)) : 0;
      if (used + nb > budget) break;
      if (nb) {
        IndexerSeg sg{};
        sg.q_row0 = rb + k;
        sg.key_row0 = rb;
        sg.out_base = static_cast<long long>(used);
        sg.pos0 = k;
        sg.n_rows = lb - k;
        sg.S = lb;
        sg.ld = round4(lb);
        segs.push_back(sg);
      }
      soff.push_back(static_cast<long long>(used));
      sld.push_back(round4(lb));
      used += nb;
      gcu.push_back(cu_seqlens[b + 1] - cu_seqlens[b0]);
      ++b;
    }
    const int ng = b - b0;
    int split = 1, n_items = 0;
    if (!segs.empty()) {
      plan_segments(segs.data(), static_cast<int>(segs.size()), tok, &split, &n_items);
      if (cudaMemcpyAsync(segs_dev, segs.data(), segs.size() * sizeof(IndexerSeg), cudaMemcpyHostToDevice, st) !=
          cudaSuccess)
        return DSA_ERR_CUDA;
      e = run_indexer_segments(q_idx, total, q_scale, k_idx, total, k_scale, w, H_I, d_I, segs_dev,
                               static_cast<int>(segs.size()), split, n_items, sc, st);
      if (e != DSA_OK) return e;
    }
    if (cudaMemcpyAsync(gcu_dev, gcu.data(), size_t(ng + 1) * 8, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaMemcpyAsync(soff_dev, soff.data(), size_t(ng) * 8, cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaMemcpyAsync(sld_dev, sld.data(), size_t(ng) * 4, cudaMemcpyHostToDevice, st) != cudaSuccess)
      return DSA_ERR_CUDA;
    const long long grows = gcu[ng];
    if (grows > 0) {
      const long long rbase = cu_seqlens[b0];
      if (launch_pdl(varlen_score_rows_kernel, dim3(static_cast<unsigned>((grows + 255) / 256)), dim3(256), 0, st,
                     static_cast<const long long*>(gcu_dev), ng, static_cast<const long long*>(soff_dev),
                     static_cast<const int*>(sld_dev), k, tk_off + rbase, tk_len + rbase) != cudaSuccess)
        return DSA_ERR_CUDA;
      e = last_launch_status();
      if (e != DSA_OK) return e;
      e = run_topk(sc, 0, tk_off + rbase, tk_len + rbase, 0, static_cast<int>(grows), k, idx + rbase * k, k, st);
      if (e != DSA_OK) return e;
    }
  }
  return run_mla(q, c, static_cast<int>(total), idx, row_off, static_cast<int>(total), H, k, scale, out, lse, st,
                 kMlaCausal);
}

uint64_t dsa_launch_count(void) { return g_launches.load(); }

int dsa_prefill_block_rows(int L, int k, int r0) {
  if (L <= 0 || k <= 0) return 0;
  return prefill_block_rows(L, k, r0);
}

dsa_status_t dsa_check_bounded_wait(int32_t* result, void* stream) {
  if (!result) return DSA_ERR_INVALID_ARG;
  if (!aligned16(result)) return DSA_ERR_ALIGNMENT;
  wait_selfcheck_kernel<<<1, 64, 0, static_cast<cudaStream_t>(stream)>>>(result);
  return last_launch_status();
}

size_t dsa_checks_selftest_bytes(void) { return size_t(1) << 20; }

dsa_status_t dsa_checks_selftest(int which, void* scratch, void* stream) {
  if (!scratch || (which != 0 && which != 1)) return DSA_ERR_INVALID_ARG;
  if (!aligned16(scratch)) return DSA_ERR_ALIGNMENT;
#ifndef DSA_CHECKS
  return DSA_ERR_UNSUPPORTED_SHAPE;
#else
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* b = static_cast<char*>(scratch);
  if (cudaMemsetAsync(b, 0, dsa_checks_selftest_bytes(), st) != cudaSuccess) return DSA_ERR_CUDA;
  if (which == 0) {
    // a top-k output row of k = 4 over n = 10 keys, not ascending: [5, 3, 7, -1]
    static const int32_t row[4] = {5, 3, 7, -1};
    static const int32_t n = 10;
    int32_t* idx = reinterpret_cast<int32_t*>(b);
    int32_t* len = reinterpret_cast<int32_t*>(b + 256);
    // (copies from pageable memory: the source is read before cudaMemcpyAsync returns)
    if (cudaMemcpyAsync(idx, row, sizeof(row), cudaMemcpyHostToDevice, st) != cudaSuccess ||
        cudaMemcpyAsync(len, &n, sizeof(n), cudaMemcpyHostToDevice, st) != cudaSuccess)
      return DSA_ERR_CUDA;
    TopkParams p{nullptr, 10, nullptr, len, 0, 1, 4, idx, 4, nullptr};
    topk_check_kernel<<<1, 256, 0, st>>>(p);
    return last_launch_status();
  }
  // one decode-style token with n = 200 keys of a 256-row zero latent, k = 128, 8 heads; its first selected
  // entry (250) lies inside the latent but beyond the token's keys
  constexpr int S = 256, H = 8, k = 128;
  uint16_t* c = reinterpret_cast<uint16_t*>(b);                           // [S, 576] bf16 zeros
  uint16_t* q = reinterpret_cast<uint16_t*>(b + S * 1152);                 // [1, H, 576] bf16 zeros
  int32_t* idx = reinterpret_cast<int32_t*>(b + S * 1152 + 16384);         // [1, k]
  int32_t* nk = idx + k;                                                   // [1]
  uint16_t* out = reinterpret_cast<uint16_t*>(b + S * 1152 + 32768);       // [1, H, 512] bf16
  float* lse = reinterpret_cast<float*>(b + S * 1152 + 49152);             // [1, H]
  struct Planted {
    int32_t v[k + 1];
    Planted() {
      for (int j = 0; j < k; ++j) v[j] = j;
      v[0] = 250;   // idx row [250, 1, 2, ..., 127]
      v[k] = 200;   // n_keys
    }
  };
  static const Planted host;
  if (cudaMemcpyAsync(idx, host.v, sizeof(host.v), cudaMemcpyHostToDevice, st) != cudaSuccess) return DSA_ERR_CUDA;
  return run_mla(q, c, S, idx, nullptr, 1, H, k, 0.0416666679f, out, lse, st, kMlaCounts, nk);
#endif
}

#ifdef DSA_TRACE
// traced build only: copy the event stamps out and clear them
__attribute__((visibility("default"))) int dsa_trace_read(unsigned long long* host) {
  if (cudaMemcpyFromSymbol(host, g_trace, sizeof(g_trace)) != cudaSuccess) return DSA_ERR_CUDA;
  static unsigned long long zero[kTraceEvents][kTraceTiles];
  return cudaMemcpyToSymbol(g_trace, zero, sizeof(zero)) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
#endif

size_t dsa_decode_workspace_size(int B, int64_t cache_rows, int H_I, int d_I, int H, int k) {
  (void)H_I; (void)d_I; (void)H;
  if (B <= 0 || cache_rows <= 0 || k <= 0) return 0;
  return decode_ws_bytes(B, decode_score_cap(B, cache_rows), k);
}

dsa_status_t dsa_forward_decode(int B, const int64_t* cache_off, const int32_t* ctx_len, const uint8_t* q_idx,
                                const float* q_scale, const float* w, const uint16_t* q, const uint8_t* k_new,
                                const float* k_scale_new, const uint16_t* c_new, uint8_t* k_cache,
                                float* k_scale_cache, uint16_t* c_cache, int64_t cache_rows, int H_I, int d_I,
                                int H, int k, float scale, int32_t* idx_out, uint16_t* out, float* lse, void* ws,
                                size_t ws_bytes, void* stream) {
  const dsa_status_t chk = decode_args_status(B, cache_off, ctx_len, q_idx, w, q, k_new, k_scale_new, c_new, k_cache,
                                              k_scale_cache, c_cache, cache_rows, H_I, d_I, H, k, idx_out, out);
  if (chk != DSA_OK) return chk;
  if (!ws || ws_bytes < dsa_decode_workspace_size(B, cache_rows, H_I, d_I, H, k)) return DSA_ERR_WORKSPACE;
  DecodeLayout lay{};
  lay.cache_off = reinterpret_cast<const long long*>(cache_off);
  lay.cache_rows = cache_rows;
  return run_decode(B, lay, ctx_len, q_idx, q_scale, w, q, k_new, k_scale_new, c_new, k_cache, k_scale_cache,
                    c_cache, decode_score_cap(B, cache_rows), H, k, scale, idx_out, out, lse, ws,
                    static_cast<cudaStream_t>(stream));
}

size_t dsa_decode_paged_workspace_size(int B, int max_pages, int page_rows, int H_I, int d_I, int H, int k) {
  (void)H_I; (void)d_I; (void)H;
  if (B <= 0 || max_pages <= 0 || page_rows <= 0 || k <= 0) return 0;
  return decode_ws_bytes(B, decode_score_cap(B, static_cast<int64_t>(B) * max_pages * page_rows), k);
}

dsa_status_t dsa_forward_decode_paged(int B, const int32_t* page_table, int max_pages, int page_rows,
                                      const int32_t* ctx_len, const uint8_t* q_idx, const float* q_scale,
                                      const float* w, const uint16_t* q, const uint8_t* k_new,
                                      const float* k_scale_new, const uint16_t* c_new, uint8_t* k_cache,
                                      float* k_scale_cache, uint16_t* c_cache, int num_pages, int H_I, int d_I,
                                      int H, int k, float scale, int32_t* idx_out, uint16_t* out, float* lse,
                                      void* ws, size_t ws_bytes, void* stream) {
  if (!page_table || max_pages <= 0 || num_pages <= 0) return DSA_ERR_INVALID_ARG;
  if (page_rows <= 0 || page_rows % 128 != 0) return DSA_ERR_UNSUPPORTED_SHAPE;
  const int64_t pool_rows = static_cast<int64_t>(num_pages) * page_rows;
  if (pool_rows > INT32_MAX) return DSA_ERR_UNSUPPORTED_SHAPE;   // tensor-map row coordinates are 32-bit
  // every check of the flat call applies, with the page pools as the caches (any non-null cache_off passes)
  const dsa_status_t chk = decode_args_status(B, reinterpret_cast<const int64_t*>(page_table), ctx_len, q_idx, w, q,
                                              k_new, k_scale_new, c_new, k_cache, k_scale_cache, c_cache, pool_rows,
                                              H_I, d_I, H, k, idx_out, out);
  if (chk != DSA_OK) return chk;
  if (!ws || ws_bytes < dsa_decode_paged_workspace_size(B, max_pages, page_rows, H_I, d_I, H, k))
    return DSA_ERR_WORKSPACE;
  DecodeLayout lay{};
  lay.cache_rows = pool_rows;
  lay.page_table = page_table;
  lay.max_pages = max_pages;
  lay.page_rows = page_rows;
  lay.num_pages = num_pages;
  return run_decode(B, lay, ctx_len, q_idx, q_scale, w, q, k_new, k_scale_new, c_new, k_cache, k_scale_cache,
                    c_cache, decode_score_cap(B, static_cast<int64_t>(B) * max_pages * page_rows), H, k, scale,
                    idx_out, out, lse, ws, static_cast<cudaStream_t>(stream));
}

// ------------------------------------------------------------------------------------------ no-allocation decode
// Scratch of dsa_forward_decode_noalloc: a file-scope device array, so the call needs no workspace from the
// caller.  Every GPU that loads the library holds it until the process exits.
static constexpr size_t kNoAllocScratchBytes = size_t(32) << 20;
static __device__ __align__(256) unsigned char g_noalloc_scratch[kNoAllocScratchBytes];

namespace {
// Device address of g_noalloc_scratch on each device, looked up with that device current (host code may not use
// the array's name as a device address).  The address belongs to the context that loaded the module: it is kept
// together with that context and looked up again when the device's current context is another one (after a
// cudaDeviceReset, for instance).
constexpr int kMaxDevices = 64;
struct ScratchAddr {
  void* ctx = nullptr;
  void* ptr = nullptr;
};
ScratchAddr g_noalloc[kMaxDevices];
std::mutex g_noalloc_mutex;

using CtxGetCurrentFn = CUresult (*)(CUcontext*);
CtxGetCurrentFn ctx_get_current_fn() {
  static CtxGetCurrentFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuCtxGetCurrent", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<CtxGetCurrentFn>(p);
  });
  return fn;
}

dsa_status_t noalloc_scratch(void** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return DSA_ERR_CUDA;
  CtxGetCurrentFn get_ctx = ctx_get_current_fn();
  CUcontext ctx = nullptr;   // null while this thread has no current context yet
  if (!get_ctx || get_ctx(&ctx) != CUDA_SUCCESS) return DSA_ERR_CUDA;
  std::lock_guard<std::mutex> lock(g_noalloc_mutex);
  ScratchAddr& a = g_noalloc[dev];
  if (!a.ptr || !ctx || a.ctx != static_cast<void*>(ctx)) {
    void* ptr = nullptr;
    // the lookup makes the device's primary context current when it is not yet
    if (cudaGetSymbolAddress(&ptr, g_noalloc_scratch) != cudaSuccess || !ptr) return DSA_ERR_CUDA;
    if (get_ctx(&ctx) != CUDA_SUCCESS || !ctx) return DSA_ERR_CUDA;
    a.ctx = ctx;
    a.ptr = ptr;
  }
  *out = a.ptr;
  return DSA_OK;
}
}  // namespace

size_t dsa_decode_noalloc_scratch_bytes(void) { return kNoAllocScratchBytes; }

dsa_status_t dsa_forward_decode_noalloc(int B, const int64_t* cache_off, const int32_t* ctx_len,
                                        const uint8_t* q_idx, const float* q_scale, const float* w,
                                        const uint16_t* q, const uint8_t* k_new, const float* k_scale_new,
                                        const uint16_t* c_new, uint8_t* k_cache, float* k_scale_cache,
                                        uint16_t* c_cache, int64_t cache_rows, int H_I, int d_I, int H, int k,
                                        float scale, int32_t* idx_out, uint16_t* out, float* lse, void* stream) {
  const dsa_status_t chk = decode_args_status(B, cache_off, ctx_len, q_idx, w, q, k_new, k_scale_new, c_new, k_cache,
                                              k_scale_cache, c_cache, cache_rows, H_I, d_I, H, k, idx_out, out);
  if (chk != DSA_OK) return chk;
  if (dsa_decode_workspace_size(B, cache_rows, H_I, d_I, H, k) > kNoAllocScratchBytes) return DSA_ERR_WORKSPACE;
  void* scratch = nullptr;
  const dsa_status_t e = noalloc_scratch(&scratch);
  if (e != DSA_OK) return e;
  // the scratch needs no clearing: every byte a call reads there is written earlier in the same call
  return dsa_forward_decode(B, cache_off, ctx_len, q_idx, q_scale, w, q, k_new, k_scale_new, c_new, k_cache,
                            k_scale_cache, c_cache, cache_rows, H_I, d_I, H, k, scale, idx_out, out, lse, scratch,
                            kNoAllocScratchBytes, stream);
}

size_t dsa_sparse_mla_attn_backward_workspace_size(int T, int S, int H, int k) {
  if (T <= 0 || S <= 0 || H <= 0 || H > 128 || !mla_k_ok(k)) return 0;
  return attn_bwd_ws(nullptr, T, S, H, k).bytes;
}

dsa_status_t dsa_sparse_mla_attn_backward(const uint16_t* q, const uint16_t* c, int S, const int32_t* idx,
                                          const uint16_t* out, const float* lse, const uint16_t* dout, int T, int H,
                                          int k, float scale, uint16_t* dq, uint16_t* dc, void* ws, size_t ws_bytes,
                                          void* stream) {
  if (T < 0 || S <= 0 || H <= 0 || k <= 0 || !dc || (T > 0 && (!q || !c || !idx || !out || !lse || !dout || !dq)))
    return DSA_ERR_INVALID_ARG;
  if (H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q) || !aligned16(c) || !aligned16(idx) || !aligned16(out) || !aligned16(dout) || !aligned16(dq) ||
      !aligned16(dc) || !aligned16(ws))
    return DSA_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(dc, 0, size_t(S) * mbw::D * 2, st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  const AttnBwdWs w = attn_bwd_ws(ws, T, S, H, k);
  if (!ws || ws_bytes < w.bytes) return DSA_ERR_WORKSPACE;
  return run_attn_bwd(q, c, S, idx, out, lse, dout, T, H, k, scale, dq, dc, w, st);
}

size_t dsa_indexer_kl_backward_workspace_size(int T) { return T > 0 ? kl_bwd_ws_bytes(T) : 0; }

dsa_status_t dsa_indexer_kl_backward(const uint16_t* q, const uint16_t* c, int S, const int32_t* idx,
                                     const float* sel_scores, const float* lse, const float* dkl, int T, int H, int k,
                                     float scale, float* dsel, void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || S <= 0 || H <= 0 || k <= 0 || (T > 0 && (!q || !c || !idx || !sel_scores || !lse || !dsel)))
    return DSA_ERR_INVALID_ARG;
  if (H > 128 || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q) || !aligned16(c) || !aligned16(idx) || !aligned16(ws)) return DSA_ERR_ALIGNMENT;
  if (T == 0) return DSA_OK;
  if (!ws || ws_bytes < kl_bwd_ws_bytes(T)) return DSA_ERR_WORKSPACE;
  return run_kl_bwd(q, c, S, idx, sel_scores, lse, dkl, T, H, k, scale, dsel, ws, static_cast<cudaStream_t>(stream));
}

size_t dsa_indexer_scores_backward_workspace_size(int T, int S, int H_I, int d_I, int k) {
  if (T <= 0 || S <= 0 || !indexer_shape_ok(H_I, d_I) || !mla_k_ok(k)) return 0;
  return index_bwd_ws(nullptr, T, S, H_I, d_I, k).bytes;
}

dsa_status_t dsa_indexer_scores_backward(const uint8_t* q_idx, const float* q_scale, const uint8_t* k_idx,
                                         const float* k_scale, const float* w, const int32_t* idx, const float* dsel,
                                         int T, int S, int H_I, int d_I, int k, uint16_t* dq, uint16_t* dk, float* dw,
                                         void* ws, size_t ws_bytes, void* stream) {
  if (T < 0 || S <= 0 || k <= 0 || !dk || (T > 0 && (!q_idx || !k_idx || !w || !idx || !dsel || !dq || !dw)))
    return DSA_ERR_INVALID_ARG;
  if (!indexer_shape_ok(H_I, d_I) || !mla_k_ok(k)) return DSA_ERR_UNSUPPORTED_SHAPE;
  if (!aligned16(q_idx) || !aligned16(k_idx) || !aligned16(idx) || !aligned16(dq) || !aligned16(dk) || !aligned16(ws))
    return DSA_ERR_ALIGNMENT;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (T == 0)
    return cudaMemsetAsync(dk, 0, size_t(S) * d_I * 2, st) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
  const IndexBwdWs a = index_bwd_ws(ws, T, S, H_I, d_I, k);
  if (!ws || ws_bytes < a.bytes) return DSA_ERR_WORKSPACE;
  IndexerBwdParams p{};
  p.q_idx = q_idx;
  p.q_scale = q_scale;
  p.k_idx = k_idx;
  p.k_scale = k_scale;
  p.w = w;
  p.idx = idx;
  p.dsel = dsel;
  p.dq = dq;
  p.dw = dw;
  p.k = k;
  p.S = S;
  return H_I == 64 ? run_index_bwd<64, 128>(p, T, dk, a, st) : run_index_bwd<4, 64>(p, T, dk, a, st);
}

dsa_status_t dsa_rope_frequencies(int rot_dim, double base, double factor, int orig_len, double turns_fast,
                                  double turns_slow, double* inv_freq, float* mscale) {
  if (rot_dim <= 0 || rot_dim % 2 || !(base > 1.0) || !(factor >= 1.0) || !inv_freq || !std::isfinite(base) ||
      !std::isfinite(factor))
    return DSA_ERR_INVALID_ARG;
  if (factor > 1.0 &&
      (orig_len <= 0 || !(turns_slow > 0.0) || !(turns_fast > turns_slow) || !std::isfinite(turns_fast)))
    return DSA_ERR_INVALID_ARG;
  const int n = rot_dim / 2;
  double low = 0.0, high = 1.0;
  if (factor > 1.0) {
    // pair index whose wavelength makes `turns` turns over orig_len positions.  Either end of the blend may lie
    // outside the pairs that there are: it is then cut off, not squeezed into them.
    auto pair_of = [&](double turns) {
      return rot_dim * std::log(orig_len / (turns * 6.283185307179586)) / (2.0 * std::log(base));
    };
    low = std::floor(pair_of(turns_fast));
    high = std::ceil(pair_of(turns_slow));
  }
  for (int i = 0; i < n; ++i) {
    const double f = std::pow(base, -2.0 * i / rot_dim);
    double slow = 0.0;
    if (factor > 1.0) slow = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 1.0)));
    inv_freq[i] = f / factor * slow + f * (1.0 - slow);
  }
  if (mscale) *mscale = factor > 1.0 ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return DSA_OK;
}

dsa_status_t dsa_rope(const void* x, int64_t x_stride_t, int64_t x_stride_h, void* out, int64_t out_stride_t,
                      int64_t out_stride_h, const int32_t* positions, int pos0, const double* inv_freq, int T, int H,
                      int D, int rot_off, int rot_dim, int interleaved, float mscale, int dtype, void* stream) {
  return run_rope(x, x_stride_t, x_stride_h, out, out_stride_t, out_stride_h, positions, pos0, inv_freq, T, H, D,
                  rot_off, rot_dim, interleaved, mscale, dtype, false, stream);
}

dsa_status_t dsa_rope_backward(const void* dout, int64_t dout_stride_t, int64_t dout_stride_h, void* dx,
                               int64_t dx_stride_t, int64_t dx_stride_h, const int32_t* positions, int pos0,
                               const double* inv_freq, int T, int H, int D, int rot_off, int rot_dim, int interleaved,
                               float mscale, int dtype, void* stream) {
  return run_rope(dout, dout_stride_t, dout_stride_h, dx, dx_stride_t, dx_stride_h, positions, pos0, inv_freq, T, H, D,
                  rot_off, rot_dim, interleaved, mscale, dtype, true, stream);
}

}  // extern "C"
