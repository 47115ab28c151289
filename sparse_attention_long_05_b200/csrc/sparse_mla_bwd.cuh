// Backward pass of the sparse MLA attention (sparse_mla.cuh) and the gradient of the indexer's objective.
//
// For token t, head h and selected entry i (row s = idx[t][i] of c), with the forward's out and lse:
//   P  = exp(scale q_h . c_s - lse_h)            the probabilities, recomputed from q, c and lse
//   dP = dout_h . c_s[:512]
//   dS = scale P (dP - delta_h),  delta_h = dout_h . out_h
//   dq_h = sum_i dS c_s                          dc_s = sum over (t, i) with idx[t][i] = s of
//                                                       sum_h dS q_h + [sum_h P dout_h, 0 over the position dims]
// Five products of 2 x 128 heads x 2048 entries x (576, 512, 576, 576, 512) per token: bound by the tensor cores.
//
// One SM cannot hold a token's q and dout (272 KB) beside its keys, nor dq's and dc's accumulators together (576 of
// the 512 columns of tensor memory each), so the pass runs as three tensor-core kernels over a chunk of tokens, each
// with a resident operand that fits, and P and dS (bf16, 1 MB a token) between them:
//   mla_bwd_p_kernel   (token) per CTA pair: keys are the M dimension; q's rows stay in one CTA's shared memory and
//                      dout's in the other's, and every gathered chunk of 256 keys x 64 dims meets both at once;
//   mla_bwd_dc_kernel  (token, 256 dims): [dS | P] (256 keys x heads) times [q ; dout] (heads x 256 dims), resident;
//                      writes each entry's own contribution to dc (16 bits a value, see scatter.cuh);
//   mla_bwd_dq_kernel  (token, 192 dims): dS^T (heads x keys) times the gathered keys (keys x 192 dims), accumulated
//                      over the token's keys in tensor memory.
// A last kernel (scatter.cuh) sums the contributions of each row of c in token order: the result does not depend on
// the order of execution, which atomics would not give.
//
// P and dS are rounded to bf16, by at most 2^-8 of their value, as the operands of the second products have to be.  All
// sums are fp32.
//
// Measured on 2048 tokens of a 32K sequence, k = 2048, 128 heads (launches one by one): P and dS 1137 us, contributions
// 1416, dq 590, their sum 831, delta and the table 176; 4.8 to 5.0 ms in a row (2.95 TFLOP: 0.42 to 0.44 of the
// sustained bf16 rate).  The objective's gradient takes 564 us (1.10 PFLOP/s).  The two pair kernels are bound by
// shared memory: in the contributions' the operand fetches of the tensor cores and the warps' own traffic (staged pieces) take
// about 45 % of its cycles each.  dq reads 40 KB a stage at 81 GB/s an SM, what gathers and tiles together reach here;
// the sum runs at 0.88 of HBM.
#pragma once
#include "common.cuh"
#include "scatter.cuh"
#include "sparse_mla.cuh"

namespace dsa {

struct MlaBwdParams {
  const int* idx;              // [T, k] selections of the chunk's tokens
  const int* n_end;            // [T] slots up to the token's last valid entry
  const uint16_t* c;           // [S, 576]
  const float* lse;            // [T, H]
  const float* delta;          // [T, H]
  uint16_t* pds;               // [T * kp, 2 HP] bf16: dS of HP heads, then P of HP heads, for every slot
  uint16_t* dq;                // [T, H, 576]
  float* dq_part;              // splits > 1: [T * splits, H, 576] sums of each split
  int T, t0;                   // tokens of the chunk; the first one's index in q and dout
  int splits;                  // a token's tiles are dealt to this many items (P and dS, contributions)
  int H, HP;                   // heads; heads rounded up to 64
  int k, kp;                   // slots of a token; rounded up to 128
  long long S;
  float scale, scale_log2;
  const float* sel;            // objective's gradient: index scores of the selected entries [T, k]
  const float* dkl;            // [T] or null (1)
  float* dsel;                 // [T, k]
};

// Instruction descriptor of bf16 operands, each K-major or MN-major (A: bit 15, B: bit 16).
__host__ __device__ constexpr uint32_t idesc_bf16_major(int M, int N, bool a_mn, bool b_mn) {
  return idesc_bf16(M, N, b_mn) | (a_mn ? 1u << 15 : 0u);
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, uint32_t src, int x, int y) {
  asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.tile.bulk_group [%0, {%2, %3}], [%1];"
               :: "l"(map), "r"(src), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// all but the last N committed stores have read their shared memory / all have been written
template <int N = 0>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" :: "n"(N) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The threads of a named barrier agree on an outcome (all of them have to be true): the warps that meet at it leave
// their loops together, so none is left waiting when a wait of another one runs out.
__device__ __forceinline__ bool named_bar_all(int id, int nthreads, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %3, 0;\n\t"
      "bar.red.and.pred p, %1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r) : "r"(id), "r"(nthreads), "r"(static_cast<uint32_t>(v)) : "memory");
  return r != 0;
}

// ---- CTA pairs (tcgen05 cta_group::2): the even CTA of the cluster issues MMAs whose A rows and whose halves of B lie
// in both CTAs' shared memory (same offsets), and whose D rows lie in both tensor memories.
__device__ __forceinline__ void mma2_bf16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}
// arrives on the barrier at this offset in both CTAs when every MMA issued so far has completed
__device__ __forceinline__ void mma2_commit(uint32_t bar) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               :: "r"(bar), "h"(static_cast<uint16_t>(3)) : "memory");
}
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];"
               :: "l"(map), "r"(x), "r"(y), "r"(z) : "memory");
}
// loads into this CTA's shared memory that complete on a barrier of either CTA of the pair (a cluster address)
__device__ __forceinline__ void tma2_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5}], [%2];"
      :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ void tma2_load_2d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];"
      :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void tma2_gather4(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x,
                                             int r0, int r1, int r2, int r3) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
      :: "r"(dst), "l"(map), "r"(bar), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3) : "memory");
}
// Relaxed: what it announces (tensor memory read to the end, or nothing at all) is complete when it is issued, and a
// release would first wait for every store of P and dS the thread has in flight.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar_cluster) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" :: "r"(bar_cluster) : "memory");
}

// one 32-byte store (32-byte aligned): a whole sector of the lane's own row
__device__ __forceinline__ void st_global_32(void* at, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
               :: "l"(at), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Tiles [j0, j1) of a token with n_end slots that split `sp` of `splits` works on (`keys` a tile).
struct TileSpan {
  int j0, j1;
};
__device__ __forceinline__ TileSpan tile_span(int n_end, int keys, int sp, int splits) {
  const int tiles = (n_end + keys - 1) / keys, per = (tiles + splits - 1) / splits;
  return {min(tiles, sp * per), min(tiles, (sp + 1) * per)};
}

// Bounded waits as mbar_wait and warp_wait, the part behind a first unsuccessful look in a function of its own: where a
// kernel's roles together overflow the instruction cache, the copies of that part cost more than the call (dq 96 -> 88
// us for 333 tokens, the index scores' pass 534 -> 494 for 2048; the probabilities' kernels fit and keep theirs in
// line).
__device__ __noinline__ bool mbar_wait_far(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const long long t0 = clock64();
  while (!mbar_test(bar, parity)) {
    if (*abort_flag) return false;
    if (clock64() - t0 > g_wait_limit) {
      *abort_flag = 1;
      raise_status(DSA_ERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
__device__ __forceinline__ bool lean_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_test(bar, parity) || mbar_wait_far(bar, parity, abort_flag);
}
__device__ __forceinline__ bool lean_warp_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag) {
  const bool ok = lean_wait(bar, parity, abort_flag);
  return __all_sync(0xffffffffu, ok);
}

namespace mbw {
constexpr int NK = 128;                 // keys per tile (the M dimension of P and dC)
constexpr int D = 576, DV = 512;
constexpr int DCH = D / 64;             // 9 chunks of 64 dims
constexpr int CHUNK = 128 * 128;        // 128 rows x 64 bf16
constexpr int HCHUNK = 64 * 128;        // 64 rows x 64 bf16
constexpr uint32_t TMEM_COLS = 512;
constexpr int BAR_BYTES = 1024;         // barriers, the tensor-memory address, the abort flag, small arrays
constexpr int OFF_TMEM = 512, OFF_ABORT = 516;

// ---- mla_bwd_p_kernel
namespace p {
constexpr int THREADS = 576;            // w0 resident rows, w1 MMA, w2 w3 w8..13 gathers, w4..7 w14..17 probabilities
constexpr int NS_MAX = 5;
constexpr int B_RES_FULL = 0, B_RES_EMPTY = B_RES_FULL + DCH, B_RING_FULL = B_RES_EMPTY + DCH;
constexpr int B_RING_EMPTY = B_RING_FULL + NS_MAX, B_ACC_FULL = B_RING_EMPTY + NS_MAX, B_ACC_EMPTY = B_ACC_FULL + 4;
constexpr int B_SUMS = B_ACC_EMPTY + 4;                       // objective: the other CTA's sums of a token (2 buffers)
constexpr int B_COUNT = B_SUMS + 2;
static_assert(B_COUNT * 8 <= OFF_TMEM, "barrier area");
constexpr int OFF_SUMS = 528;                                 // objective: [2 buffers] of 16 bytes from the other CTA
constexpr int OFF_HEADS = BAR_BYTES;                          // lse and delta of the token's heads, 2 buffers x 1 KB
constexpr int OFF_RES = OFF_HEADS + 2048;
template <bool KL> struct Map {
  static constexpr int RES_CHUNK = KL ? HCHUNK : CHUNK;       // a 64-dim chunk of the resident rows (the last: 64 rows)
  static constexpr int RES = 8 * RES_CHUNK + HCHUNK;          // 72 KB, 136 KB
  static constexpr int SC = KL ? 3 : 1;                       // gathered chunks (16 KB) of a ring stage
  static constexpr int NS = KL ? 3 : 5;                       // ring stages
  static constexpr int WPS = KL ? 4 : 2;                      // warps that fill a stage
  static constexpr int NACC = KL ? 4 : 2;                     // accumulators of 128, 256 columns
  static constexpr int OFF_RING = OFF_RES + RES;
  static constexpr int SMEM = OFF_RING + NS * SC * CHUNK + 1024;
  static_assert(DCH % SC == 0 && SC * 32 % WPS == 0 && SC * 32 / WPS <= 32, "stage split");
};
static_assert(Map<false>::SMEM <= 232448 && Map<true>::SMEM <= 232448, "shared memory per CTA");
static_assert(OFF_RES % 1024 == 0 && OFF_SUMS + 32 <= BAR_BYTES && Map<true>::NS <= NS_MAX, "layout");
}  // namespace p

// ---- mla_bwd_dc_kernel
namespace dc {
constexpr int THREADS = 384;            // w0 resident rows, w1 MMA, w2 dS and P, w4..7 w8..11 contributions
constexpr int NS = 3;                   // ring stages: dS or P of 128 keys x all heads (two 64-head blocks, 32 KB)
constexpr int UNIT = 2 * HCHUNK;        // resident operand of 64 heads: 64 heads x 128 dims (16 KB)
constexpr int NU = 4;                   // units: q of heads 0..63, 64..127, dout of the same
constexpr int B_RES_FULL = 0, B_RES_EMPTY = B_RES_FULL + NU, B_RING_FULL = B_RES_EMPTY + NU;
constexpr int B_RING_EMPTY = B_RING_FULL + NS, B_ACC_FULL = B_RING_EMPTY + NS, B_ACC_EMPTY = B_ACC_FULL + 2;
static_assert((B_ACC_EMPTY + 2) * 8 <= OFF_TMEM, "barrier area");
constexpr int OFF_RES = BAR_BYTES, OFF_RING = OFF_RES + NU * UNIT, OFF_OUT = OFF_RING + NS * 2 * CHUNK;
constexpr int SMEM = OFF_OUT + 8 * 2 * 4096 + 1024;   // two staging areas (32 keys x 64 dims) of each of eight warps
static_assert(SMEM <= 232448, "shared memory per CTA");
}  // namespace dc

// ---- mla_bwd_dq_kernel
namespace dq {
constexpr int THREADS = 448;
constexpr int KT = 64;                  // keys per stage
constexpr int A_BYTES = 2 * HCHUNK, STAGE = A_BYTES + 3 * HCHUNK;   // dS: 64 keys x 128 heads; keys: 64 x 192 dims
constexpr int NS = 5;
constexpr int B_RING_FULL = 0, B_RING_EMPTY = B_RING_FULL + NS;
constexpr int B_ACC_FULL = B_RING_EMPTY + NS, B_ACC_EMPTY = B_ACC_FULL + 2;
static_assert((B_ACC_EMPTY + 2) * 8 <= OFF_TMEM, "barrier area");
constexpr int OFF_RING = BAR_BYTES;
constexpr int SMEM = OFF_RING + NS * STAGE + 1024;
static_assert(SMEM <= 232448 && STAGE % 1024 == 0 && KT == 64, "stages");
}  // namespace dq
}  // namespace mbw

// Shared start and end of the three kernels: barriers, tensor memory, launch order.
struct BwdCta {
  uint8_t* smem;
  uint32_t sbase;
  volatile int* abort_flag;
  uint32_t tmem;
  __device__ __forceinline__ uint32_t bar(int slot) const { return sbase + 8 * slot; }
};
__device__ __forceinline__ BwdCta bwd_base(uint8_t* raw) {
  BwdCta c;
  c.smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~static_cast<uintptr_t>(1023));
  c.sbase = smem_u32(c.smem);
  c.abort_flag = reinterpret_cast<volatile int*>(c.smem + mbw::OFF_ABORT);
  c.tmem = 0;
  return c;
}
// after the barriers are initialised by thread 0: tensor memory by warp 1 (of both CTAs of a pair), then the
// predecessor's results
template <bool PAIR = false>
__device__ __forceinline__ void bwd_begin(BwdCta& c) {
  if (threadIdx.x == 0) {
    *c.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp_id() == 1) {
    if constexpr (PAIR) {
      asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                   :: "r"(c.sbase + mbw::OFF_TMEM), "r"(mbw::TMEM_COLS) : "memory");
      asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
      tmem_alloc(c.sbase + mbw::OFF_TMEM, mbw::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();      // the barriers of both CTAs are initialised
  tc_fence_after();
  c.tmem = *reinterpret_cast<volatile uint32_t*>(c.smem + mbw::OFF_TMEM);
  pdl_allow_next();
  pdl_wait();
}
template <bool PAIR = false>
__device__ __forceinline__ void bwd_end(BwdCta& c) {
  tc_fence_before();
  __syncthreads();
  if constexpr (PAIR) {
    if (*c.abort_flag) {                   // loads that complete on the other CTA's barriers land meanwhile
      const long long t0 = clock64();
      while (clock64() - t0 < (g_wait_limit >> 8)) {
      }
    }
    cluster_sync();                        // no CTA leaves while its peer may still touch its shared memory
  }
  if (warp_id() == 1) {
    tc_fence_after();
    if constexpr (PAIR)
      asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;"
                   :: "r"(c.tmem), "r"(mbw::TMEM_COLS) : "memory");
    else
      tmem_dealloc(c.tmem, mbw::TMEM_COLS);
  }
}

// 16 bytes into shared memory, or zeros where nothing is to be read
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" :: "r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
// one arrival on `bar` (of those it was initialised to expect) when this thread's copies so far have landed
__device__ __forceinline__ void cp_async_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" :: "r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// P and dS of one token per CTA pair, or (KL) the gradient of the objective of one token per pair.
//
// M = 256 keys (128 in each CTA, which gathers only its own), N = 2 HP: CTA 0 holds q's rows and CTA 1 dout's, so that
// one MMA gives S^T (columns 0 .. HP - 1) and dP^T (HP .. 2 HP - 1) of all heads; the position dims, which dout lacks,
// are an N = HP product with half of q's rows in each CTA.  KL: N = HP, half of q's rows in each CTA.  With both CTAs
// of a token sharing their halves, each key is gathered once per token: gathers land after 1.5 to 2 us under load
// (80 KB are in flight a CTA, KL 144 KB).  The resident rows are released chunk by chunk during the token's last tile,
// so the next token's loads overlap it.
template <bool KL>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(mbw::p::THREADS, 1)
mla_bwd_p_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_do,
                 const __grid_constant__ CUtensorMap tm_c, const MlaBwdParams p) {
  using namespace mbw;
  using namespace mbw::p;
  using M = Map<KL>;
  constexpr int NS = M::NS, NACC = M::NACC, SC = M::SC, SPT = DCH / SC;   // stages of a tile
  extern __shared__ uint8_t smem_raw[];
  BwdCta cta = bwd_base(smem_raw);
  const uint32_t sbase = cta.sbase;
  volatile int* abort_flag = cta.abort_flag;
  const int warp = warp_id(), lane = lane_id();
  const int rank = static_cast<int>(cluster_rank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < DCH; ++i) { mbar_init(cta.bar(B_RES_FULL + i), 2); mbar_init(cta.bar(B_RES_EMPTY + i), 1); }
    for (int i = 0; i < NS; ++i) {
      mbar_init(cta.bar(B_RING_FULL + i), 2 * M::WPS);
      mbar_init(cta.bar(B_RING_EMPTY + i), 1);
    }
    for (int i = 0; i < NACC; ++i) { mbar_init(cta.bar(B_ACC_FULL + i), 1); mbar_init(cta.bar(B_ACC_EMPTY + i), 8); }
    for (int i = 0; i < 2; ++i) mbar_init(cta.bar(B_SUMS + i), 1);
  }
  bwd_begin<true>(cta);
  const uint32_t tmem = cta.tmem;
  const uint32_t res = sbase + OFF_RES, ring = sbase + M::OFF_RING;
  const uint32_t lead = map_cluster(sbase, 0);     // CTA 0's barriers, where every load of the pair completes
  const int first = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);
  const int splits = KL ? 1 : p.splits, items = p.T * splits;
  auto token = [&](int item) { return splits == 1 ? item : item / splits; };
  auto span = [&](int item) {
    return tile_span(p.n_end[token(item)], 2 * NK, splits == 1 ? 0 : item % splits, splits);
  };
  bool ok = true;
  int n = 0;                              // items with tiles, walked so far

  if (warp == 0) {
    // ===================================================================== resident rows of q (and dout)
    // Three lanes take a chunk each: one thread alone needs about 300 ns a load, 5 us an item, which nothing overlaps.
    // The next item's rows are brought into L2 meanwhile.
    for (int item = first; item < items && ok; item += stride) {
      const TileSpan sp = span(item);
      if (sp.j0 >= sp.j1) continue;
      const int t = token(item);
      auto rows = [&](int c, int tok, bool ahead) {      // this CTA's boxes of chunk c
        const CUtensorMap* map = !KL && c < 8 && rank ? &tm_do : &tm_q;
        const bool part = KL || c == 8;
        const int boxes = part ? 1 : p.HP / 64, h0 = part ? rank * (p.HP / 2) : 0;
        const uint32_t full = lead + 8 * (B_RES_FULL + c);
        if (!ahead) mbar_arrive_expect_tx_remote(full, boxes * HCHUNK);
        for (int i = 0; i < boxes; ++i) {
          if (ahead) tma_prefetch_3d(map, 64 * c, h0 + 64 * i, p.t0 + tok);
          else tma2_load_3d(res + c * M::RES_CHUNK + i * HCHUNK, map, full, 64 * c, h0 + 64 * i, p.t0 + tok);
        }
      };
      for (int c0 = 0; c0 < DCH && ok; c0 += 3) {
        bool got = true;
        if (lane < 3) {
          got = mbar_wait(cta.bar(B_RES_EMPTY + c0 + lane), (n & 1) ^ 1, abort_flag);
          if (got) rows(c0 + lane, t, false);
        }
        ok = __all_sync(0xffffffffu, got);
      }
      if (item + stride < items && token(item + stride) != t && lane < DCH) rows(lane, token(item + stride), true);
      __syncwarp();
      ++n;
    }
  } else if (warp == 2 || warp == 3 || (warp >= 8 && warp < 14)) {
    // ===================================================================== gathers (gather4: four rows x 64 dims)
    // One lane issues one gather4 of a stage; the warps that fill a stage share its 32 SC of them, and stages go round
    // the groups of such warps.  The entries of the next tile are read while this one is gathered.
    // An empty or invalid slot reads row slot % S (any row would do, its P and dS are set to zero; one row for all
    // would be one L2 line for the whole GPU: 30 us against 18 for 96 short tokens); a CTA whose keys of a tile are all
    // behind the token's last entry reads nothing.
    constexpr int PER = SC * 32 / M::WPS, GROUPS = 8 / M::WPS;
    // a group that comes to a stage again has seen the chunk before last of it consumed (its own last stage could not
    // be filled before): the barrier's parity tells the two last phases apart
    static_assert(GROUPS <= NS, "stages");
    const int gw = (warp < 8) ? warp - 2 : warp - 6;
    const int grp = gw / M::WPS, gi = (gw % M::WPS) * PER + lane, cc = gi / 32, rg = gi % 32;
    const bool active = lane < PER;
    int m = 0;                             // stages of the tiles before this one
    for (int item = first; item < items && ok; item += stride) {
      const TileSpan sp = span(item);
      if (sp.j0 >= sp.j1) continue;
      const int* ids = p.idx + static_cast<long long>(token(item)) * p.k;
      const int n_end = p.n_end[token(item)];
      auto entries = [&](int j) {          // k is a multiple of 64, a lane's four slots lie on one side of it
        const int slot = (2 * j + rank) * NK + 4 * rg;
        return slot < p.k ? __ldg(reinterpret_cast<const int4*>(ids + slot)) : make_int4(-1, -1, -1, -1);
      };
      int4 e = entries(sp.j0);
      for (int j = sp.j0; j < sp.j1 && ok; ++j, m += SPT) {
        const int slot = (2 * j + rank) * NK + 4 * rg;
        auto row = [&](int x, int i) {
          return (x >= 0 && x < p.S) ? x : static_cast<int>(slot + i < p.S ? slot + i : (slot + i) % p.S);
        };
        const bool any = (2 * j + rank) * NK < n_end;
        const int r0 = row(e.x, 0), r1 = row(e.y, 1), r2 = row(e.z, 2), r3 = row(e.w, 3);
        if (j + 1 < sp.j1) e = entries(j + 1);
        for (int s = (grp + (GROUPS - 1) * m) % GROUPS; s < SPT; s += GROUPS) {   // (m + s) % GROUPS == grp
          const int st = (m + s) % NS;
          const uint32_t full = lead + 8 * (B_RING_FULL + st);
          bool got = true;
          if (lane == 0) {
            got = mbar_wait(cta.bar(B_RING_EMPTY + st), (((m + s) / NS) & 1) ^ 1, abort_flag);
            if (got && any) mbar_arrive_expect_tx_remote(full, PER * 512);
            else if (got) mbar_arrive_remote(full);
          }
          if (!(ok = __shfl_sync(0xffffffffu, got, 0))) break;
          if (active && any)
            tma2_gather4(ring + (st * SC + cc) * CHUNK + rg * 512, &tm_c, full, 64 * (s * SC + cc), r0, r1, r2, r3);
        }
      }
    }
  } else if (warp == 1) {
    // ===================================================================== MMA issue (CTA 0 for the pair)
    if (rank == 0) {
      Pipe<NS> rp;
      int g = 0;
      const uint32_t wide = idesc_bf16(256, KL ? p.HP : 2 * p.HP, false), narrow = idesc_bf16(256, p.HP, false);
      for (int item = first; item < items && ok; item += stride) {
        const TileSpan sp = span(item);
        if (sp.j0 >= sp.j1) continue;
        for (int j = sp.j0; j < sp.j1 && ok; ++j, ++g) {
          const int ab = g % NACC;
          if (!(ok = warp_wait<true>(cta.bar(B_ACC_EMPTY + ab), ((g / NACC) & 1) ^ 1, abort_flag))) break;
          tc_fence_after();
          for (int sg = 0; sg < SPT; ++sg, rp.advance()) {
            if (j == sp.j0)
              for (int c = sg * SC; c < (sg + 1) * SC && ok; ++c)
                ok = warp_wait<true>(cta.bar(B_RES_FULL + c), n & 1, abort_flag);
            if (!(ok = ok && warp_wait<true>(cta.bar(B_RING_FULL + rp.stage), rp.phase, abort_flag))) break;
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
              for (int cc = 0; cc < SC; ++cc) {
                const int c = sg * SC + cc;
                const uint64_t ad = smem_desc(ring + (rp.stage * SC + cc) * CHUNK, 16, 1024, kLayoutSW128);
                const uint64_t bd = smem_desc(res + c * M::RES_CHUNK, 16, 1024, kLayoutSW128);
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma2_bf16_ss(tmem + (512 / NACC) * ab, ad + 2 * k, bd + 2 * k, c < 8 ? wide : narrow,
                               (c | k) ? 1u : 0u);
                if (j == sp.j1 - 1) mma2_commit(cta.bar(B_RES_EMPTY + c));
              }
              mma2_commit(cta.bar(B_RING_EMPTY + rp.stage));
            }
            __syncwarp();
          }
          if (!ok) break;
          if (elect_one()) mma2_commit(cta.bar(B_ACC_FULL + ab));
          __syncwarp();
        }
        ++n;
      }
    }
  } else {
    // ===================================================================== probabilities (one key a thread)
    // Two groups of four warps take tiles in turn: the work on a tile is a chain of tensor-memory loads, exponentials
    // and stores that takes longer than the tile's MMAs (the objective's gradient: 716 us for 2048 tokens with one
    // group, 616 with two).
    const int grp = warp >= 14 ? 1 : 0;
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    constexpr float kLog2e = 1.4426950408889634f;
    int g = 0;
    for (int item = first; item < items && ok; item += stride) {
      const TileSpan sp = span(item);
      const int t = token(item);
      const long long base = static_cast<long long>(t) * p.k;
      if constexpr (KL) {
        for (int i = (2 * (sp.j1 + grp) + rank) * NK + row; i < p.k; i += 4 * NK) p.dsel[base + i] = 0.f;
      }
      if (sp.j0 >= sp.j1) continue;
      // the token's -lse (in log2 units) and -scale delta.  A head without any probability mass (lse = -inf) and the
      // heads that only fill up the tile get -inf: P = 0.
      float* hs = reinterpret_cast<float*>(cta.smem + OFF_HEADS) + (n & 1) * 256;
      if (grp == 0) {
        const long long at = static_cast<long long>(t) * p.H + row;
        const float l = row < p.H ? p.lse[at] : -INFINITY;
        hs[row] = l == -INFINITY ? -INFINITY : -l * kLog2e;
        if (!KL) hs[128 + row] = row < p.H ? -p.delta[at] * p.scale : 0.f;
      }
      if (!(ok = named_bar_all(1, 256, ok))) break;
      [[maybe_unused]] float m_i = -INFINITY, z_i = 0.f, s_a = 0.f;
      // the entry (KL: and its index score) of the next tile is read while this one is worked on
      auto entry = [&](int j) {
        const int slot = (2 * j + rank) * NK + row;
        return slot < p.k ? __ldg(p.idx + base + slot) : -1;
      };
      auto score = [&](int j) {
        const int slot = (2 * j + rank) * NK + row;
        return KL && slot < p.k ? __ldg(p.sel + base + slot) : 0.f;
      };
      // tile j is the CTA's tile g + j - j0; this group takes those of its parity
      const int j0 = sp.j0 + ((g ^ grp) & 1);
      int e_next = j0 < sp.j1 ? entry(j0) : -1;
      [[maybe_unused]] float x_next = j0 < sp.j1 ? score(j0) : 0.f;
      for (int j = j0; j < sp.j1; j += 2) {
        const int gj = g + j - sp.j0, ab = gj % NACC, slot = (2 * j + rank) * NK + row;
        const bool valid = e_next >= 0 && e_next < p.S;
        [[maybe_unused]] const float x = x_next;
        if (j + 2 < sp.j1) {
          e_next = entry(j + 2);
          x_next = score(j + 2);
        }
        if (!(ok = warp_wait(cta.bar(B_ACC_FULL + ab), (gj / NACC) & 1, abort_flag))) break;
        tc_fence_after();
        const uint32_t acc = lane_addr + tmem + (512 / NACC) * ab;
        auto release = [&]() {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(lead + 8 * (B_ACC_EMPTY + ab));
        };
        if constexpr (KL) {
          float a0 = 0.f, a1 = 0.f;
#pragma unroll 1
          for (int c = 0; c < p.HP / 32; ++c) {
            uint32_t v[32];
            tmem_ld32(acc + 32 * c, v);
            tmem_wait_ld();
            if (c == p.HP / 32 - 1) release();
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 l = *reinterpret_cast<const float4*>(hs + 32 * c + i);
              a0 += ex2_approx(fmaf(__uint_as_float(v[i]), p.scale_log2, l.x));
              a1 += ex2_approx(fmaf(__uint_as_float(v[i + 1]), p.scale_log2, l.y));
              a0 += ex2_approx(fmaf(__uint_as_float(v[i + 2]), p.scale_log2, l.z));
              a1 += ex2_approx(fmaf(__uint_as_float(v[i + 3]), p.scale_log2, l.w));
            }
          }
          if (slot < p.k) {
            const float a = valid ? a0 + a1 : 0.f;
            p.dsel[base + slot] = a;       // read back below, behind a barrier
            if (valid) {
              s_a += a;
              if (x > m_i) {
                z_i = z_i * ex2_approx((m_i - x) * kLog2e) + 1.f;
                m_i = x;
              } else if (x != -INFINITY) {     // (a NaN stays in the sum, and with it in the token's gradient)
                z_i += ex2_approx((x - m_i) * kLog2e);
              }
            }
          }
        } else {
          // the warp's 32 keys; kp is a multiple of 128: they lie on one side of it
          const int slot0 = slot - lane;
          uint16_t* out = p.pds + (static_cast<long long>(t) * p.kp + slot) * (2 * p.HP);
          const uint32_t keep = valid ? 0xffffffffu : 0u;     // an empty slot's S or dP may be NaN: its bits go
#pragma unroll 1
          for (int c = 0; c < p.HP / 32; ++c) {
            uint32_t s[32], d[32], ps[16], ds[16];
            tmem_ld32(acc + 32 * c, s);
            tmem_ld32(acc + p.HP + 32 * c, d);
            tmem_wait_ld();
            if (c == p.HP / 32 - 1) release();
            const float* hl = hs + 32 * c;
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
              const float4 l = *reinterpret_cast<const float4*>(hl + i);
              const float4 m = *reinterpret_cast<const float4*>(hl + 128 + i);
              const float p0 = ex2_approx(fmaf(__uint_as_float(s[i]), p.scale_log2, l.x));
              const float p1 = ex2_approx(fmaf(__uint_as_float(s[i + 1]), p.scale_log2, l.y));
              const float p2 = ex2_approx(fmaf(__uint_as_float(s[i + 2]), p.scale_log2, l.z));
              const float p3 = ex2_approx(fmaf(__uint_as_float(s[i + 3]), p.scale_log2, l.w));
              ps[i / 2] = pack_bf16(p0, p1) & keep;
              ps[i / 2 + 1] = pack_bf16(p2, p3) & keep;
              ds[i / 2] = pack_bf16(p0 * fmaf(__uint_as_float(d[i]), p.scale, m.x),
                                    p1 * fmaf(__uint_as_float(d[i + 1]), p.scale, m.y)) & keep;
              ds[i / 2 + 1] = pack_bf16(p2 * fmaf(__uint_as_float(d[i + 2]), p.scale, m.z),
                                        p3 * fmaf(__uint_as_float(d[i + 3]), p.scale, m.w)) & keep;
            }
            // Straight from the lanes' own rows, a sector a store.  Turned in shared memory to 64-byte pieces the
            // stores are as fast, but the 16 KB that takes are a ring stage (1274 us for 2048 tokens, against 1159 so);
            // staged for TMA they were slower, and 16 bytes a store took 1466 in an earlier form against 1252.
            if (slot0 < p.kp) {
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                st_global_32(out + 32 * c + 16 * i, ds + 8 * i);
                st_global_32(out + p.HP + 32 * c + 16 * i, ps + 8 * i);
              }
            }
          }
        }
      }
      g += sp.j1 - sp.j0;
      if (!(ok = named_bar_all(1, 256, ok))) break;
      if constexpr (KL) {
        // the token's sums over the pair's 512 threads, then g (softmax(I) - p) for each slot
        float mm = m_i;
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
        float* rs = hs + 128;              // [8 warps][max, sum of exp, sum of a]
        float z = m_i == -INFINITY ? z_i : z_i * ex2_approx((m_i - mm) * kLog2e);      // (then 0 or NaN)
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          z += __shfl_xor_sync(0xffffffffu, z, d);
          s_a += __shfl_xor_sync(0xffffffffu, s_a, d);
        }
        const int wi = 4 * grp + quad;
        if (lane == 0) { rs[3 * wi] = mm; rs[3 * wi + 1] = z; rs[3 * wi + 2] = s_a; }
        named_bar_sync(1, 256);
        auto join = [&](float& ma, float& za, float mb, float zb) {
          const float mx = fmaxf(ma, mb);
          const float fa = ma > -INFINITY ? ex2_approx((ma - mx) * kLog2e) : 0.f;
          const float fb = mb > -INFINITY ? ex2_approx((mb - mx) * kLog2e) : 0.f;
          za = za * fa + zb * fb;
          ma = mx;
        };
        float m_all = rs[0], z_all = rs[1], a_all = rs[2];
#pragma unroll
        for (int w = 1; w < 8; ++w) {
          join(m_all, z_all, rs[3 * w], rs[3 * w + 1]);
          a_all += rs[3 * w + 2];
        }
        // the other CTA's sums (buffer n & 1: it cannot be two tokens ahead, as it needs this CTA's sums of each)
        const int sb = n & 1;
        if (row == 0 && grp == 0) {
          mbar_arrive_expect_tx(cta.bar(B_SUMS + sb), 16);
          st_async_v4(map_cluster(sbase + OFF_SUMS + 16 * sb, rank ^ 1),
                      make_uint4(__float_as_uint(m_all), __float_as_uint(z_all), __float_as_uint(a_all), 0),
                      map_cluster(cta.bar(B_SUMS + sb), rank ^ 1));
        }
        ok = warp_wait<true>(cta.bar(B_SUMS + sb), (n >> 1) & 1, abort_flag);
        if (!(ok = named_bar_all(1, 256, ok))) break;
        const float4 other = *reinterpret_cast<const float4*>(cta.smem + OFF_SUMS + 16 * sb);
        if (rank == 0) {                   // both CTAs join the two halves in the same order
          join(m_all, z_all, other.x, other.y);
          a_all = a_all + other.z;
        } else {
          float mo = other.x, zo = other.y;
          join(mo, zo, m_all, z_all);
          m_all = mo;
          z_all = zo;
          a_all = other.z + a_all;
        }
        const float up = p.dkl ? p.dkl[t] : 1.f;
        // (divisions, not products with reciprocals: a token with one entry has both exactly 1, and a gradient of 0)
        const float z_div = z_all == 0.f ? INFINITY : z_all, a_div = a_all > 0.f ? a_all : INFINITY;
        for (int i = (2 * grp + rank) * NK + row; i < min(sp.j1 * 2 * NK, p.k); i += 4 * NK) {
          const int e = __ldg(p.idx + base + i);
          const float x = p.sel[base + i];
          const float soft = (x == -INFINITY ? 0.f : ex2_approx((x - m_all) * kLog2e)) / z_div;
          p.dsel[base + i] = (e >= 0 && e < p.S) ? up * (soft - __ldcg(p.dsel + base + i) / a_div) : 0.f;
        }
      }
      ++n;
    }
  }
  bwd_end<true>(cta);
}

// Contributions to dc: contrib[t kp + slot][d] = sum_h dS q[t][h][d] + P dout[t][h][d], one (token, 256 dims) per CTA
// pair and item, the 64 position dims (dS q alone) as a third item.
//
// M = 256 keys (128 in each CTA), N = 256 dims (128 of q and dout in each CTA, resident), K = heads of dS, then of P.
// As single CTAs with N = 192 each MMA read 10 KB of shared memory in 96 cycles, and a token's dS and P three times:
// 1426 us for 2048 tokens, against 1407.  HBM: the contributions (2.3 MB a token) written, P and dS (1 MB) read.
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(mbw::dc::THREADS, 1)
mla_bwd_dc_kernel(const __grid_constant__ CUtensorMap tm_pds, const __grid_constant__ CUtensorMap tm_q,
                  const __grid_constant__ CUtensorMap tm_do, const __grid_constant__ CUtensorMap tm_out,
                  const MlaBwdParams p) {
  using namespace mbw;
  using namespace mbw::dc;
  extern __shared__ uint8_t smem_raw[];
  BwdCta cta = bwd_base(smem_raw);
  const uint32_t sbase = cta.sbase;
  volatile int* abort_flag = cta.abort_flag;
  const int warp = warp_id(), lane = lane_id();
  const int rank = static_cast<int>(cluster_rank());
  if (threadIdx.x == 0) {
    for (int i = 0; i < NU; ++i) { mbar_init(cta.bar(B_RES_FULL + i), 2); mbar_init(cta.bar(B_RES_EMPTY + i), 1); }
    for (int i = 0; i < NS; ++i) { mbar_init(cta.bar(B_RING_FULL + i), 2); mbar_init(cta.bar(B_RING_EMPTY + i), 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(cta.bar(B_ACC_FULL + i), 1); mbar_init(cta.bar(B_ACC_EMPTY + i), 8); }
  }
  bwd_begin<true>(cta);
  const uint32_t tmem = cta.tmem;
  const uint32_t res = sbase + OFF_RES, ring = sbase + OFF_RING;
  const uint32_t lead = map_cluster(sbase, 0);     // CTA 0's barriers, where every load of the pair completes
  const int first = static_cast<int>(blockIdx.x >> 1), stride = static_cast<int>(gridDim.x >> 1);
  const int hb = p.HP / 64;                        // 64-head blocks
  const int items = 3 * p.T * p.splits;
  auto part = [&](int item, int& t, int& d3) {     // item: (token, split, 256 or 64 dims)
    d3 = item % 3;
    const int ts = item / 3;
    t = p.splits == 1 ? ts : ts / p.splits;
    return tile_span(p.n_end[t], 2 * NK, p.splits == 1 ? 0 : ts % p.splits, p.splits);
  };
  bool ok = true;
  int n = 0;

  if (warp == 0) {
    // ===================================================================== resident q and dout
    for (int item = first; item < items && ok; item += stride) {
      int t, d3;
      const TileSpan sp = part(item, t, d3);
      if (sp.j0 >= sp.j1) continue;
      const int units = d3 == 2 ? hb : 2 * hb, boxes = d3 == 2 ? 1 : 2;
      // (CTA 1's columns of the third item lie behind dim 576: zeros)
      const int d0 = d3 == 2 ? 512 + 64 * rank : 256 * d3 + 128 * rank;
      for (int u = 0; u < units; ++u) {            // a box of 64 dims a lane
        const uint32_t full = lead + 8 * (B_RES_FULL + u);
        if (!(ok = warp_wait(cta.bar(B_RES_EMPTY + u), (n & 1) ^ 1, abort_flag))) break;
        if (lane == 0) mbar_arrive_expect_tx_remote(full, boxes * HCHUNK);
        __syncwarp();
        if (lane < boxes)
          tma2_load_3d(res + u * UNIT + lane * HCHUNK, u < hb ? &tm_q : &tm_do, full, d0 + 64 * lane, 64 * (u % hb),
                       p.t0 + t);
      }
      // the third item leaves dout's units alone: their phase goes on without a load
      if (d3 == 2)
        for (int u = units; u < 2 * hb && ok; ++u) {
          ok = warp_wait(cta.bar(B_RES_EMPTY + u), (n & 1) ^ 1, abort_flag);
          if (ok && lane == 0) mbar_arrive_remote(lead + 8 * (B_RES_FULL + u));
        }
      ++n;
    }
  } else if (warp == 2) {
    // ===================================================================== dS and P tiles
    if (lane == 0) {
      Pipe<NS> rp;
      for (int item = first; item < items && ok; item += stride) {
        int t, d3;
        const TileSpan sp = part(item, t, d3);
        const int n_end = p.n_end[t];
        for (int j = sp.j0; j < sp.j1 && ok; ++j) {
          const bool any = (2 * j + rank) * NK < n_end;            // this CTA has keys in the tile
          for (int u = 0; u < (d3 == 2 ? 1 : 2); ++u, rp.advance()) {
            if (!(ok = mbar_wait(cta.bar(B_RING_EMPTY + rp.stage), rp.phase ^ 1, abort_flag))) break;
            const uint32_t full = lead + 8 * (B_RING_FULL + rp.stage);
            if (!any) {
              mbar_arrive_remote(full);
              continue;
            }
            mbar_arrive_expect_tx_remote(full, hb * CHUNK);
            for (int i = 0; i < hb; ++i)
              tma2_load_2d(ring + (2 * rp.stage + i) * CHUNK, &tm_pds, full, 64 * (u * hb + i),
                           t * p.kp + (2 * j + rank) * NK);
          }
        }
      }
    }
  } else if (warp == 1) {
    // ===================================================================== MMA issue (CTA 0 for the pair)
    if (rank == 0) {
      Pipe<NS> rp;
      int g = 0;
      for (int item = first; item < items && ok; item += stride) {
        int t, d3;
        const TileSpan sp = part(item, t, d3);
        if (sp.j0 >= sp.j1) continue;
        const uint32_t idesc = idesc_bf16(256, d3 == 2 ? 128 : 256, true);
        for (int j = sp.j0; j < sp.j1 && ok; ++j, ++g) {
          const int ab = g & 1;
          const bool last = j == sp.j1 - 1;
          if (!(ok = warp_wait<true>(cta.bar(B_ACC_EMPTY + ab), ((g >> 1) & 1) ^ 1, abort_flag))) break;
          tc_fence_after();
          for (int half = 0; half < 2; ++half) {   // dS . q, then P . dout
            if (j == sp.j0)
              for (int i = 0; i < hb && ok; ++i)
                ok = warp_wait<true>(cta.bar(B_RES_FULL + half * hb + i), n & 1, abort_flag);
            if (!ok) break;
            if (half && d3 == 2) {
              if (last && elect_one())
                for (int i = 0; i < hb; ++i) mma2_commit(cta.bar(B_RES_EMPTY + hb + i));
              __syncwarp();
              continue;
            }
            if (!(ok = warp_wait<true>(cta.bar(B_RING_FULL + rp.stage), rp.phase, abort_flag))) break;
            tc_fence_after();
            const uint64_t ad = smem_desc(ring + 2 * rp.stage * CHUNK, 16, 1024, kLayoutSW128);
            // heads x dims, dims contiguous (MN-major): 64-dim atoms 8 KB apart, 8-head groups 1 KB apart
            const uint64_t bd = smem_desc(res + half * hb * UNIT, HCHUNK, 1024, kLayoutSW128);
            if (elect_one()) {
              for (int i = 0; i < hb; ++i) {
#pragma unroll
                for (int k = 0; k < 4; ++k)
                  mma2_bf16_ss(tmem + 256 * ab, ad + ((i * CHUNK) >> 4) + 2 * k, bd + ((i * UNIT + k * 2048) >> 4),
                               idesc, (half | i | k) ? 1u : 0u);
                if (last) mma2_commit(cta.bar(B_RES_EMPTY + half * hb + i));
              }
              mma2_commit(cta.bar(B_RING_EMPTY + rp.stage));
            }
            __syncwarp();
            rp.advance();
          }
          if (!ok) break;
          if (elect_one()) mma2_commit(cta.bar(B_ACC_FULL + ab));
          __syncwarp();
        }
        ++n;
      }
    }
  } else if (warp >= 4) {
    // ===================================================================== contributions out (one key a thread)
    // two groups of four warps take tiles in turn, each with an accumulator of its own
    const int grp = (warp - 4) >> 2;
    const int quad = warp & 3;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    int g = 0, put = 0;
    for (int item = first; item < items && ok; item += stride) {
      int t, d3;
      const TileSpan sp = part(item, t, d3);
      const int n_end = p.n_end[t], blocks = d3 == 2 ? 1 : 4;
      for (int j = sp.j0 + ((g ^ grp) & 1); j < sp.j1; j += 2) {
        const int ab = grp;                // tile j is the CTA's tile g + j - j0, of this group's parity
        const int slot0 = (2 * j + rank) * NK + quad * 32;
        if (!(ok = warp_wait(cta.bar(B_ACC_FULL + ab), ((g + j - sp.j0) >> 1) & 1, abort_flag))) break;
        tc_fence_after();
        const bool any = slot0 < n_end;    // the warp's keys are not all behind the token's last entry
#pragma unroll 1
        for (int c = 0; c < blocks; ++c) {
          uint32_t v[64], w[32];
          tmem_ld32(lane_addr + tmem + 256 * ab + 64 * c, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_ld32(lane_addr + tmem + 256 * ab + 64 * c + 32, *reinterpret_cast<uint32_t(*)[32]>(&v[32]));
          tmem_wait_ld();
          if (c == blocks - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(lead + 8 * (B_ACC_EMPTY + ab));
          }
          if (!any) continue;
          scatter_pack64(v, w);
          // the warp's 32 rows of 64 dims (128-byte swizzled: 16-byte unit u of row r at unit u ^ (r % 8)) go out by
          // TMA, the previous piece's area being read meanwhile
          const int area = OFF_OUT + ((2 * (4 * grp + quad)) + (put & 1)) * 4096;
          if (lane == 0) bulk_wait_read<1>();
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(cta.smem + area + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_out, sbase + area, 256 * d3 + 64 * c, t * p.kp + slot0);
            bulk_commit();
          }
          __syncwarp();                      // the warp's next load of tensor memory wants all its lanes
          ++put;
        }
      }
      g += sp.j1 - sp.j0;
    }
    if (lane == 0) bulk_wait_all();
  }
  bwd_end<true>(cta);
}

// dq[t][:, 192 dims] = dS^T . C per item, accumulated over the token's keys (or, with splits, over the split's) in
// tensor memory (lane = head).
__global__ void __launch_bounds__(mbw::dq::THREADS, 1)
mla_bwd_dq_kernel(const __grid_constant__ CUtensorMap tm_ds, const MlaBwdParams p) {
  using namespace mbw;
  using namespace mbw::dq;
  extern __shared__ uint8_t smem_raw[];
  BwdCta cta = bwd_base(smem_raw);
  const uint32_t sbase = cta.sbase;
  volatile int* abort_flag = cta.abort_flag;
  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(cta.bar(B_ACC_FULL + i), 1);
      mbar_init(cta.bar(B_ACC_EMPTY + i), 4);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(cta.bar(B_RING_FULL + i), 128 + 1);
      mbar_init(cta.bar(B_RING_EMPTY + i), 1);
    }
  }
  bwd_begin(cta);
  const uint32_t tmem = cta.tmem;
  const uint32_t ring = sbase + OFF_RING;
  const int items = 3 * p.T * p.splits;
  auto part = [&](int item, int& ts, int& d3) {        // item: (token, split, 192 dims)
    d3 = item % 3;
    ts = item / 3;
    return p.splits == 1 ? tile_span(p.n_end[ts], KT, 0, 1)
                         : tile_span(p.n_end[ts / p.splits], KT, ts % p.splits, p.splits);
  };
  auto token = [&](int ts) { return p.splits == 1 ? ts : ts / p.splits; };
  bool ok = true;
  int n = 0;

  if (warp == 0) {
    // ===================================================================== dS tiles
    if (lane == 0) {
      Pipe<NS> rp;
      int issued = 0;
      for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
        int ts, d3;
        const TileSpan sp = part(item, ts, d3);
        const int t = token(ts);
        for (int j = sp.j0; j < sp.j1; ++j, rp.advance(), ++issued) {
          if (!(ok = lean_wait(cta.bar(B_RING_EMPTY + rp.stage), rp.phase ^ 1, abort_flag))) break;
          const uint32_t full = cta.bar(B_RING_FULL + rp.stage), dst = ring + rp.stage * STAGE;
          mbar_arrive_expect_tx(full, A_BYTES);
          for (int i = 0; i < 2; ++i)      // HP = 64: the second block is P's columns, its products are not stored
            tma_load_2d(dst + i * HCHUNK, &tm_ds, full, 64 * i, t * p.kp + j * KT);
        }
      }
      if (*abort_flag)
        for (int i = max(0, issued - NS); i < issued; ++i)
          mbar_wait_drain(cta.bar(B_RING_FULL + i % NS), (i / NS) & 1);
    }
  } else if (warp == 2 || warp == 3 || warp >= 8) {
    // ===================================================================== gathers (cp.async)
    // Stages of 64 keys x 192 dims go round two groups of four warps, 16 keys a warp; eight lanes copy 128 bytes of a
    // row.  (TMA's gather4, whose warp issues one of four rows about every 50 ns: 1006 us against 860 for 2048 tokens.)
    // An empty slot's row is filled with zeros: a NaN in a row that no token selects must not meet its dS = 0.
    const int gw = (warp < 8) ? warp - 2 : warp - 6;
    const int grp = gw >> 2, rows = (gw & 3) * 16, sub = lane >> 3, unit = lane & 7;
    static_assert(2 <= NS, "stages (as in mla_bwd_p_kernel)");
    int m = 0;                             // stages of the items before this one
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      int ts, d3;
      const TileSpan sp = part(item, ts, d3);
      const int* ids = p.idx + static_cast<long long>(token(ts)) * p.k;
      // k is a multiple of the tile: every slot of a tile is below k
      auto entry = [&](int j) { return j < sp.j1 ? __ldg(ids + j * KT + rows + (lane & 15)) : -1; };
      const int j0 = sp.j0 + ((grp + m) & 1);            // tile j is the CTA's stage m + j - j0
      int mine = entry(j0);
      for (int j = j0; j < sp.j1; j += 2) {
        const int at = m + j - sp.j0, st = at % NS;
        const int next = entry(j + 2);
        if (!(ok = lean_warp_wait(cta.bar(B_RING_EMPTY + st), ((at / NS) & 1) ^ 1, abort_flag))) break;
        const uint32_t dst = ring + st * STAGE + A_BYTES + (rows + sub) * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = __shfl_sync(0xffffffffu, mine, 4 * i + sub);
          const bool valid = e >= 0 && e < p.S;
          const char* src = reinterpret_cast<const char*>(p.c) + (valid ? static_cast<long long>(e) * (D * 2) : 0) +
                            384 * d3 + 16 * unit;
          const uint32_t to = dst + i * 512 + ((unit ^ ((4 * i + sub) & 7)) << 4);
#pragma unroll
          for (int c = 0; c < 3; ++c) cp_async16(to + c * HCHUNK, src + 128 * c, valid);
        }
        cp_async_arrive(cta.bar(B_RING_FULL + st));
        mine = next;
      }
      m += sp.j1 - sp.j0;
    }
    cp_async_wait_all();
  } else if (warp == 1) {
    // ===================================================================== MMA issue
    Pipe<NS> rp;
    constexpr uint32_t idesc = idesc_bf16_major(128, 192, true, true);
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      int ts, d3;
      const TileSpan sp = part(item, ts, d3);
      if (sp.j0 >= sp.j1) continue;
      const int ab = n & 1;
      if (!(ok = lean_warp_wait(cta.bar(B_ACC_EMPTY + ab), ((n >> 1) & 1) ^ 1, abort_flag))) break;
      tc_fence_after();
      for (int j = sp.j0; j < sp.j1; ++j, rp.advance()) {
        if (!(ok = lean_warp_wait(cta.bar(B_RING_FULL + rp.stage), rp.phase, abort_flag))) break;
        fence_proxy_async_smem();            // the gathered keys were written through the generic proxy
        tc_fence_after();
        const uint32_t at = ring + rp.stage * STAGE;
        const uint64_t ad = smem_desc(at, HCHUNK, 1024, kLayoutSW128);
        const uint64_t bd = smem_desc(at + A_BYTES, HCHUNK, 1024, kLayoutSW128);
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k)
            mma_bf16_ss(tmem + 256 * ab, ad + ((k * 2048) >> 4), bd + ((k * 2048) >> 4), idesc,
                        (j > sp.j0 || k) ? 1u : 0u);
          mma_commit(cta.bar(B_RING_EMPTY + rp.stage));
        }
        __syncwarp();
      }
      if (!ok) break;
      if (elect_one()) mma_commit(cta.bar(B_ACC_FULL + ab));
      __syncwarp();
      ++n;
    }
  } else {
    // ===================================================================== dq out (one head a thread)
    const int quad = warp & 3, h = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      int ts, d3;
      const TileSpan sp = part(item, ts, d3);
      const long long at = (static_cast<long long>(ts) * p.H + h) * D + 192 * d3;
      if (sp.j0 >= sp.j1) {                // nothing selected: dq = 0 (an empty split is not read)
        if (h < p.H && p.splits == 1)
          for (int i = 0; i < 24; ++i) reinterpret_cast<uint4*>(p.dq + at)[i] = make_uint4(0, 0, 0, 0);
        continue;
      }
      const int ab = n & 1;
      if (!(ok = lean_warp_wait(cta.bar(B_ACC_FULL + ab), (n >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      for (int c = 0; c < 6; ++c) {
        uint32_t v[32];
        tmem_ld32(lane_addr + tmem + 256 * ab + 32 * c, v);
        tmem_wait_ld();
        if (h >= p.H) {
          // a head that only fills up the tile: nothing to store
        } else if (p.splits == 1) {
          uint4* dst = reinterpret_cast<uint4*>(p.dq + at + 32 * c);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            auto pk = [&](int q) {
              return pack_bf16(__uint_as_float(v[8 * i + 2 * q]), __uint_as_float(v[8 * i + 2 * q + 1]));
            };
            dst[i] = make_uint4(pk(0), pk(1), pk(2), pk(3));
          }
        } else {
          uint4* dst = reinterpret_cast<uint4*>(p.dq_part + at + 32 * c);
#pragma unroll
          for (int i = 0; i < 8; ++i) dst[i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        __syncwarp();                        // the warp's next load of tensor memory wants all its lanes
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(cta.bar(B_ACC_EMPTY + ab));
      ++n;
    }
  }
  bwd_end(cta);
}

// The splits' sums of a token joined in order: out[t][i] = sum over its splits of part[t splits + sp][i], i < width
// (bf16), and the last `tail` values of a part (fp32 results).  width and tail are multiples of 4.
__global__ void __launch_bounds__(256) join_splits_kernel(const float* part, const int* n_end, int keys, int splits,
                                                          int width, int tail, uint16_t* out, float* out_tail) {
  pdl_allow_next();
  pdl_wait();
  const int t = blockIdx.y, i = 4 * (blockIdx.x * 256 + threadIdx.x);
  if (i >= width + tail) return;
  const int tiles = (n_end[t] + keys - 1) / keys, per = (tiles + splits - 1) / splits;
  const int used = tiles > 0 ? (tiles + per - 1) / per : 0;
  const float* at = part + static_cast<long long>(t) * splits * (width + tail) + i;
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int sp = 0; sp < used; ++sp, at += width + tail) {
    const float4 v = *reinterpret_cast<const float4*>(at);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  if (i < width)
    *reinterpret_cast<uint2*>(out + static_cast<long long>(t) * width + i) =
        make_uint2(pack_bf16(s.x, s.y), pack_bf16(s.z, s.w));
  else {
    float* to = out_tail + static_cast<long long>(t) * tail + i - width;   // a caller's array: aligned to its type only
    to[0] = s.x; to[1] = s.y; to[2] = s.z; to[3] = s.w;
  }
}

// What the other kernels of a chunk start from: delta[t][h] = dout . out over the 512 value dims (one warp a row, eight
// rows a block) and the scatter table, cleared in equal shares by all blocks.
__global__ void __launch_bounds__(256) mla_bwd_begin_kernel(const uint16_t* dout, const uint16_t* out, long long rows,
                                                            float* delta, uint4* table, long long n) {
  pdl_allow_next();
  pdl_wait();
  const long long r = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  if (r < rows) {
    const uint4* a = reinterpret_cast<const uint4*>(dout + r * mbw::DV);
    const uint4* b = reinterpret_cast<const uint4*>(out + r * mbw::DV);
    uint4 x[2], y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[i] = __ldcs(a + lane_id() + 32 * i);
      y[i] = __ldcs(b + lane_id() + 32 * i);
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        s = fmaf(__uint_as_float(xs[u] << 16), __uint_as_float(ys[u] << 16), s);
        s = fmaf(__uint_as_float(xs[u] & 0xffff0000u), __uint_as_float(ys[u] & 0xffff0000u), s);
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    if (lane_id() == 0) delta[r] = s;
  }
  scatter_clear(table, n);
}

}  // namespace dsa
