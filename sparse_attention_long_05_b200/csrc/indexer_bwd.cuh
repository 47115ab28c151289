// Backward pass of the lightning-indexer scores (indexer.cuh) at the selected entries.
//
// I[t,i] = sum_j w_j relu(q_j . k_s), s = idx[t][i], q_j = qs_t q_idx[t][j] and k_s = ks_s k_idx[s] the dequantised
// operands.  With the gradient e = dsel[t][i], x = q_idx[t][j] . k_idx[s] and the live pairs 1[x > 0]:
//   dw_j = qs sum_i e ks relu(x)     dq_j = sum_i (G ks) k_idx[s]     dk_s = sum_(t,i) sum_j (G qs) q_idx[j]
// with G = e w_j 1[x > 0]: three products of 2 x 64 heads x 128 dims per entry (G qs and G ks are what is stored).  dq
// and dk are gradients of the dequantised values (what a straight-through quantiser passes on).
//
// One CTA per token (or per split of a token's tiles, where tokens are few), keys are the M dimension.  e4m3 rows are
// gathered with plain 16-byte loads and written as bf16 (exact) in the swizzled form the tensor core reads, so the one
// copy serves x (K-major), dq (transposed, MN-major) and, for q, dk; kind::f16 needs both operands bf16 and G is.
// Products of e4m3 are exact and their sum is held in fp32: it is exact for small integers, else off by less than 2^-15
// of sum |q k| (eight instructions that each add 17 terms, aligned to the largest and cut at 24 bits or more: 8 x 17 x
// 2^-23).  Closer to 0 than that the sign, which decides what is live, may be another than the exact one, as in the
// forward's sum; the jump of the gradient at x = 0 is as large on either side.  G qs and G ks are rounded to bf16 once
// (by 2^-8 at most).  dw is summed from the fp32 x.  Per token: 16 tiles of 128 keys, each x -> G -> (dk, dq); x of the
// next tile is issued before G of this one is waited for.
// HBM sees each entry's contribution to dk twice (written here, summed by scatter.cuh).
// Measured on 2048 tokens of a 32K sequence, k = 2048, 64 heads: 533 us here, 219 for the sums, 115 for the table;
// bound by the latency of G's chain (x from tensor memory -> G to shared memory) and by the issue slots its warps
// share.  The small indexer (4 heads, 64 dims) runs in the same layout, its missing heads and dims zero.
#pragma once
#include "common.cuh"
#include "sparse_mla_bwd.cuh"

namespace dsa {

struct IndexerBwdParams {
  const uint8_t* q_idx;        // [T, HI, DI] e4m3
  const float* q_scale;        // [T] or null
  const uint8_t* k_idx;        // [S, DI] e4m3
  const float* k_scale;        // [S] or null
  const float* w;              // [T, HI]
  const int* idx;              // [T, k]
  const float* dsel;           // [T, k]
  const int* n_end;            // [T]
  uint16_t* dq;                // [T, HI, DI] bf16
  float* dw;                   // [T, HI]
  float* part;                 // splits > 1: [T * splits, HI * DI + HI] dq and dw of each split
  int T, k, kp, splits;        // a token's tiles are dealt to `splits` items
  long long S;
};

namespace ixb {
// w0 index rows, w1 MMA, w2 w3 w8..13 keys, w4..7 w18..21 G, w14..17 results
constexpr int THREADS = 704, PRODUCERS = 8;
constexpr int NK = 128, HP = 64;
constexpr int KCH = 128 * 128, QCH = 64 * 128;   // 128 keys (64 heads) x 64 dims bf16
constexpr int K_BYTES = 2 * KCH, Q_BYTES = 2 * QCH, G_BYTES = 128 * 128;
constexpr int B_IDX_FULL = 0, B_IDX_EMPTY = 2, B_Q_FULL = 4, B_Q_EMPTY = 6, B_K_FULL = 8, B_K_EMPTY = 10;
constexpr int B_X_FULL = 12, B_X_EMPTY = 14, B_G_FULL = 16, B_G_EMPTY = 18, B_DK_FULL = 20, B_DK_EMPTY = 22;
constexpr int B_DQ_FULL = 24, B_DQ_EMPTY = 26;
constexpr int OFF_W = 1024, OFF_DW = OFF_W + 512;            // w of the token (2 buffers), dw of the eight warps
constexpr int OFF_IDX = 4096, OFF_Q = OFF_IDX + 2 * mla::KMAX * 4, OFF_K = OFF_Q + 2 * Q_BYTES;
constexpr int OFF_G = OFF_K + 2 * K_BYTES;                   // 2 x (G qs, G ks)
constexpr int OFF_OUT = OFF_G + 4 * G_BYTES;
constexpr int SMEM = OFF_OUT + 2 * KCH + 1024;
constexpr uint32_t TX = 0, TDK = 128, TDQ = 384;             // x 2 x 64, dk 2 x 128, dq 2 x 64 columns
static_assert(SMEM <= 232448 && OFF_DW + 2048 <= OFF_IDX, "shared memory");
}  // namespace ixb

// two e4m3 -> two bf16 (exact)
__device__ __forceinline__ uint32_t e4m3x2_to_bf16x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  float lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
      : "=f"(lo), "=f"(hi) : "r"(h));
  return pack_bf16(lo, hi);
}
// 16 e4m3 (dims 16 u .. 16 u + 15 of a row) into a swizzled bf16 tile of 64-dim chunks `chunk` bytes apart
__device__ __forceinline__ void put_e4m3_row16(uint8_t* tile, int chunk, int row, int u, uint4 v) {
  const uint32_t x[4] = {v.x, v.y, v.z, v.w};
  uint32_t y[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    y[2 * i] = e4m3x2_to_bf16x2(x[i] & 0xffff);
    y[2 * i + 1] = e4m3x2_to_bf16x2(x[i] >> 16);
  }
  uint8_t* line = tile + (u >> 2) * chunk + row * 128;
  const int unit = 2 * (u & 3);
  *reinterpret_cast<uint4*>(line + ((unit ^ (row & 7)) << 4)) = make_uint4(y[0], y[1], y[2], y[3]);
  *reinterpret_cast<uint4*>(line + (((unit + 1) ^ (row & 7)) << 4)) = make_uint4(y[4], y[5], y[6], y[7]);
}

template <int HI, int DI>
__global__ void __launch_bounds__(ixb::THREADS, 1)
indexer_bwd_kernel(const __grid_constant__ CUtensorMap tm_out, const IndexerBwdParams p) {
  using namespace ixb;
  extern __shared__ uint8_t smem_raw[];
  BwdCta cta = bwd_base(smem_raw);
  const uint32_t sbase = cta.sbase;
  volatile int* abort_flag = cta.abort_flag;
  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(cta.bar(B_IDX_FULL + i), 1);
      mbar_init(cta.bar(B_IDX_EMPTY + i), PRODUCERS);
      mbar_init(cta.bar(B_Q_FULL + i), PRODUCERS);
      mbar_init(cta.bar(B_Q_EMPTY + i), 1);
      mbar_init(cta.bar(B_K_FULL + i), PRODUCERS);
      mbar_init(cta.bar(B_K_EMPTY + i), 1);
      mbar_init(cta.bar(B_X_FULL + i), 1);
      mbar_init(cta.bar(B_X_EMPTY + i), 4);
      mbar_init(cta.bar(B_G_FULL + i), 4);
      mbar_init(cta.bar(B_G_EMPTY + i), 1);
      mbar_init(cta.bar(B_DK_FULL + i), 1);
      mbar_init(cta.bar(B_DK_EMPTY + i), 4);
      mbar_init(cta.bar(B_DQ_FULL + i), 1);
      mbar_init(cta.bar(B_DQ_EMPTY + i), 4);
    }
  }
  if constexpr (HI < HP || DI < 128) {
    // the heads and dims that are never written stay zero
    for (int i = threadIdx.x; i < (2 * Q_BYTES + 2 * K_BYTES + 4 * G_BYTES) / 16; i += THREADS)
      reinterpret_cast<uint4*>(cta.smem + OFF_Q)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
  }
  bwd_begin(cta);
  const uint32_t tmem = cta.tmem;
  bool ok = true;
  int n = 0;                             // items with tiles, walked so far
  const int items = p.T * p.splits;
  auto token = [&](int item) { return p.splits == 1 ? item : item / p.splits; };
  auto span = [&](int item) {
    return tile_span(p.n_end[token(item)], NK, p.splits == 1 ? 0 : item % p.splits, p.splits);
  };

  if (warp == 0) {
    // ===================================================================== index rows
    if (lane == 0) {
      for (int item = blockIdx.x; item < items; item += gridDim.x) {
        const TileSpan sp = span(item);
        if (sp.j0 >= sp.j1) continue;
        const int t = token(item);
        const int ib = n & 1;
        if (!(ok = lean_wait(cta.bar(B_IDX_EMPTY + ib), ((n >> 1) & 1) ^ 1, abort_flag))) break;
        mbar_arrive_expect_tx(cta.bar(B_IDX_FULL + ib), p.k * 4);
        bulk_load(sbase + OFF_IDX + ib * mla::KMAX * 4, p.idx + static_cast<long long>(t) * p.k, p.k * 4,
                  cta.bar(B_IDX_FULL + ib));
        ++n;
      }
      if (*abort_flag)
        for (int i = max(0, n - 2); i < n; ++i) mbar_wait_drain(cta.bar(B_IDX_FULL + (i & 1)), (i >> 1) & 1);
    }
  } else if (warp == 2 || warp == 3 || (warp >= 8 && warp < 14)) {
    // ===================================================================== keys and queries to bf16 tiles
    const int pw = (warp < 8) ? warp - 2 : warp - 6;
    constexpr int U = DI / 16;                    // 16-byte units of a row
    constexpr int ROWS = 32 / U;                  // rows a warp reads at once
    constexpr int STEPS = NK / PRODUCERS / ROWS;  // 4 (DI = 128), 2 (64)
    const int sub = lane / U, u = lane % U;
    int g = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const TileSpan sp = span(item);
      if (sp.j0 >= sp.j1) continue;
      const int t = token(item);
      const int ib = n & 1;
      if (!(ok = lean_warp_wait(cta.bar(B_IDX_FULL + ib), (n >> 1) & 1, abort_flag))) break;
      const int* ids = reinterpret_cast<const int*>(cta.smem + OFF_IDX + ib * mla::KMAX * 4);
      // the rows of the next tile are read while this one waits for its buffer; an empty slot's row is zero
      auto load = [&](int j, uint4 (&v)[STEPS]) {
#pragma unroll
        for (int s = 0; s < STEPS; ++s) {
          const int slot = j * NK + pw * (NK / PRODUCERS) + s * ROWS + sub;
          const int e = slot < p.k ? ids[slot] : -1;
          v[s] = make_uint4(0, 0, 0, 0);
          if (e >= 0 && e < p.S)
            v[s] = __ldg(reinterpret_cast<const uint4*>(p.k_idx + static_cast<long long>(e) * DI) + u);
        }
      };
      uint4 v[STEPS];
      load(sp.j0, v);
      if (!(ok = lean_warp_wait(cta.bar(B_Q_EMPTY + ib), ((n >> 1) & 1) ^ 1, abort_flag))) break;
      const uint4* qrow = reinterpret_cast<const uint4*>(p.q_idx + static_cast<long long>(t) * HI * DI);
      for (int i = pw * 32 + lane; i < HI * U; i += PRODUCERS * 32)
        put_e4m3_row16(cta.smem + OFF_Q + ib * Q_BYTES, QCH, i / U, i % U, __ldg(qrow + i));
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(cta.bar(B_Q_FULL + ib));
      for (int j = sp.j0; j < sp.j1; ++j, ++g) {
        const int kb = g & 1;
        uint4 next[STEPS];
        if (j + 1 < sp.j1) load(j + 1, next);
        if (!(ok = lean_warp_wait(cta.bar(B_K_EMPTY + kb), ((g >> 1) & 1) ^ 1, abort_flag))) break;
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
          put_e4m3_row16(cta.smem + OFF_K + kb * K_BYTES, KCH, pw * (NK / PRODUCERS) + s * ROWS + sub, u, v[s]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(cta.bar(B_K_FULL + kb));
#pragma unroll
        for (int s = 0; s < STEPS; ++s) v[s] = next[s];
      }
      if (lane == 0) mbar_arrive(cta.bar(B_IDX_EMPTY + ib));
      ++n;
    }
  } else if (warp == 1) {
    // ===================================================================== MMA issue
    struct Cursor { int item, j, tiles, n, g; } a{static_cast<int>(blockIdx.x), 0, 0, 0, 0}, b;
    auto seek = [&](Cursor& c) {          // first item at or after c.item with tiles
      for (; c.item < items; c.item += gridDim.x) {
        const TileSpan sp = span(c.item);
        if ((c.tiles = sp.j1 - sp.j0) > 0) break;
      }
    };
    auto step = [&](Cursor& c) {
      ++c.g;
      if (++c.j == c.tiles) { c.j = 0; ++c.n; c.item += gridDim.x; seek(c); }
    };
    seek(a);
    b = a;
    constexpr uint32_t ix = idesc_bf16(128, HP, false), idk = idesc_bf16(128, DI, true);
    constexpr uint32_t idq = idesc_bf16_major(128, HP, true, true);
    auto scores = [&]() -> bool {         // x of cursor a's tile
      const int s = a.g & 1, qb = a.n & 1;
      if (a.j == 0 && !lean_warp_wait(cta.bar(B_Q_FULL + qb), (a.n >> 1) & 1, abort_flag)) return false;
      if (!lean_warp_wait(cta.bar(B_K_FULL + s), (a.g >> 1) & 1, abort_flag)) return false;
      if (!lean_warp_wait(cta.bar(B_X_EMPTY + s), ((a.g >> 1) & 1) ^ 1, abort_flag)) return false;
      tc_fence_after();
      const uint64_t kd = smem_desc(sbase + OFF_K + s * K_BYTES, 16, 1024, kLayoutSW128);
      const uint64_t qd = smem_desc(sbase + OFF_Q + qb * Q_BYTES, 16, 1024, kLayoutSW128);
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < DI / 16; ++i)
          mma_bf16_ss(tmem + TX + 64 * s, kd + (((i >> 2) * KCH) >> 4) + 2 * (i & 3),
                      qd + (((i >> 2) * QCH) >> 4) + 2 * (i & 3), ix, i ? 1u : 0u);
        mma_commit(cta.bar(B_X_FULL + s));
      }
      __syncwarp();
      step(a);
      return true;
    };
    if (a.item < items) ok = scores();
    while (ok && b.item < items) {
      if (a.item < items && !(ok = scores())) break;
      const int s = b.g & 1, qb = b.n & 1;
      if (b.j == 0 && !(ok = lean_warp_wait(cta.bar(B_DQ_EMPTY + qb), ((b.n >> 1) & 1) ^ 1, abort_flag))) break;
      if (!(ok = lean_warp_wait(cta.bar(B_DK_EMPTY + s), ((b.g >> 1) & 1) ^ 1, abort_flag))) break;
      if (!(ok = lean_warp_wait(cta.bar(B_G_FULL + s), (b.g >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      const uint32_t gb = sbase + OFF_G + 2 * s * G_BYTES;
      const uint64_t gd = smem_desc(gb, 16, 1024, kLayoutSW128);                             // keys x heads, K = heads
      const uint64_t qd = smem_desc(sbase + OFF_Q + qb * Q_BYTES, QCH, 1024, kLayoutSW128);  // heads x dims, N = dims
      const uint64_t kd = smem_desc(sbase + OFF_K + s * K_BYTES, KCH, 1024, kLayoutSW128);   // keys x dims, M = dims
      const uint64_t hd = smem_desc(gb + G_BYTES, 8192, 1024, kLayoutSW128);                 // keys x heads, N = heads
      const bool last = b.j == b.tiles - 1;
      if (elect_one()) {
#pragma unroll
        for (int i = 0; i < HP / 16; ++i)
          mma_bf16_ss(tmem + TDK + 128 * s, gd + 2 * i, qd + ((i * 2048) >> 4), idk, i ? 1u : 0u);
        mma_commit(cta.bar(B_DK_FULL + s));
#pragma unroll
        for (int i = 0; i < NK / 16; ++i)
          mma_bf16_ss(tmem + TDQ + 64 * qb, kd + ((i * 2048) >> 4), hd + ((i * 2048) >> 4), idq, (b.j | i) ? 1u : 0u);
        mma_commit(cta.bar(B_K_EMPTY + s));
        mma_commit(cta.bar(B_G_EMPTY + s));
        if (last) {
          mma_commit(cta.bar(B_Q_EMPTY + qb));
          mma_commit(cta.bar(B_DQ_FULL + qb));
        }
      }
      __syncwarp();
      step(b);
    }
  } else if (warp < 8 || warp >= 18) {
    // ===================================================================== G qs, G ks and dw (one key a thread)
    // Two groups of four warps take tiles in turn (one group alone: 707 us for 2048 tokens, against 596).  The entry of
    // a thread's next tile but one, and the gradient and key scale of its next tile, are on their way meanwhile.
    const int grp = warp >= 18 ? 1 : 0;
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    constexpr int BLOCKS = (HI + 15) / 16;               // 16 heads at a time
    float* dw_s = reinterpret_cast<float*>(cta.smem + OFF_DW);
    int g = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const TileSpan sp = span(item);
      const int t = token(item);
      // where dw goes: the token's results, or the split's part
      float* dw_out = p.splits == 1 ? p.dw + static_cast<long long>(t) * HI
                                    : p.part + static_cast<long long>(item) * (HI * DI + HI) + HI * DI;
      if (sp.j0 >= sp.j1) {                              // (an empty split is not read)
        if (p.splits == 1 && grp == 0 && row < HI) dw_out[row] = 0.f;
        continue;
      }
      float* ws = reinterpret_cast<float*>(cta.smem + OFF_W) + 64 * (n & 1);
      if (grp == 0 && row < 64) ws[row] = row < HI ? p.w[static_cast<long long>(t) * HI + row] : 0.f;
      const long long base = static_cast<long long>(t) * p.k;
      const float qs = p.q_scale ? p.q_scale[t] : 1.f;
      auto entry = [&](int j) {
        const int slot = j * NK + row;
        const int id = j < sp.j1 && slot < p.k ? __ldg(p.idx + base + slot) : -1;
        return id < p.S ? id : -1;
      };
      auto grad = [&](int j, int id) { return id >= 0 ? __ldg(p.dsel + base + j * NK + row) : 0.f; };
      auto scale = [&](int id) { return id < 0 ? 0.f : p.k_scale ? __ldg(p.k_scale + id) : 1.f; };
      const int j0 = sp.j0 + ((g ^ grp) & 1);            // tile j is the CTA's tile g + j - j0
      int id = entry(j0), id_next = entry(j0 + 2);
      float e = grad(j0, id), ks = scale(id);
      if (!(ok = named_bar_all(1, 256, ok))) break;
      float dw[BLOCKS] = {};
      for (int j = j0; j < sp.j1; j += 2) {
        const int s = grp, use = (g + j - sp.j0) >> 1;
        const float e_next = grad(j + 2, id_next), ks_next = scale(id_next);
        id_next = entry(j + 4);
        ok = lean_warp_wait(cta.bar(B_X_FULL + s), use & 1, abort_flag);
        ok = ok && lean_warp_wait(cta.bar(B_G_EMPTY + s), (use & 1) ^ 1, abort_flag);
        if (!ok) break;
        tc_fence_after();
        uint8_t* gl = cta.smem + OFF_G + 2 * s * G_BYTES + row * 128;
        const float eks = e * ks, eqs = e * qs;
        // not unrolled (nor are the loops over 64 dims below): the roles' code together has to stay in the instruction
        // cache, fetches from behind it were a sixth of all stalls (680 us for 2048 tokens, against 560)
#pragma unroll 1
        for (int c = 0; c < BLOCKS; ++c) {
          uint32_t v[16];
          tmem_ld16(lane_addr + tmem + TX + 64 * s + 16 * c, v);
          tmem_wait_ld();
          if (c == BLOCKS - 1) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(cta.bar(B_X_EMPTY + s));
          }
          float x[16];
          uint32_t a[8], b[8];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 w4 = *reinterpret_cast<const float4*>(ws + 16 * c + i);
            const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
            float gv[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float xv = __uint_as_float(v[i + q]);
              const bool live = xv > 0.f;
              gv[q] = live ? wv[q] : 0.f;
              x[i + q] = live ? eks * xv : 0.f;
            }
            a[i / 2] = pack_bf16(eqs * gv[0], eqs * gv[1]);
            a[i / 2 + 1] = pack_bf16(eqs * gv[2], eqs * gv[3]);
            b[i / 2] = pack_bf16(eks * gv[0], eks * gv[1]);
            b[i / 2 + 1] = pack_bf16(eks * gv[2], eks * gv[3]);
          }
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int unit = ((2 * c + i) ^ (row & 7)) << 4;
            *reinterpret_cast<uint4*>(gl + unit) = make_uint4(a[4 * i], a[4 * i + 1], a[4 * i + 2], a[4 * i + 3]);
            *reinterpret_cast<uint4*>(gl + G_BYTES + unit) =
                make_uint4(b[4 * i], b[4 * i + 1], b[4 * i + 2], b[4 * i + 3]);
          }
          // sums over the warp's 32 keys: four halving steps, then the two half-warps; lane l has head 16 c + l % 16
#define DSA_IXB_HALVE(O)                                                                \
  {                                                                                     \
    const bool up = (lane & (O)) != 0;                                                  \
    _Pragma("unroll") for (int i = 0; i < (O); ++i) {                                   \
      const float keep = up ? x[(O) + i] : x[i];                                        \
      const float send = up ? x[i] : x[(O) + i];                                        \
      x[i] = keep + __shfl_xor_sync(0xffffffffu, send, (O));                            \
    }                                                                                   \
  }
          DSA_IXB_HALVE(8)
          DSA_IXB_HALVE(4)
          DSA_IXB_HALVE(2)
          DSA_IXB_HALVE(1)
#undef DSA_IXB_HALVE
          const float sum = x[0] + __shfl_xor_sync(0xffffffffu, x[0], 16);
#pragma unroll
          for (int i = 0; i < BLOCKS; ++i) dw[i] += i == c ? sum : 0.f;
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(cta.bar(B_G_FULL + s));
        e = e_next;
        ks = ks_next;
      }
      g += sp.j1 - sp.j0;
      if (lane < 16) {
#pragma unroll
        for (int c = 0; c < BLOCKS; ++c) dw_s[(4 * grp + quad) * 64 + 16 * c + lane] = dw[c];
      }
      if (!(ok = named_bar_all(1, 256, ok))) break;
      if (grp == 0 && row < HI) {
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) sum += dw_s[64 * w + row];
        dw_out[row] = sum * qs;
      }
      // the next token's first barrier comes before anyone writes dw_s again
      ++n;
    }
  } else {
    // ===================================================================== contributions to dk, and dq (w14..17)
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_addr = static_cast<uint32_t>(quad * 32) << 16;
    int g = 0;
    for (int item = blockIdx.x; item < items && ok; item += gridDim.x) {
      const TileSpan sp = span(item);
      const int t = token(item);
      uint16_t* dq = p.dq + static_cast<long long>(t) * HI * DI;
      if (sp.j0 >= sp.j1) {
        if (p.splits > 1) continue;
        for (int i = row; i < HI * DI / 8; i += 128) reinterpret_cast<uint4*>(dq)[i] = make_uint4(0, 0, 0, 0);
        continue;
      }
      for (int j = sp.j0; j < sp.j1; ++j, ++g) {
        const int s = g & 1;
        if (!(ok = lean_warp_wait(cta.bar(B_DK_FULL + s), (g >> 1) & 1, abort_flag))) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < DI / 64; ++c) {
          // each warp stages and stores its own 32 rows, 64 dims at a time
          uint32_t v[64];
          uint32_t (&v0)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[0]);
          uint32_t (&v1)[32] = *reinterpret_cast<uint32_t(*)[32]>(&v[32]);
          tmem_ld32(lane_addr + tmem + TDK + 128 * s + 64 * c, v0);
          tmem_ld32(lane_addr + tmem + TDK + 128 * s + 64 * c + 32, v1);
          if (lane == 0) bulk_wait_read<DI / 64 - 1>();
          __syncwarp();
          tmem_wait_ld();
          if (c == DI / 64 - 1) tc_fence_before();
          __syncwarp();
          if (c == DI / 64 - 1 && lane == 0) mbar_arrive(cta.bar(B_DK_EMPTY + s));
          uint8_t* line = cta.smem + OFF_OUT + c * KCH + row * 128;
          uint32_t w[32];
          scatter_pack64(v, w);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(line + ((i ^ (row & 7)) << 4)) =
                make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tm_out, sbase + OFF_OUT + c * KCH + quad * 32 * 128, 64 * c, t * p.kp + j * NK + quad * 32);
            bulk_commit();
          }
          __syncwarp();                      // the warp's next load of tensor memory wants all its lanes
        }
      }
      if (!ok) break;
      // dq^T: lane = dim, column = head
      const int qb = n & 1;
      if (!(ok = lean_warp_wait(cta.bar(B_DQ_FULL + qb), (n >> 1) & 1, abort_flag))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < (HI + 31) / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(lane_addr + tmem + TDQ + 64 * qb + 32 * c, v);
        tmem_wait_ld();
        if (row < DI && p.splits == 1) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i < HI)
              dq[(32 * c + i) * DI + row] = __bfloat16_as_ushort(__float2bfloat16_rn(__uint_as_float(v[i])));
        } else if (row < DI) {
          float* part = p.part + static_cast<long long>(item) * (HI * DI + HI) + row;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (32 * c + i < HI) part[(32 * c + i) * DI] = __uint_as_float(v[i]);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(cta.bar(B_DQ_EMPTY + qb));
      ++n;
    }
    if (lane == 0) bulk_wait_all();
  }
  bwd_end(cta);
}

}  // namespace dsa
