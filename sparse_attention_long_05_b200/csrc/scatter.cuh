// Sums of per-entry contributions into the rows they belong to: out[s] = sum over tokens t and slots i with
// idx[t][i] = s of contrib[t][i], in a fixed order.
//
// The backward passes write one bf16 row per selected entry (a chunk of tokens at a time).  A table of the chunk,
// slot[s][t] = the slot in which token t selected row s (16 bits, empty: 0xffff), turns the scatter into a gather:
// one CTA per row s lists the row's entries in token order and adds them up.  Every sum has one order whatever the
// kernels' timing, so results repeat bit for bit; with atomics they would not.  Bound by HBM: each contribution is
// read once (2 W bytes), the table once (2 bytes per row and token, 64 rows' worth per selected entry at 128K rows).
#pragma once
#include "common.cuh"

namespace dsa {

namespace sct {
constexpr int MAX_T = 2048;               // tokens of a chunk at most (a row's list sits in shared memory)
constexpr int MAX_K = 2048;               // slots of a token at most: 11 bits of a table entry
constexpr uint16_t EMPTY = 0xffff;
constexpr uint16_t TWICE = 0x0800;        // the token selected the row more than once: see mult
}  // namespace sct

__global__ void __launch_bounds__(256) scatter_clear_kernel(uint4* table, long long n) {
  pdl_allow_next();
  pdl_wait();
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step)
    table[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}

// One CTA per token: n_end (slots up to the last valid entry), fill (the row of the first valid one, 0 without any),
// and with a table its entries.  A row selected twice by a token is entered once, with its lowest slot, and the
// number of times in mult: the entries' contributions are equal.  An entry outside [-1, S) counts as empty and is
// recorded as DSA_ERR_BAD_INDEX.
__global__ void __launch_bounds__(256) scatter_build_kernel(const int* idx, int k, long long S, int* n_end, int* fill,
                                                            uint16_t* table, int ld, uint16_t* mult) {
  __shared__ int last, first;
  __shared__ int times[sct::MAX_K];
  const int t = blockIdx.x;
  if (threadIdx.x == 0) { last = 0; first = sct::MAX_K; }
  for (int i = threadIdx.x; i < k; i += blockDim.x) times[i] = 1;
  __syncthreads();
  pdl_allow_next();
  pdl_wait();
  const int* row = idx + static_cast<long long>(t) * k;
  auto valid = [&](int e) { return e >= 0 && e < S; };
  auto cell = [&](int e) { return table + static_cast<long long>(e) * ld + t; };
  int my_last = 0, my_first = sct::MAX_K;
  for (int i = threadIdx.x; i < k; i += blockDim.x) {
    const int e = row[i];
    if (valid(e)) {
      my_last = i + 1;
      my_first = min(my_first, i);
      if (table) *cell(e) = static_cast<uint16_t>(i);
    } else if (e != -1) {
      raise_status(DSA_ERR_BAD_INDEX);
    }
  }
  atomicMax(&last, my_last);
  atomicMin(&first, my_first);
  __syncthreads();
  if (threadIdx.x == 0) {
    n_end[t] = last;
    fill[t] = first < k ? row[first] : 0;
  }
  if (!table) return;
  // the lowest slot wins: repeated until no slot is below the one entered
  while (true) {
    bool moved = false;
    for (int i = threadIdx.x; i < k; i += blockDim.x) {
      const int e = row[i];
      if (valid(e) && __ldcg(cell(e)) > i) {
        *cell(e) = static_cast<uint16_t>(i);
        moved = true;
      }
    }
    if (!__syncthreads_or(moved)) break;
  }
  bool again = false;
  for (int i = threadIdx.x; i < k; i += blockDim.x) {
    const int e = row[i];
    if (!valid(e)) continue;
    const int won = __ldcg(cell(e));
    if (won != i) { atomicAdd(&times[won], 1); again = true; }
  }
  if (!__syncthreads_or(again)) return;
  for (int i = threadIdx.x; i < k; i += blockDim.x)
    if (times[i] > 1) {
      *cell(row[i]) = static_cast<uint16_t>(i) | sct::TWICE;
      mult[static_cast<long long>(t) * k + i] = static_cast<uint16_t>(times[i]);
    }
}

struct ScatterParams {
  const uint16_t* contrib;    // [T * kp, W] bf16
  const uint16_t* table;      // [S, ld]
  const uint16_t* mult;       // [T, k]
  int T, ld, k, kp;
  float* acc;                 // [S, W] sums of the chunks so far, or null (one chunk)
  int first, last;            // first / last chunk
  uint16_t* out;              // [S, W] bf16, written with the last chunk
};

// One CTA per row: W / 8 threads hold the row's W values (16-byte loads), as many groups of them as fit the CTA take
// equal runs of the row's list, four rows in flight each.
template <int W>
struct ScatterCfg {
  static constexpr int PER_ROW = W / 8;
  static constexpr int GROUPS = 288 / PER_ROW;        // 4 (W = 576), 18 (128), 36 (64)
  static constexpr int THREADS = GROUPS * PER_ROW;    // 288
};

template <int W>
__global__ void __launch_bounds__(ScatterCfg<W>::THREADS) scatter_sum_kernel(const ScatterParams p) {
  using C = ScatterCfg<W>;
  static_assert(C::THREADS % 32 == 0, "whole warps");
  __shared__ uint32_t list[sct::MAX_T];
  __shared__ int warp_n[C::THREADS / 32];
  __shared__ float part[C::GROUPS][W];
  pdl_allow_next();
  pdl_wait();
  const long long s = blockIdx.x;
  const uint16_t* row = p.table + s * p.ld;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
  for (int t0 = 0; t0 < p.T; t0 += C::THREADS) {
    const int t = t0 + threadIdx.x;
    const uint16_t v = t < p.T ? row[t] : sct::EMPTY;
    const uint32_t have = __ballot_sync(0xffffffffu, v != sct::EMPTY);
    if (lane == 0) warp_n[warp] = __popc(have);
    __syncthreads();
    int at = n;
    for (int w = 0; w < C::THREADS / 32; ++w) {
      if (w < warp) at += warp_n[w];
      n += warp_n[w];
    }
    // token and slot; the flag goes to the top bit
    if (v != sct::EMPTY)
      list[at + __popc(have & ((1u << lane) - 1))] =
          (static_cast<uint32_t>(t) << 11) | (v & (sct::TWICE - 1)) | ((v & sct::TWICE) ? 0x80000000u : 0u);
    __syncthreads();
  }
  const int group = threadIdx.x / C::PER_ROW, col = threadIdx.x % C::PER_ROW;
  float sum[8] = {};
  const int each = (n + C::GROUPS - 1) / C::GROUPS, end = min(n, (group + 1) * each);
  for (int i = group * each; i < end; i += 4) {
    uint4 v[4];
    float m[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      m[u] = 0.f;
      v[u] = make_uint4(0, 0, 0, 0);
      if (i + u < end) {
        const uint32_t e = list[i + u];
        const long long t = (e >> 11) & 0xfffff;
        const int slot = e & (sct::TWICE - 1);
        v[u] = reinterpret_cast<const uint4*>(p.contrib + (t * p.kp + slot) * W)[col];
        m[u] = (e >> 31) ? static_cast<float>(p.mult[t * p.k + slot]) : 1.f;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t x[4] = {v[u].x, v[u].y, v[u].z, v[u].w};
      if (i + u < end) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          sum[2 * q] = fmaf(m[u], __uint_as_float(x[q] << 16), sum[2 * q]);
          sum[2 * q + 1] = fmaf(m[u], __uint_as_float(x[q] & 0xffff0000u), sum[2 * q + 1]);
        }
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) part[group][8 * col + q] = sum[q];
  __syncthreads();
  for (int d = threadIdx.x; d < W; d += C::THREADS) {
    float total = 0.f;
    for (int g = 0; g < C::GROUPS; ++g) total += part[g][d];
    const long long at = s * W + d;
    if (p.acc && !p.first) total += p.acc[at];
    if (p.last) p.out[at] = __bfloat16_as_ushort(__float2bfloat16_rn(total));
    else p.acc[at] = total;
  }
}

}  // namespace dsa
