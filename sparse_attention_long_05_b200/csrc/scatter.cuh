// Sums of per-entry contributions into the rows they belong to: out[s] = sum over tokens t and slots i with
// idx[t][i] = s of contrib[t][i], in a fixed order.
//
// The backward passes write one row of 16-bit values per selected entry (a chunk of tokens at a time): fp16 with a
// power-of-two scale for each 64, whose exponent sits in the lowest bits of every eight.  Ten significant bits are
// left, to which a value is rounded to nearest: it is off by 2^-10 of itself at most and by 2^-11.5 on average (by
// 2^-37 of the largest of its 64, where it is smaller than 2^-28 of that), over the whole range of fp32, and up as
// often as down, so that long lists and sums over many calls do not drift (cut off at ten bits, dc and dk came out
// 3.5e-4 too small; both ways in turn, the rounding takes 879 us instead of 852 for the index scores' pass of 2048
// tokens, the attention's 5007 and 5007).  bf16 rows, no longer, would round four times as much: as much as the
// operands that made them, and gradients would be 1.7 steps of their own rounding off instead of 1.4.  A table of the
// chunk, slot[s][t] = the slot in which token t selected row s (16 bits, empty: 0xffff), turns the scatter into a
// gather: one CTA per row s lists the row's entries in token order and adds them up.  Every sum has one order whatever
// the kernels' timing, so results repeat bit for bit; with atomics they would not.  Bound by HBM: each contribution is
// read once (2 W bytes), the table once (2 bytes per row and token).
#pragma once
#include <cuda_fp16.h>

#include "common.cuh"

namespace dsa {

namespace sct {
constexpr int MAX_T = 2048;               // tokens of a chunk at most (a row's list sits in shared memory)
constexpr int MAX_K = 2048;               // slots of a token at most: 11 bits of a table entry
constexpr uint16_t EMPTY = 0xffff;
constexpr uint16_t TWICE = 0x0800;        // the token selected the row again in later slots
}  // namespace sct

// the whole grid's share of the table
__device__ __forceinline__ void scatter_clear(uint4* table, long long n) {
  const long long step = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step)
    table[i] = make_uint4(~0u, ~0u, ~0u, ~0u);
}
// 64 values as pieces of eight: fp16 of x 2^(141 - E), E the exponent of the largest magnitude of the 64 (29 at least,
// where any fp32 value that is not itself denormal keeps its digits), bit i of E in the lowest bit of a piece's value 2
// i, bit i + 4 in that of value 2 i + 1.
//
// Rounding to ten bits: with y = x 2^(141 - E), t = y (1 + 2^14) in fp32 holds y in steps of 2^14 times y's own, and t
// - 2^14 y is y to nearest in such steps, ties to even, exactly.
//
// Infinities and NaN pass through the scale.  An infinity beside finite values is a sum that left fp32's range (an
// infinite operand leaves nothing finite in the row): it counts as 2^127 to 2^128.  There y = x f / 2 + x f / 2, which
// keeps the infinity, and the lowest bit is cut off.
__device__ __forceinline__ void scatter_pack64(const uint32_t (&v)[64], uint32_t (&w)[32]) {
  float top[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 64; i += 2)
    top[(i >> 1) & 3] = fmaxf(fmaxf(top[(i >> 1) & 3], fabsf(__uint_as_float(v[i]))), fabsf(__uint_as_float(v[i + 1])));
  const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));      // (NaN are not looked at)
  const uint32_t e = min(254u, max(29u, __float_as_uint(most) >> 23));
  const float f = __uint_as_float((268u - e) << 23);
  const float f1 = f * (most == INFINITY ? 0.5f : 16385.f), f2 = f * (most == INFINITY ? 0.5f : -16384.f);
  const uint32_t bits = e | (e << 12);
  const uint32_t b4[4] = {bits & 0x00010001u, (bits >> 1) & 0x00010001u, (bits >> 2) & 0x00010001u,
                          (bits >> 3) & 0x00010001u};
  const uint64_t ff1 = pack_f32x2(f1, f1), ff2 = pack_f32x2(f2, f2);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const uint64_t x = pack_f32x2(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    float lo, hi;
    unpack_f32x2(fma_f32x2(x, ff2, mul_f32x2(x, ff1)), lo, hi);
    const __half2 h = __floats2half2_rn(lo, hi);
    w[i] = (*reinterpret_cast<const uint32_t*>(&h) & 0xfffefffeu) | b4[i & 3];
  }
}
// sum += the piece's values
__device__ __forceinline__ void scatter_add(uint4 v, float (&sum)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  const uint32_t t = (w[0] & 0x00010001u) | ((w[1] & 0x00010001u) << 1) | ((w[2] & 0x00010001u) << 2) |
                     ((w[3] & 0x00010001u) << 3);
  const uint32_t e = (t | (t >> 12)) & 0xffu;
  const float f = __uint_as_float((e - 14u) << 23);    // (e = 0 in the zeros that stand for no entry: -2^115, 0 f = 0)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = w[i] & 0xfffefffeu;
    const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&x));
    sum[2 * i] = fmaf(y.x, f, sum[2 * i]);
    sum[2 * i + 1] = fmaf(y.y, f, sum[2 * i + 1]);
  }
}

__global__ void __launch_bounds__(256) scatter_clear_kernel(uint4* table, long long n) {
  pdl_allow_next();
  pdl_wait();
  scatter_clear(table, n);
}

// One CTA per token: n_end (slots up to the last valid entry), and with a table its entries.  A row selected more than
// once by a token is entered with its lowest slot and flagged.  An entry outside [-1, S) counts as empty and is
// recorded as DSA_ERR_BAD_INDEX.
__global__ void __launch_bounds__(256) scatter_build_kernel(const int* idx, int k, long long S, int* n_end,
                                                            uint16_t* table, int ld) {
  __shared__ int last;
  const int t = blockIdx.x;
  if (threadIdx.x == 0) last = 0;
  __syncthreads();
  pdl_allow_next();
  pdl_wait();
  const int* row = idx + static_cast<long long>(t) * k;
  auto valid = [&](int e) { return e >= 0 && e < S; };
  auto cell = [&](int e) { return table + static_cast<long long>(e) * ld + t; };
  constexpr int PER = sct::MAX_K / 256;
  int e[PER];
  int my_last = 0;
  bool rising = true;                    // ascending entries, then empty slots: no row repeats
#pragma unroll
  for (int u = 0; u < PER; ++u) {
    const int i = u * 256 + threadIdx.x;
    e[u] = i < k ? row[i] : -1;
    if (i + 1 < k) {
      const int next = row[i + 1];
      rising &= !valid(next) || (valid(e[u]) && next > e[u]);
    }
    if (valid(e[u])) {
      my_last = i + 1;
      if (table) *cell(e[u]) = static_cast<uint16_t>(i);
    } else if (e[u] != -1) {
      raise_status(DSA_ERR_BAD_INDEX);
      e[u] = -1;
    }
  }
  my_last = __reduce_max_sync(0xffffffffu, my_last);
  if (lane_id() == 0) atomicMax(&last, my_last);
  rising = __syncthreads_and(rising);
  if (threadIdx.x == 0) n_end[t] = last;
  if (!table || rising) return;
  // the lowest slot wins: repeated until no slot is below the one entered (one round where no row repeats)
  bool again = false;
  while (true) {
    bool moved = false;
    again = false;
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      const int i = u * 256 + threadIdx.x;
      if (e[u] >= 0) {
        const int won = __ldcg(cell(e[u]));
        if (won > i) {
          *cell(e[u]) = static_cast<uint16_t>(i);
          moved = true;
        }
        again |= won != i;
      }
    }
    if (!__syncthreads_or(moved)) break;
  }
  // the last round's reads saw the final slots: whoever is not the winner flags the row
  if (again) {
#pragma unroll
    for (int u = 0; u < PER; ++u) {
      if (e[u] < 0) continue;
      const int won = __ldcg(cell(e[u])) & (sct::TWICE - 1);
      if (won != u * 256 + static_cast<int>(threadIdx.x)) *cell(e[u]) = static_cast<uint16_t>(won | sct::TWICE);
    }
  }
}

struct ScatterParams {
  const uint16_t* contrib;    // [T * kp, W] in pieces of eight (scatter_pack64)
  const uint16_t* table;      // [S, ld]
  const int* idx;             // [T, k]
  int ld, k, kp;
  float* acc;                 // [S, W] sums of the chunks so far, or null (one chunk)
  int first, last;            // first / last chunk
  uint16_t* out;              // [S, W] bf16, written with the last chunk
};

// One CTA per row: W / 8 threads hold the row's W values (16-byte loads), as many groups of them as fit the CTA take
// equal runs of the row's list, eight rows in flight each.
template <int W>
struct ScatterCfg {
  static constexpr int PER_ROW = W / 8;
  static constexpr int GROUPS = W == 576 ? 2 : 160 / PER_ROW;   // 2 (W = 576), 10 (128), 20 (64)
  static constexpr int THREADS = GROUPS * PER_ROW;              // 144, 160, 160
  static constexpr int WARPS = (THREADS + 31) / 32;
  static constexpr int SCAN = (sct::MAX_T / 8 + THREADS - 1) / THREADS;   // 16-byte table reads of a thread
};

template <int W>
__global__ void __launch_bounds__(ScatterCfg<W>::THREADS, W == 576 ? 7 : 8) scatter_sum_kernel(const ScatterParams p) {
  using C = ScatterCfg<W>;
  __shared__ uint32_t list[sct::MAX_T];
  __shared__ int warp_n[C::WARPS];
  __shared__ alignas(16) float part[C::GROUPS][W];
  pdl_allow_next();
  pdl_wait();
  const long long s = blockIdx.x;
  const uint4* row = reinterpret_cast<const uint4*>(p.table + s * p.ld);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int n = 0;
#pragma unroll
  for (int it = 0; it < C::SCAN; ++it) {
    // eight tokens a thread; the last warp may be half full, so every thread of it takes part in the exchange
    const int at = it * C::THREADS + threadIdx.x;
    if (it * C::THREADS * 8 >= p.ld) break;
    const uint4 q = at < p.ld / 8 ? row[at] : make_uint4(~0u, ~0u, ~0u, ~0u);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    int mine = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) mine += ((w[u >> 1] >> (16 * (u & 1))) & 0xffffu) != sct::EMPTY;
    const uint32_t in_warp = __activemask();
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(in_warp, upto, d);
      if (lane >= d) upto += v;
    }
    if (lane == 31 || threadIdx.x == C::THREADS - 1) warp_n[warp] = upto;
    __syncthreads();
    int to = n + upto - mine;
#pragma unroll
    for (int v = 0; v < C::WARPS; ++v) {
      if (v < warp) to += warp_n[v];
      n += warp_n[v];
    }
    // token, slot, and the flag in the top bit
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t v = (w[u >> 1] >> (16 * (u & 1))) & 0xffffu;
      if (v != sct::EMPTY)
        list[to++] = (static_cast<uint32_t>(8 * at + u) << 11) | (v & (sct::TWICE - 1)) | ((v & sct::TWICE) << 20);
    }
    __syncthreads();
  }
  const int group = threadIdx.x / C::PER_ROW, col = threadIdx.x % C::PER_ROW;
  float sum[8] = {};
  auto read = [&](uint32_t t, int slot) {
    return __ldcs(reinterpret_cast<const uint4*>(p.contrib + (static_cast<long long>(t) * p.kp + slot) * W) + col);
  };
  const int each = (n + C::GROUPS - 1) / C::GROUPS, end = min(n, (group + 1) * each);
  for (int i = group * each; i < end; i += 8) {
    uint4 v[8];
    uint32_t any = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t e = i + u < end ? list[i + u] : 0;
      any |= e;
      v[u] = i + u < end ? read((e >> 11) & 0xfffff, e & (sct::TWICE - 1)) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int u = 0; u < 8; ++u) scatter_add(v[u], sum);
    if (any >> 31) {                     // the row's later slots of a token that selected it more than once
#pragma unroll 1
      for (int u = i; u < min(end, i + 8); ++u) {
        const uint32_t e = list[u], t = (e >> 11) & 0xfffff;
        if (!(e >> 31)) continue;
        const int* ids = p.idx + static_cast<long long>(t) * p.k;
#pragma unroll 1
        for (int j = (e & (sct::TWICE - 1)) + 1; j < p.k; ++j)
          if (ids[j] == s) scatter_add(read(t, j), sum);
      }
    }
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) part[group][8 * col + q] = sum[q];
  __syncthreads();
  for (int d = 4 * threadIdx.x; d < W; d += 4 * C::THREADS) {
    float4 total = *reinterpret_cast<const float4*>(&part[0][d]);
#pragma unroll
    for (int g = 1; g < C::GROUPS; ++g) {
      const float4 v = *reinterpret_cast<const float4*>(&part[g][d]);
      total.x += v.x; total.y += v.y; total.z += v.z; total.w += v.w;
    }
    const long long at = s * W + d;
    if (p.acc && !p.first) {
      const float4 v = *reinterpret_cast<const float4*>(p.acc + at);
      total.x += v.x; total.y += v.y; total.z += v.z; total.w += v.w;
    }
    if (p.last) {
      const __nv_bfloat162 lo = __floats2bfloat162_rn(total.x, total.y), hi = __floats2bfloat162_rn(total.z, total.w);
      *reinterpret_cast<uint2*>(p.out + at) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
    } else {
      *reinterpret_cast<float4*>(p.acc + at) = total;
    }
  }
}

// The same for short lists: one warp per row, nothing shared between warps.  W >= 256: the warp reads an entry's pieces
// in W / 256 rounds of loads, four entries in flight; less: 256 / W entries at once, one to each part of the warp,
// whose sums are joined at the end.  With few entries a row the time is the chain table -> entries -> result, which
// eight rows a CTA walk at once here (20 tokens over 20020 rows, W = 576: 16 us against 58).
constexpr int kSumWarps = 8;
template <int W>
__global__ void __launch_bounds__(32 * kSumWarps) scatter_sum_short_kernel(const ScatterParams p, long long S) {
  constexpr int PIECES = W / 8;
  constexpr int PARTS = PIECES < 32 ? 32 / PIECES : 1;       // entries at once
  constexpr int L = (PIECES + 31) / 32;                      // pieces of a lane
  __shared__ uint32_t lists[kSumWarps][256];
  pdl_allow_next();
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long s = static_cast<long long>(blockIdx.x) * kSumWarps + warp;
  if (s >= S) return;
  uint32_t* list = lists[warp];
  const uint4* row = reinterpret_cast<const uint4*>(p.table + s * p.ld);
  const int part = PARTS > 1 ? lane / PIECES : 0, col = PARTS > 1 ? lane % PIECES : lane;
  float sum[L][8] = {};
  auto read = [&](uint32_t t, int slot, uint4 (&v)[L]) {
    const uint4* at = reinterpret_cast<const uint4*>(p.contrib + (static_cast<long long>(t) * p.kp + slot) * W);
#pragma unroll
    for (int i = 0; i < L; ++i)
      v[i] = col + 32 * i < PIECES ? __ldcs(at + col + 32 * i) : make_uint4(0, 0, 0, 0);
  };
  for (int q0 = 0; q0 < p.ld / 8; q0 += 32) {
    // 256 tokens: eight a lane, listed in token order
    const uint4 q = q0 + lane < p.ld / 8 ? row[q0 + lane] : make_uint4(~0u, ~0u, ~0u, ~0u);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    int mine = 0;
#pragma unroll
    for (int u = 0; u < 8; ++u) mine += ((w[u >> 1] >> (16 * (u & 1))) & 0xffffu) != sct::EMPTY;
    int upto = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, d);
      if (lane >= d) upto += v;
    }
    const int n = __shfl_sync(0xffffffffu, upto, 31);
    int to = upto - mine;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t v = (w[u >> 1] >> (16 * (u & 1))) & 0xffffu;
      if (v != sct::EMPTY)
        list[to++] = (static_cast<uint32_t>(8 * (q0 + lane) + u) << 11) | (v & (sct::TWICE - 1)) |
                     ((v & sct::TWICE) << 20);
    }
    __syncwarp();
    for (int i = part; i < n; i += 4 * PARTS) {
      uint4 v[4][L];
      uint32_t any = 0;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t e = i + u * PARTS < n ? list[i + u * PARTS] : 0;
        any |= e;
        if (i + u * PARTS < n) {
          read((e >> 11) & 0xfffff, e & (sct::TWICE - 1), v[u]);
        } else {
#pragma unroll
          for (int j = 0; j < L; ++j) v[u][j] = make_uint4(0, 0, 0, 0);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int j = 0; j < L; ++j) scatter_add(v[u][j], sum[j]);
      if (any >> 31) {                     // the row's later slots of a token that selected it more than once
#pragma unroll 1
        for (int u = 0; u < 4 && i + u * PARTS < n; ++u) {
          const uint32_t e = list[i + u * PARTS], t = (e >> 11) & 0xfffff;
          if (!(e >> 31)) continue;
          const int* ids = p.idx + static_cast<long long>(t) * p.k;
#pragma unroll 1
          for (int j = (e & (sct::TWICE - 1)) + 1; j < p.k; ++j)
            if (ids[j] == s) {
              read(t, j, v[0]);
#pragma unroll
              for (int x = 0; x < L; ++x) scatter_add(v[0][x], sum[x]);
            }
        }
      }
    }
    __syncwarp();
  }
#pragma unroll
  for (int d = PIECES; d < 32; d *= 2)     // the parts' sums
#pragma unroll
    for (int q = 0; q < 8; ++q) sum[0][q] += __shfl_xor_sync(0xffffffffu, sum[0][q], d);
  if (part != 0) return;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    if (col + 32 * i >= PIECES) break;
    const long long at = s * W + 8 * (col + 32 * i);
    float* x = sum[i];
    if (p.acc && !p.first) {
#pragma unroll
      for (int q = 0; q < 8; q += 4) {
        const float4 v = *reinterpret_cast<const float4*>(p.acc + at + q);
        x[q] += v.x; x[q + 1] += v.y; x[q + 2] += v.z; x[q + 3] += v.w;
      }
    }
    if (p.last) {
      uint32_t b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * q], x[2 * q + 1]);
        b[q] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p.out + at) = make_uint4(b[0], b[1], b[2], b[3]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; q += 4)
        *reinterpret_cast<float4*>(p.acc + at + q) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
    }
  }
}

}  // namespace dsa
