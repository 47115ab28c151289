// Rotary positions: R of a head's D dims, from rot_off on, turned pairwise by theta = position * f_i.
//   y_a = m (x_a cos theta - x_b sin theta),  y_b = m (x_a sin theta + x_b cos theta)
// with (a, b) = (2 i, 2 i + 1) (interleaved) or (i, i + R/2) (halves); the backward pass is the transpose (-theta).
// The other dims are copied, or left alone when the result replaces its input.
//
// Bound by HBM: each value is read and written once.  A thread owns one 16-byte piece of a head (halves: the two pieces
// of its pairs) and walks over tokens and, for each, over some of the token's heads, so that the turn per position of
// its pairs is formed once and the angles, which the heads share, once a token.  f / 2 pi is taken as a fraction of a
// turn in units of 2^-64, so that position times it wraps to the fraction of a turn by itself (a position of 10^6
// leaves no digit of an fp32 angle); what f / 2 pi itself is off by, f 2^-54.8 (its constant and its product in fp64),
// grows with the position, to 2^-23.8 turns at 2^31.  The fraction reaches sine and cosine as fp32 (2^-26 turns near
// half a turn, and as much again for each of the two roundings of its product with 2 pi / 2^32, bf16 only), and bf16
// results take the hardware's functions (absolute error 2^-20, against 2^-8 of the rounding).
// Measured: 53 us for fp32 [5000, 64, 128] (328 MB, 0.95 of HBM), 10.4 us for the 64 position dims of 131072 rows of
// 576 (33.5 MB: 128 bytes of every 1152; what bounds it has not been profiled), 2.4 us for 64 x 128 heads of a decode
// step.
#pragma once
#include "common.cuh"

namespace dsa {

struct RopeParams {
  const void* x;
  void* out;
  long long x_st, x_sh, o_st, o_sh;   // strides of tokens and heads (elements)
  const int* positions;               // [T] or null: pos0 + t
  const double* freq;                 // [R / 2]
  int pos0, T, H, D, off, R;
  int rot_units, copy_units;          // pieces of a head: rotated ones (pairs of pieces), copied ones
  int heads_per;                      // heads of a thread; blockIdx.y counts their groups
  float m;
  int backward;
};

template <typename E> __device__ __forceinline__ float rope_get(E v);
template <> __device__ __forceinline__ float rope_get<float>(float v) { return v; }
template <> __device__ __forceinline__ float rope_get<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename E> __device__ __forceinline__ E rope_put(float v);
template <> __device__ __forceinline__ float rope_put<float>(float v) { return v; }
template <> __device__ __forceinline__ __nv_bfloat16 rope_put<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// N elements moved as one access where N * sizeof(E) = 16, one by one otherwise (N = 1: any alignment)
template <typename E, int N> struct alignas(N * sizeof(E)) RopePiece { E v[N]; };

// B: heads in flight (1 where a thread has one head)
template <typename E, int N, bool INTER, int B>
__global__ void __launch_bounds__(256, B == 1 ? 4 : sizeof(E) == 4 ? 3 : 2) rope_kernel(const RopeParams p) {
  pdl_allow_next();
  pdl_wait();
  // block (x, y): x over the pieces of a head, y over tokens; blockIdx.z = 1: the copied pieces (a warp with both kinds
  // would do both in turn: for the fp32 indexer queries, half of whose dims are copied, 81 us against 55)
  constexpr int PAIRS = INTER && N > 1 ? N / 2 : N;
  using Piece = RopePiece<E, N>;
  const int h0 = blockIdx.y * p.heads_per, h1 = min(p.H, h0 + p.heads_per);
  const int t0 = blockIdx.x * blockDim.y + threadIdx.y, dt = gridDim.x * blockDim.y;
  auto xrow = [&](int t, int h) { return static_cast<const E*>(p.x) + t * p.x_st + h * p.x_sh; };
  auto yrow = [&](int t, int h) { return static_cast<E*>(p.out) + t * p.o_st + h * p.o_sh; };
  if (blockIdx.z) {
    for (int unit = threadIdx.x; unit < p.copy_units; unit += blockDim.x) {
      // copied dims: those before rot_off, then those after the rotated ones
      int d = unit * N;
      if (d >= p.off) d += p.R;
      for (int t = t0; t < p.T; t += dt) {
        for (int h = h0; h < h1; h += B) {
          Piece v[B];
#pragma unroll
          for (int u = 0; u < B; ++u)
            if (h + u < h1) v[u] = *reinterpret_cast<const Piece*>(xrow(t, h + u) + d);
#pragma unroll
          for (int u = 0; u < B; ++u)
            if (h + u < h1) *reinterpret_cast<Piece*>(yrow(t, h + u) + d) = v[u];
        }
      }
    }
    return;
  }
  for (int unit = threadIdx.x; unit < p.rot_units; unit += blockDim.x) {
    // first pair of the piece, and where its two elements are
    const int pair = unit * PAIRS;
    const int da = p.off + (INTER ? 2 * pair : pair), db = p.off + (INTER ? 2 * pair + 1 : pair + p.R / 2);
    constexpr bool BOTH = !(INTER && N > 1);   // the pairs' second elements lie in a piece of their own
    Piece va[B], vb[BOTH ? B : 1];
    auto load = [&](int t, int h) {
#pragma unroll
      for (int u = 0; u < B; ++u) {
        if (h + u >= h1) break;
        va[u] = *reinterpret_cast<const Piece*>(xrow(t, h + u) + da);
        if constexpr (BOTH) vb[u] = *reinterpret_cast<const Piece*>(xrow(t, h + u) + db);
      }
    };
    int pos = 0;
    if (t0 < p.T) {                       // on their way while the turns are formed
      load(t0, h0);
      pos = p.positions ? p.positions[t0] : p.pos0 + t0;
    }
    unsigned long long turn[PAIRS];
#pragma unroll
    for (int q = 0; q < PAIRS; ++q) {
      double x = p.freq[pair + q] * 0.15915494309189533577;                 // 1 / (2 pi)
      if (fabs(x) >= 0.5) x -= rint(x);
      turn[q] = static_cast<unsigned long long>(__double2ll_rn(x * 18446744073709551616.0));
    }
    for (int t = t0; t < p.T; t += dt) {
      float c[PAIRS], s[PAIRS];
#pragma unroll
      for (int q = 0; q < PAIRS; ++q) {
        const unsigned long long at = turn[q] * static_cast<unsigned long long>(static_cast<long long>(pos));
        const float r = static_cast<float>(static_cast<int>(at >> 32));     // units of 2^-32 turns
        if constexpr (sizeof(E) == 2) {
          c[q] = __cosf(r * 1.4629180792671596e-9f);                        // 2 pi / 2^32
          s[q] = __sinf(r * 1.4629180792671596e-9f);
        } else {
          sincospif(r * 4.6566128730773926e-10f, &s[q], &c[q]);             // 2 / 2^32
        }
        c[q] *= p.m;
        s[q] *= p.backward ? -p.m : p.m;
      }
      for (int h = h0; h < h1; h += B) {
        if (h != h0 || (B > 1 && t != t0)) load(t, h);
        Piece ya[B], yb[BOTH ? B : 1];
#pragma unroll
        for (int u = 0; u < B; ++u) {
#pragma unroll
          for (int q = 0; q < PAIRS; ++q) {
            const float a = rope_get<E>(BOTH ? va[u].v[q] : va[u].v[2 * q]);
            const float b = rope_get<E>(BOTH ? vb[BOTH ? u : 0].v[q] : va[u].v[BOTH ? 0 : 2 * q + 1]);
            (BOTH ? ya[u].v[q] : ya[u].v[2 * q]) = rope_put<E>(a * c[q] - b * s[q]);
            (BOTH ? yb[BOTH ? u : 0].v[q] : ya[u].v[BOTH ? 0 : 2 * q + 1]) = rope_put<E>(a * s[q] + b * c[q]);
          }
        }
        if (h + B >= h1 && t + dt < p.T) {  // the next token's head (with one a thread), ahead of the stores
          if (B == 1) load(t + dt, h0);
          pos = p.positions ? p.positions[t + dt] : p.pos0 + t + dt;
        }
#pragma unroll
        for (int u = 0; u < B; ++u) {
          if (h + u >= h1) break;
          *reinterpret_cast<Piece*>(yrow(t, h + u) + da) = ya[u];
          if constexpr (BOTH) *reinterpret_cast<Piece*>(yrow(t, h + u) + db) = yb[u];
        }
      }
    }
  }
}

}  // namespace dsa
