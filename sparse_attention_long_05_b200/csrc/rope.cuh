// Rotary positions: R of a head's D dims, from rot_off on, turned pairwise by theta = position * f_i.
//   y_a = m (x_a cos theta - x_b sin theta),  y_b = m (x_a sin theta + x_b cos theta)
// with (a, b) = (2 i, 2 i + 1) (interleaved) or (i, i + R/2) (halves); the backward pass is the transpose (-theta).
// The other dims are copied, or left alone when the result replaces its input.
//
// Bound by HBM: each value is read and written once.  A thread owns one 16-byte piece (halves: the two pieces of its
// pairs) of a token and walks over the token's heads, so that the angles, which the heads share, are formed once per
// thread.  theta / 2 pi is formed and reduced to [-1/2, 1/2] in fp64 (a position of 10^6 leaves no digit of an fp32
// angle), its sine and cosine in fp32; bf16 results take the hardware's sine and cosine (absolute error 2^-20, against
// 2^-9 of the rounding).
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
  int units;                          // pieces of a token's head: rotated ones first
  int rot_units;
  int head_groups, heads_per;         // threads a piece's heads are spread over; heads of each
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

template <typename E, int N, bool INTER>
__global__ void __launch_bounds__(256) rope_kernel(const RopeParams p) {
  pdl_allow_next();
  pdl_wait();
  // interleaved pieces hold whole pairs: N pairs over two adjacent pieces' worth of elements when N = 1
  constexpr int PAIRS = INTER && N > 1 ? N / 2 : N;
  using Piece = RopePiece<E, N>;
  const unsigned i = blockIdx.x * 256u + threadIdx.x;
  const unsigned per = static_cast<unsigned>(p.units) * p.head_groups;
  const int t = static_cast<int>(i / per);
  if (t >= p.T) return;
  const int rest = static_cast<int>(i % per), hg = rest / p.units, unit = rest % p.units;
  const int h0 = hg * p.heads_per, h1 = min(p.H, h0 + p.heads_per);
  const E* x = static_cast<const E*>(p.x) + t * p.x_st;
  E* out = static_cast<E*>(p.out) + t * p.o_st;
  if (unit >= p.rot_units) {
    // copied dims: those before rot_off, then those after the rotated ones
    int d = (unit - p.rot_units) * N;
    if (d >= p.off) d += p.R;
#pragma unroll 4
    for (int h = h0; h < h1; ++h)
      *reinterpret_cast<Piece*>(out + h * p.o_sh + d) = *reinterpret_cast<const Piece*>(x + h * p.x_sh + d);
    return;
  }
  // first pair of the piece, and where its two elements are
  const int pair = unit * PAIRS;
  const int da = p.off + (INTER ? 2 * pair : pair), db = p.off + (INTER ? 2 * pair + 1 : pair + p.R / 2);
  const double pos = p.positions ? p.positions[t] : p.pos0 + t;
  float c[PAIRS], s[PAIRS];
#pragma unroll
  for (int q = 0; q < PAIRS; ++q) {
    const double turns = pos * p.freq[pair + q] * 0.15915494309189533577;   // 1 / (2 pi)
    const float r = static_cast<float>(turns - rint(turns));
    if constexpr (sizeof(E) == 2) {
      c[q] = __cosf(r * 6.2831853071795865f);
      s[q] = __sinf(r * 6.2831853071795865f);
    } else {
      sincospif(2.f * r, &s[q], &c[q]);
    }
    c[q] *= p.m;
    s[q] *= p.backward ? -p.m : p.m;
  }
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    const E* xr = x + h * p.x_sh;
    E* yr = out + h * p.o_sh;
    if constexpr (INTER && N > 1) {
      Piece v = *reinterpret_cast<const Piece*>(xr + da);
#pragma unroll
      for (int q = 0; q < PAIRS; ++q) {
        const float a = rope_get<E>(v.v[2 * q]), b = rope_get<E>(v.v[2 * q + 1]);
        v.v[2 * q] = rope_put<E>(a * c[q] - b * s[q]);
        v.v[2 * q + 1] = rope_put<E>(a * s[q] + b * c[q]);
      }
      *reinterpret_cast<Piece*>(yr + da) = v;
    } else {
      Piece va = *reinterpret_cast<const Piece*>(xr + da), vb = *reinterpret_cast<const Piece*>(xr + db);
#pragma unroll
      for (int q = 0; q < PAIRS; ++q) {
        const float a = rope_get<E>(va.v[q]), b = rope_get<E>(vb.v[q]);
        va.v[q] = rope_put<E>(a * c[q] - b * s[q]);
        vb.v[q] = rope_put<E>(a * s[q] + b * c[q]);
      }
      *reinterpret_cast<Piece*>(yr + da) = va;
      *reinterpret_cast<Piece*>(yr + db) = vb;
    }
  }
}

}  // namespace dsa
