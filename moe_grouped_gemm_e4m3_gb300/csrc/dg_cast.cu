// dg_cast.cu — E4M3 casts of BF16 activations and of the gated activation's gradients.
//
// Three forms of a matrix [M, N], each with one scale per group of 128 contracted elements, in the
// layouts the products read:
//   rows:   1x128 groups along the columns (A of the NT and NN products), scales [ceil(N/128)][align4(M)];
//   cols:   128x1 groups along the rows (A, stored [K, M], of the TN and K-grouped products: rows are the
//           contraction there), scales [ceil(M/128)][align4(N)];
//   blocks: 128x128 blocks (B of every product), scales [ceil(M/128)][ceil(N/128)] (B stored [N, K]) and/or
//           transposed [ceil(N/128)][ceil(M/128)] (B stored [K, N]).
// All keep the matrix's own order, so no form needs a transposed copy.
//
// The cast of a group, with a = max(amax, 2^-100), amax the largest magnitude (amax = 0: codes 0,
// scale 1):
//   FP32 scales:  code = e4m3_rne(clamp(x · (448/a), ±448)), scale = a/448 (IEEE divisions);
//   UE8M0 scales: scale = the smallest power of two s with a/s <= 448, code = e4m3_rne(x/s) (x/s is exact).
// (2^-100 keeps 448/a finite.) A NaN becomes the NaN code. A group with an infinity dequantises to
// NaN: its scale is infinite, or UE8M0's NaN.
//
// One CTA takes one 128x128 tile, which holds whole groups of every form: the input is read once
// into registers, and the maxima along rows (shuffles within 16 lanes), columns and the block (shared
// memory) come from there. Bound by HBM: 2 bytes read and 1 byte written per form and element.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_vec.cuh"

namespace dg {

namespace {

// The factor to codes and the scale of a group: FP32 bits, or a UE8M0 code.
template <bool UE>
__device__ __forceinline__ void group_scale(float amax, float& factor, uint32_t& scale) {
  const float a = fmaxf(amax, 0x1p-100f);
  if constexpr (UE) {
    const uint32_t bits = __float_as_uint(a), e = bits >> 23;
    uint32_t code = e - 8u + ((bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u);   // 448 = 1.75 · 2^8
    if (amax == 0.0f) code = 127u;
    factor = __uint_as_float((254u - code) << 23);
    if (e == 255u) { code = 255u; factor = 0.0f; }
    scale = code;
  } else {
    factor = amax == 0.0f ? 1.0f : __fdiv_rn(448.0f, a);
    scale = __float_as_uint(amax == 0.0f ? 1.0f : __fdiv_rn(a, 448.0f));
  }
}

// Puts the scale of group `kb` (of nkb along the contraction) of line `i`: FP32 at [kb][i] of lines of
// `stride`, or byte kb % 4 of word [kb / 4][i]; the last group also fills its word's unused bytes.
template <bool UE>
__device__ __forceinline__ void put_scale_major(void* base, size_t first_kb, int kb, int nkb, size_t stride, size_t i,
                                                uint32_t scale) {
  if constexpr (UE) {
    uint8_t* p = static_cast<uint8_t*>(base) + ((first_kb + kb / 4) * stride + i) * 4;
    p[kb & 3] = (uint8_t)scale;
    if (kb == nkb - 1)
      for (int j = (kb & 3) + 1; j < 4; ++j) p[j] = 127;
  } else {
    static_cast<uint32_t*>(base)[(first_kb + kb) * stride + i] = scale;
  }
}

// The same where the contraction is the last axis: FP32 at [line][kb], or byte kb % 4 of word [line][kb / 4].
template <bool UE>
__device__ __forceinline__ void put_scale_last(void* base, size_t line, int kb, int nkb, uint32_t scale) {
  if constexpr (UE) {
    uint8_t* p = static_cast<uint8_t*>(base) + (line * ((nkb + 3) / 4) + kb / 4) * 4;
    p[kb & 3] = (uint8_t)scale;
    if (kb == nkb - 1)
      for (int j = (kb & 3) + 1; j < 4; ++j) p[j] = 127;
  } else {
    static_cast<uint32_t*>(base)[line * nkb + kb] = scale;
  }
}

__device__ __forceinline__ uint32_t codes4(const float* v, float f0, float f1, float f2, float f3) {
  return e4m3x2_satfinite(__fmul_rn(v[0], f0), __fmul_rn(v[1], f1)) |
         (e4m3x2_satfinite(__fmul_rn(v[2], f2), __fmul_rn(v[3], f3)) << 16);
}

template <int THREADS>
struct TileShared {
  float part[THREADS / 32][128];   // each warp's column maxima
  float factor[128];
  float top[4];
};

// One tile's place: group g of matrices [M, N] (N is the stored width), tile row mb, tile column nb.
struct TilePlace {
  int g, mb, nb, M, N;
};

// Casts one 128x128 tile into the asked forms. Thread t holds, for i < ROWS, the eight columns
// 8·(t % 16).. of tile row i·(THREADS/16) + t/16, given by value(i, float (&)[8]): zeros where the matrix
// has no such row or column.
template <bool UE, int THREADS, typename Value>
__device__ __forceinline__ void cast_tile(TileShared<THREADS>& sh, const CastForms& f, const TilePlace& at,
                                          const Value& value) {
  constexpr int kRows = 128 * 16 / THREADS, kStep = THREADS / 16;
  const int t = threadIdx.x, cg = t % 16, warp = t / 32, lane = t % 32;
  const int row0 = at.mb * 128 + t / 16, col = at.nb * 128 + cg * 8;
  const int Mb = (at.M + 127) / 128, Nb = (at.N + 127) / 128;
  const bool col_live = col < at.N;
  const size_t line0 = (size_t)at.g * at.M;

  if (f.q_row) {
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float v[8];
      value(i, v);
      float m = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(v[j]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      float fac;
      uint32_t scale;
      group_scale<UE>(m, fac, scale);
      if (cg == i) mine = scale;
      const int row = row0 + i * kStep;
      if (row < at.M && col_live)
        *reinterpret_cast<uint2*>(f.q_row + (line0 + row) * at.N + col) =
            make_uint2(codes4(v, fac, fac, fac, fac), codes4(v + 4, fac, fac, fac, fac));
    }
    // lane cg = i of a row's 16 puts the scale of row i; the rows past M up to align4(M) get the filler
    const int ldm = (at.M + 3) / 4 * 4, row = row0 + cg * kStep;
    if (cg < kRows && row < ldm)
      put_scale_major<UE>(f.s_row, (size_t)at.g * (UE ? (Nb + 3) / 4 : Nb), at.nb, Nb, ldm, row,
                          row < at.M ? mine : (UE ? 127u : 0u));
  }
  if (!f.q_col && !f.q_blk) return;

  float m[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = 0.0f;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float v[8];
    value(i, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], fabsf(v[j]));
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) m[j] = fmaxf(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
  __syncthreads();   // the previous tile's factors have been read
  if (lane < 16) {
#pragma unroll
    for (int j = 0; j < 8; ++j) sh.part[warp][cg * 8 + j] = m[j];
  }
  __syncthreads();
  if (t < 128) {
    float top = 0.0f;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) top = fmaxf(top, sh.part[w][t]);
    if (f.q_col) {
      float fac;
      uint32_t scale;
      group_scale<UE>(top, fac, scale);
      sh.factor[t] = fac;
      const int n = at.nb * 128 + t, ldn = (at.N + 3) / 4 * 4;
      if (n < ldn)
        put_scale_major<UE>(f.s_col, (size_t)at.g * (UE ? (Mb + 3) / 4 : Mb), at.mb, Mb, ldn, n,
                            n < at.N ? scale : (UE ? 127u : 0u));
    }
    const uint32_t block = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // magnitudes: ordered as integers
    if (lane == 0) sh.top[warp] = __uint_as_float(block);
  }
  __syncthreads();
  float cf[8], bf = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) cf[j] = f.q_col ? sh.factor[cg * 8 + j] : 0.0f;
  if (f.q_blk) {
    uint32_t scale;
    group_scale<UE>(fmaxf(fmaxf(sh.top[0], sh.top[1]), fmaxf(sh.top[2], sh.top[3])), bf, scale);
    if (t == 0) {
      if (f.s_blk) put_scale_last<UE>(f.s_blk, (size_t)at.g * Mb + at.mb, at.nb, Nb, scale);
      if (f.s_blk_t) put_scale_last<UE>(f.s_blk_t, (size_t)at.g * Nb + at.nb, at.mb, Mb, scale);
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kStep;
    if (row >= at.M || !col_live) continue;
    float v[8];
    value(i, v);
    const size_t off = (line0 + row) * at.N + col;
    if (f.q_col)
      *reinterpret_cast<uint2*>(f.q_col + off) =
          make_uint2(codes4(v, cf[0], cf[1], cf[2], cf[3]), codes4(v + 4, cf[4], cf[5], cf[6], cf[7]));
    if (f.q_blk)
      *reinterpret_cast<uint2*>(f.q_blk + off) = make_uint2(codes4(v, bf, bf, bf, bf), codes4(v + 4, bf, bf, bf, bf));
  }
}

constexpr int kCastThreads = 256;

template <bool UE>
__global__ void __launch_bounds__(kCastThreads) cast_kernel(const uint16_t* __restrict__ x,
                                                            const int32_t* __restrict__ m_indices, const CastForms f,
                                                            int M, int N) {
  __shared__ TileShared<kCastThreads> sh;
  constexpr int kRows = 128 * 16 / kCastThreads, kStep = kCastThreads / 16;
  griddep_wait();
  griddep_launch_dependents();
  const int Mb = (M + 127) / 128, Nb = (N + 127) / 128;
  TilePlace at;
  at.nb = blockIdx.x % Nb;
  at.mb = blockIdx.x / Nb % Mb;
  at.g = blockIdx.x / Nb / Mb;
  at.M = M;
  at.N = N;
  const int row0 = at.mb * 128 + threadIdx.x / 16, col = at.nb * 128 + threadIdx.x % 16 * 8;
  const uint16_t* src = x + ((size_t)at.g * M + row0) * N + col;
  uint4 raw[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kStep;
    const bool live = row < M && col < N && (!m_indices || __ldg(m_indices + row) >= 0);
    raw[i] = live ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)i * kStep * N)) : make_uint4(0, 0, 0, 0);
  }
  cast_tile<UE, kCastThreads>(sh, f, at, [&](int i, float(&v)[8]) { unpack8(raw[i], v); });
}

// The backward pass of H = dropout(silu(g)·u), from the saved BF16 g and u and the gradient dH:
//   t = dropout(dH) (the forward pass's mask and scale), s = 1/(1 + e^-g),
//   dg = t·u·s·(1 + g·(1 - s)),  du = t·g·s,
// in FP32, cast straight to the row and column forms of [dG dU] ([M, 2I]); and, if asked, the blocks of H
// formed again from g and u. The tile of dG and the tile of dU use the same inputs.
constexpr int kGateThreads = 512;

template <bool UE>
__global__ void __launch_bounds__(kGateThreads) swiglu_backward_kernel(const uint16_t* __restrict__ dh,
                                                                       const uint16_t* __restrict__ gu,
                                                                       const int32_t* __restrict__ m_indices,
                                                                       const Dropout d, const CastForms f_gu,
                                                                       const CastForms f_h, int M, int I) {
  __shared__ TileShared<kGateThreads> sh;
  constexpr int kRows = 128 * 16 / kGateThreads, kStep = kGateThreads / 16;
  griddep_wait();
  griddep_launch_dependents();
  const int nI = I / 128;
  const int nb = blockIdx.x % nI, mb = blockIdx.x / nI;
  const int row0 = mb * 128 + threadIdx.x / 16, col = nb * 128 + threadIdx.x % 16 * 8;
  uint4 rt[kRows], rg[kRows], ru[kRows];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int row = row0 + i * kStep;
    const bool live = row < M && (!m_indices || __ldg(m_indices + row) >= 0);
    const size_t at = (size_t)row * I + col, at2 = (size_t)row * 2 * I + col;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    rt[i] = live ? __ldg(reinterpret_cast<const uint4*>(dh + at)) : zero;
    rg[i] = live ? __ldg(reinterpret_cast<const uint4*>(gu + at2)) : zero;
    ru[i] = live ? __ldg(reinterpret_cast<const uint4*>(gu + at2 + I)) : zero;
  }
  const bool drop = d.threshold != 0;
  const Philox gen = drop ? Philox(d.rng) : Philox();
  float dg[kRows][8], du[kRows][8], h[kRows][8];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    float t[8], g[8], u[8];
    unpack8(rt[i], t);
    unpack8(rg[i], g);
    unpack8(ru[i], u);
    uint4 w = make_uint4(0, 0, 0, 0);
    if (drop) {
      w = gen(((uint64_t)(row0 + i * kStep) * I + col) / 8);
      dropout8(t, w, d.threshold, d.scale);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float s = __fdividef(1.0f, 1.0f + __expf(-g[j])), a = g[j] * s;
      dg[i][j] = t[j] * u[j] * s * (1.0f + g[j] * (1.0f - s));
      du[i][j] = t[j] * a;
      h[i][j] = a * u[j];
    }
    if (drop) dropout8(h[i], w, d.threshold, d.scale);
  }
  TilePlace at{0, mb, nb, M, 2 * I};
  auto take = [](const float(&from)[8], float(&v)[8]) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = from[j];
  };
  cast_tile<UE, kGateThreads>(sh, f_gu, at, [&](int i, float(&v)[8]) { take(dg[i], v); });
  at.nb = nI + nb;
  cast_tile<UE, kGateThreads>(sh, f_gu, at, [&](int i, float(&v)[8]) { take(du[i], v); });
  if (f_h.q_blk) {
    at = TilePlace{0, mb, nb, M, I};
    cast_tile<UE, kGateThreads>(sh, f_h, at, [&](int i, float(&v)[8]) { take(h[i], v); });
  }
}

}  // namespace

cudaError_t launch_cast(const uint16_t* x, const int32_t* m_indices, const CastForms& f, int G, int M, int N,
                        bool ue8m0, const StreamArgs& s) {
  const int tiles = G * ((M + 127) / 128) * ((N + 127) / 128);
  return launch_plain(ue8m0 ? cast_kernel<true> : cast_kernel<false>, tiles, kCastThreads, 0, s, x, m_indices, f, M, N);
}

cudaError_t launch_swiglu_backward(const uint16_t* dh, const uint16_t* gu, const int32_t* m_indices,
                                   const Dropout& d, const CastForms& dgu, const CastForms& h, int M, int I,
                                   bool ue8m0, const StreamArgs& s) {
  const int tiles = (M + 127) / 128 * (I / 128);
  return launch_plain(ue8m0 ? swiglu_backward_kernel<true> : swiglu_backward_kernel<false>, tiles, kGateThreads, 0, s,
                      dh, gu, m_indices, d, dgu, h, M, I);
}

}  // namespace dg
