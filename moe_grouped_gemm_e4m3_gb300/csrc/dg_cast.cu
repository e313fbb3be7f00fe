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
// One CTA takes a 128x128 tile at a time, which holds whole groups of every form: the input is read once
// into registers, and the maxima along rows (shuffles within 16 lanes), columns and the block (shared
// memory) come from there. Bound by HBM: 2 bytes read and 1 byte written per form and element
// (8192x7168, three forms: 52 us back to back, 5.7 TB/s; issue slots 72% busy, two thirds of it products and conversions).
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

// Eight codes of eight values, the products two a instruction (each rounded by itself).
__device__ __forceinline__ void put_codes8(uint8_t* p, const float2 (&v)[4], const float2 (&f)[4]) {
  uint32_t w[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = __fmul2_rn(v[k], f[k]);
    w[k] = e4m3x2_satfinite(x.x, x.y);
  }
  *reinterpret_cast<uint2*>(p) = make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

__device__ __forceinline__ void put_codes8(uint8_t* p, const float2 (&v)[4], float f) {
  const float2 two = make_float2(f, f), all[4] = {two, two, two, two};
  put_codes8(p, v, all);
}

__device__ __forceinline__ void unpack8(const uint4& w, float2 (&v)[4]) {
  v[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
  v[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
  v[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
  v[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
}

// The maxima of LINES (a power of two) lines over 16 lanes, lane c of them getting line c % LINES: while there
// are several, a lane passes on the half that its partner keeps (8 shuffles for eight lines; reducing line by
// line takes 32).
template <int LINES>
__device__ __forceinline__ float max_over_16(const float (&v)[LINES], int c, int bit = 1) {
  if constexpr (LINES == 1) {
    float m = v[0];
    for (; bit < 16; bit <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, bit));
    return m;
  } else {
    float half[LINES / 2];
#pragma unroll
    for (int k = 0; k < LINES / 2; ++k) {
      const float keep = c & bit ? v[2 * k + 1] : v[2 * k], pass = c & bit ? v[2 * k] : v[2 * k + 1];
      half[k] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, pass, bit));
    }
    return max_over_16<LINES / 2>(half, c, bit << 1);
  }
}

// Asynchronous copy of 16 bytes to this thread's own place in shared memory (zeros if !live). No other thread
// reads it, so wait_copies is all the synchronisation it needs.
__device__ __forceinline__ void copy_16(uint4* to, const void* from, bool live) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(from), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void commit_copies() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void wait_copies() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// ---------------------------------------------------------------------------------------------
// The cast of a BF16 matrix. Thread t holds columns 8·(t % 16).. of the tile's rows i·16 + t/16, i < 8. A
// persistent CTA copies its next tile into shared memory while it works on this one.
constexpr int kCastThreads = 256, kCastRows = 8, kCastStep = 16, kCastCtas = 3;

struct CastShared {
  uint4 next[2][kCastRows][kCastThreads];
  float part[kCastThreads / 32][128];   // each warp's column maxima
  float factor[128];
  float top[4];
};

template <bool UE>
__global__ void __launch_bounds__(kCastThreads, kCastCtas) cast_kernel(const uint16_t* __restrict__ x,
                                                                       const int32_t* __restrict__ m_indices,
                                                                       const CastForms f, int M, int N, int tiles) {
  extern __shared__ __align__(16) uint8_t smem[];
  CastShared& sh = *reinterpret_cast<CastShared*>(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, cg = t % 16, warp = t / 32, lane = t % 32;
  const int Mb = (M + 127) / 128, Nb = (N + 127) / 128, ldm = (M + 3) / 4 * 4;
  const bool across = f.q_col || f.q_blk;   // anything beside rows

  // This thread's rows' indices (0 without m_indices): loaded a tile before the copies that need them are
  // issued, and not looked at until then, so that nothing waits for them.
  auto load_rows = [&](int tile, int (&idx)[kCastRows]) {
#pragma unroll
    for (int i = 0; i < kCastRows; ++i) {
      const int row = tile / Nb % Mb * 128 + t / 16 + i * kCastStep;
      idx[i] = m_indices && tile < tiles && row < M ? __ldg(m_indices + row) : 0;
    }
  };
  auto fetch = [&](int tile, int buf, const int (&idx)[kCastRows]) {
    const int nb = tile % Nb, mb = tile / Nb % Mb, g = tile / Nb / Mb;
    const int row0 = mb * 128 + t / 16, col = nb * 128 + cg * 8;
    const uint16_t* src = x + ((size_t)g * M + row0) * N + col;
#pragma unroll
    for (int i = 0; i < kCastRows; ++i) {
      const bool live = row0 + i * kCastStep < M && col < N && idx[i] >= 0;
      copy_16(&sh.next[buf][i][t], live ? src + (size_t)i * kCastStep * N : x, live);
    }
  };

  int buf = 0;
  const int step = (int)gridDim.x;
  int idx[kCastRows];
  load_rows(blockIdx.x, idx);
  fetch(blockIdx.x, 0, idx);
  commit_copies();
  load_rows((int)blockIdx.x + step, idx);
  for (int tile = blockIdx.x; tile < tiles; tile += step, buf ^= 1) {
    if (tile + step < tiles) fetch(tile + step, buf ^ 1, idx);
    commit_copies();
    load_rows(tile + 2 * step, idx);
    wait_copies<1>();
    const int nb = tile % Nb, mb = tile / Nb % Mb, g = tile / Nb / Mb;
    const int row0 = mb * 128 + t / 16, col = nb * 128 + cg * 8;
    const bool col_live = col < N;
    const size_t off0 = ((size_t)g * M + row0) * N + col;
    uint4 raw[kCastRows];
#pragma unroll
    for (int i = 0; i < kCastRows; ++i) raw[i] = sh.next[buf][i][t];
    // magnitudes, two BF16 a step; a NaN gives way to the other operand, here at the latest to 0
    auto mag = [](uint32_t w) { w &= 0x7FFF7FFFu; return *reinterpret_cast<__nv_bfloat162*>(&w); };
    const __nv_bfloat162 none = mag(0);

    if (f.q_row) {
      float m[8];
#pragma unroll
      for (int i = 0; i < kCastRows; ++i) {
        const __nv_bfloat162 w = __hmax2(__hmax2(__hmax2(mag(raw[i].x), none), mag(raw[i].y)), __hmax2(__hmax2(mag(raw[i].z), none), mag(raw[i].w)));
        m[i] = fmaxf(__low2float(w), __high2float(w));
      }
      float fac;
      uint32_t scale;
      group_scale<UE>(max_over_16(m, cg), fac, scale);   // of row cg % 8
      // the rows past M up to align4(M) get the filler
      const int row = row0 + cg * kCastStep;
      if (cg < 8 && row < ldm)
        put_scale_major<UE>(f.s_row, (size_t)g * (UE ? (Nb + 3) / 4 : Nb), nb, Nb, ldm, row, row < M ? scale : (UE ? 127u : 0u));
#pragma unroll
      for (int i = 0; i < kCastRows; ++i) {
        const float fi = __shfl_sync(0xffffffffu, fac, i, 16);
        float2 v[4];
        unpack8(raw[i], v);
        if (row0 + i * kCastStep < M && col_live) put_codes8(f.q_row + off0 + (size_t)i * kCastStep * N, v, fi);
      }
    }
    if (!across) continue;

    __nv_bfloat162 m[4] = {none, none, none, none};
#pragma unroll
    for (int i = 0; i < kCastRows; ++i) {
      m[0] = __hmax2(m[0], mag(raw[i].x));
      m[1] = __hmax2(m[1], mag(raw[i].y));
      m[2] = __hmax2(m[2], mag(raw[i].z));
      m[3] = __hmax2(m[3], mag(raw[i].w));
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = __hmax2(m[j], __shfl_xor_sync(0xffffffffu, m[j], 16));
    if (lane < 16) {
      float4* to = reinterpret_cast<float4*>(&sh.part[warp][cg * 8]);
      to[0] = make_float4(__low2float(m[0]), __high2float(m[0]), __low2float(m[1]), __high2float(m[1]));
      to[1] = make_float4(__low2float(m[2]), __high2float(m[2]), __low2float(m[3]), __high2float(m[3]));
    }
    __syncthreads();   // (every thread has read the previous tile's factors by then)
    if (t < 128) {
      float top = 0.0f;
#pragma unroll
      for (int w = 0; w < kCastThreads / 32; ++w) top = fmaxf(top, sh.part[w][t]);
      if (f.q_col) {
        float fac;
        uint32_t scale;
        group_scale<UE>(top, fac, scale);
        sh.factor[t] = fac;
        const int n = nb * 128 + t;
        if (n < N) put_scale_major<UE>(f.s_col, (size_t)g * (UE ? (Mb + 3) / 4 : Mb), mb, Mb, N, n, scale);   // (N % 16 == 0)
      }
      const uint32_t block = __reduce_max_sync(0xffffffffu, __float_as_uint(top));   // magnitudes: ordered as integers
      if (lane == 0) sh.top[warp] = __uint_as_float(block);
    }
    __syncthreads();
    float2 cf[4];
    float bf = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) cf[k] = *reinterpret_cast<const float2*>(&sh.factor[cg * 8 + 2 * k]);
    if (f.q_blk) {
      uint32_t scale;
      group_scale<UE>(fmaxf(fmaxf(sh.top[0], sh.top[1]), fmaxf(sh.top[2], sh.top[3])), bf, scale);
      if (t == 0) {
        if (f.s_blk) put_scale_last<UE>(f.s_blk, (size_t)g * Mb + mb, nb, Nb, scale);
        if (f.s_blk_t) put_scale_last<UE>(f.s_blk_t, (size_t)g * Nb + nb, mb, Mb, scale);
      }
    }
#pragma unroll
    for (int i = 0; i < kCastRows; ++i) {
      if (row0 + i * kCastStep >= M || !col_live) continue;
      float2 v[4];
      unpack8(raw[i], v);
      const size_t off = off0 + (size_t)i * kCastStep * N;
      if (f.q_col) put_codes8(f.q_col + off, v, cf);
      if (f.q_blk) put_codes8(f.q_blk + off, v, bf);
    }
  }
  wait_copies<0>();
}

// 1/(1 + e^-x) from the hardware's base-2 exponential and reciprocal, subnormals flushed (1 + e^-x is at least
// 1, and infinite, with the quotient 0, below about -88). Relative error below 1e-5 where |x| < 88.
__device__ __forceinline__ float2 gate_sigmoid(float2 x) {
  const float2 y = __fmul2_rn(x, make_float2(-1.4426950408889634f, -1.4426950408889634f));
  float2 e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(y.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(y.y));
  e = __fadd2_rn(e, make_float2(1.0f, 1.0f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.x) : "f"(e.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s.y) : "f"(e.y));
  return s;
}

// ---------------------------------------------------------------------------------------------
// The backward pass of H = dropout(silu(g)·u), from the saved BF16 g and u and the gradient dH:
//   t = dropout(dH) (the forward pass's mask and scale), s = 1/(1 + e^-g),
//   dg = t·u·s·(1 + g·(1 - s)),  du = t·g·s,
// in FP32, cast straight to the row and column forms of [dG dU] ([M, 2I]); and, if asked (BLOCKS), the blocks
// of H formed again from g and u. One tile of inputs gives a tile of dG and a tile of dU. Thread t holds
// columns 8·(t % 16).. of the tile's rows i·32 + t/16, i < 4. Persistent, with the next tile's inputs
// copied ahead as above: one CTA of 512 threads an SM, since dG and dU stay in registers between their
// maxima and their codes.
//
// SPLIT > 1: a tile's rows are shared by a cluster of SPLIT CTAs (one tile a cluster), which exchange their
// column maxima through distributed shared memory. For few tiles, where one CTA's arithmetic on a whole tile is most of
// the call: 200x512 rows 5.1 us with SPLIT = 1, 4.1 with 4.
constexpr int kGateThreads = 512;

template <int SPLIT>
struct GatePlan {
  static constexpr int kRows = 4 / SPLIT, kStep = 32;   // rows a thread, this many apart
};

template <int SPLIT>
struct GateShared {
  uint4 next[2][3 * GatePlan<SPLIT>::kRows][kGateThreads];
  float part[2][kGateThreads / 32][128];   // each warp's column maxima of dG and dU
  float factor[2][128];
  float h_top[kGateThreads / 32];
  float h_factor;
  float cta_top[2][128], cta_h_top;        // SPLIT > 1: this CTA's maxima, read by its peers
};

// The largest of a float at the same place of every CTA of a cluster of SPLIT.
template <int SPLIT>
__device__ __forceinline__ float cluster_max(const float* mine) {
  uint32_t v[SPLIT], top = 0;
#pragma unroll
  for (int r = 0; r < SPLIT; ++r) v[r] = ld_cluster_u32(cluster_map(smem_u32(mine), (uint32_t)r));
#pragma unroll
  for (int r = 0; r < SPLIT; ++r) top = max(top, v[r]);   // magnitudes: ordered as integers
  return __uint_as_float(top);
}

template <bool UE, bool BLOCKS, int SPLIT>
__global__ void __launch_bounds__(kGateThreads, 1) swiglu_backward_kernel(const uint16_t* __restrict__ dh,
                                                                          const uint16_t* __restrict__ gu,
                                                                          const int32_t* __restrict__ m_indices,
                                                                          const Dropout d, const CastForms f,
                                                                          const CastForms f_h, int M, int I, int tiles) {
  constexpr int kGateRows = GatePlan<SPLIT>::kRows, kGateStep = GatePlan<SPLIT>::kStep;
  extern __shared__ __align__(16) uint8_t smem[];
  GateShared<SPLIT>& sh = *reinterpret_cast<GateShared<SPLIT>*>(smem);
  griddep_wait();
  griddep_launch_dependents();
  const int t = threadIdx.x, cg = t % 16, warp = t / 32, lane = t % 32;
  const int nI = I / 128, Mb = (M + 127) / 128, ldm = (M + 3) / 4 * 4;
  const bool drop = d.threshold != 0;
  const Philox gen = drop ? Philox(d.rng) : Philox();
  const int rank = SPLIT > 1 ? (int)(blockIdx.x % SPLIT) : 0, tile0 = (int)blockIdx.x / SPLIT;
  const int t_row = rank * kGateRows * kGateStep + t / 16;   // this thread's first row in a tile

  // This thread's rows' indices (0 without m_indices): loaded a tile before the copies that need them are
  // issued, and not looked at until then, so that nothing waits for them.
  auto load_rows = [&](int tile, int (&idx)[kGateRows]) {
#pragma unroll
    for (int i = 0; i < kGateRows; ++i) {
      const int row = tile / nI * 128 + t_row + i * kGateStep;
      idx[i] = m_indices && tile < tiles && row < M ? __ldg(m_indices + row) : 0;
    }
  };
  auto fetch = [&](int tile, int buf, const int (&idx)[kGateRows]) {
    const int row0 = tile / nI * 128 + t_row, col = tile % nI * 128 + cg * 8;
#pragma unroll
    for (int i = 0; i < kGateRows; ++i) {
      const int row = row0 + i * kGateStep;
      const bool live = row < M && idx[i] >= 0;
      const size_t at = live ? (size_t)row * I + col : 0, at2 = live ? (size_t)row * 2 * I + col : 0;
      copy_16(&sh.next[buf][3 * i][t], dh + at, live);
      copy_16(&sh.next[buf][3 * i + 1][t], gu + at2, live);
      copy_16(&sh.next[buf][3 * i + 2][t], gu + at2 + I, live);
    }
  };

  int buf = 0;
  const int step = (int)gridDim.x / SPLIT;
  int idx[kGateRows];
  load_rows(tile0, idx);
  fetch(tile0, 0, idx);
  commit_copies();
  load_rows(tile0 + step, idx);
  for (int tile = tile0; tile < tiles; tile += step, buf ^= 1) {
    if (tile + step < tiles) fetch(tile + step, buf ^ 1, idx);
    commit_copies();
    load_rows(tile + 2 * step, idx);
    wait_copies<1>();
    const int nb = tile % nI, mb = tile / nI;
    const int row0 = mb * 128 + t_row, col = nb * 128 + cg * 8;
    float2 v[2][kGateRows][4], h[BLOCKS ? kGateRows : 1][4];   // dG and dU; H
    float line[2 * kGateRows], cmax[2][8], hmax = 0.0f;         // row maxima of dG, then of dU; column maxima
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int j = 0; j < 8; ++j) cmax[a][j] = 0.0f;
#pragma unroll
    for (int i = 0; i < kGateRows; ++i) {
      float2 dt[4], g[4], u[4];
      unpack8(sh.next[buf][3 * i][t], dt);
      unpack8(sh.next[buf][3 * i + 1][t], g);
      unpack8(sh.next[buf][3 * i + 2][t], u);
      uint4 w = make_uint4(0, 0, 0, 0);
      if (drop) {
        w = gen(((uint64_t)(row0 + i * kGateStep) * I + col) / 8);
        dropout8(reinterpret_cast<float(&)[8]>(dt), w, d.threshold, d.scale);
      }
      line[i] = line[kGateRows + i] = 0.0f;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 s = gate_sigmoid(g[k]), gs = __fmul2_rn(g[k], s);
        // dg = t·u·(s + gs·(1 - s)), du = t·gs
        const float2 one = make_float2(1.0f, 1.0f), minus = make_float2(-1.0f, -1.0f);
        v[0][i][k] = __fmul2_rn(__fmul2_rn(dt[k], u[k]), __ffma2_rn(gs, __ffma2_rn(s, minus, one), s));
        v[1][i][k] = __fmul2_rn(dt[k], gs);
        if constexpr (BLOCKS) h[i][k] = __fmul2_rn(gs, u[k]);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const float x = fabsf(v[a][i][k].x), y = fabsf(v[a][i][k].y);
          line[a * kGateRows + i] = fmaxf(fmaxf(line[a * kGateRows + i], x), y);
          cmax[a][2 * k] = fmaxf(cmax[a][2 * k], x);
          cmax[a][2 * k + 1] = fmaxf(cmax[a][2 * k + 1], y);
        }
      }
      if constexpr (BLOCKS) {
        if (drop) dropout8(reinterpret_cast<float(&)[8]>(h[i]), w, d.threshold, d.scale);
#pragma unroll
        for (int k = 0; k < 4; ++k) hmax = fmaxf(fmaxf(hmax, fabsf(h[i][k].x)), fabsf(h[i][k].y));
      }
    }
    const size_t off0 = (size_t)row0 * 2 * I + col;

    if (f.q_row) {
      float fac;
      uint32_t scale;
      group_scale<UE>(max_over_16(line, cg), fac, scale);   // lines: dG's rows, then dU's
      const int row = row0 + cg % kGateRows * kGateStep;
      if (cg < 2 * kGateRows && row < ldm)
        put_scale_major<UE>(f.s_row, 0, nb + cg / kGateRows * nI, 2 * nI, ldm, row, row < M ? scale : (UE ? 127u : 0u));
#pragma unroll
      for (int a = 0; a < 2; ++a)
#pragma unroll
        for (int i = 0; i < kGateRows; ++i) {
          const float fi = __shfl_sync(0xffffffffu, fac, a * kGateRows + i, 16);
          if (row0 + i * kGateStep < M) put_codes8(f.q_row + off0 + (size_t)i * kGateStep * 2 * I + a * I, v[a][i], fi);
        }
    }
    if (!f.q_col && !BLOCKS) continue;

#pragma unroll
    for (int a = 0; a < 2; ++a) {
#pragma unroll
      for (int j = 0; j < 8; ++j) cmax[a][j] = fmaxf(cmax[a][j], __shfl_xor_sync(0xffffffffu, cmax[a][j], 16));
      if (lane < 16) {
        float4* to = reinterpret_cast<float4*>(&sh.part[a][warp][cg * 8]);
        to[0] = make_float4(cmax[a][0], cmax[a][1], cmax[a][2], cmax[a][3]);
        to[1] = make_float4(cmax[a][4], cmax[a][5], cmax[a][6], cmax[a][7]);
      }
    }
    if constexpr (BLOCKS) {
      const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(hmax));   // magnitudes: ordered as integers
      if (lane == 0) sh.h_top[warp] = __uint_as_float(top);
    }
    __syncthreads();   // (every thread has read the previous tile's factors by then)
    const bool h_warp = BLOCKS && warp == 8;
    float top = 0.0f;
    if (t < 256) {
#pragma unroll
      for (int w = 0; w < kGateThreads / 32; ++w) top = fmaxf(top, sh.part[t / 128][w][t % 128]);
    } else if (h_warp) {
      top = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(lane < kGateThreads / 32 ? sh.h_top[lane] : 0.0f)));
    }
    if constexpr (SPLIT > 1) {
      if (t < 256) sh.cta_top[t / 128][t % 128] = top;
      else if (h_warp && lane == 0) sh.cta_h_top = top;
      cluster_sync_all();
      if (t < 256) top = cluster_max<SPLIT>(&sh.cta_top[t / 128][t % 128]);
      else if (h_warp) top = cluster_max<SPLIT>(&sh.cta_h_top);
    }
    if (t < 256) {
      const int a = t / 128, c = t % 128;
      float fac;
      uint32_t scale;
      group_scale<UE>(top, fac, scale);
      sh.factor[a][c] = fac;
      if (f.q_col && rank == 0) put_scale_major<UE>(f.s_col, 0, mb, Mb, 2 * I, a * I + nb * 128 + c, scale);
    } else if (h_warp) {
      float fac;
      uint32_t scale;
      group_scale<UE>(top, fac, scale);
      if (lane == 0) {
        sh.h_factor = fac;
        if (rank == 0) put_scale_last<UE>(f_h.s_blk_t, nb, mb, Mb, scale);
      }
    }
    __syncthreads();
    if (f.q_col) {
#pragma unroll
      for (int a = 0; a < 2; ++a) {
        float2 cf[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) cf[k] = *reinterpret_cast<const float2*>(&sh.factor[a][cg * 8 + 2 * k]);
#pragma unroll
        for (int i = 0; i < kGateRows; ++i)
          if (row0 + i * kGateStep < M) put_codes8(f.q_col + off0 + (size_t)i * kGateStep * 2 * I + a * I, v[a][i], cf);
      }
    }
    if constexpr (BLOCKS) {
      const float hf = sh.h_factor;
#pragma unroll
      for (int i = 0; i < kGateRows; ++i)
        if (row0 + i * kGateStep < M) put_codes8(f_h.q_blk + (size_t)(row0 + i * kGateStep) * I + col, h[i], hf);
    }
  }
  wait_copies<0>();
  // no CTA of a cluster leaves while a peer may still read its maxima
  if (SPLIT > 1 && (f.q_col || BLOCKS)) cluster_sync_all();
}

template <typename Kernel>
cudaError_t allow_smem(Kernel kernel, size_t bytes, bool (&done)[64]) {   // once per device and kernel
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  done[dev] = e == cudaSuccess;
  return e;
}

template <bool UE>
cudaError_t launch_cast_as(const uint16_t* x, const int32_t* m_indices, const CastForms& f, int G, int M, int N,
                           const StreamArgs& s) {
  static bool done[64] = {};
  const cudaError_t e = allow_smem(cast_kernel<UE>, sizeof(CastShared), done);
  if (e != cudaSuccess) return e;
  const int tiles = G * ((M + 127) / 128) * ((N + 127) / 128), most = (int)s.limit.ctas(kCastCtas);
  return launch_plain(cast_kernel<UE>, tiles < most ? tiles : most, kCastThreads, sizeof(CastShared), s, x, m_indices, f, M,
                      N, tiles);
}

template <bool UE, bool BLOCKS, int SPLIT>
cudaError_t launch_backward_as(const uint16_t* dh, const uint16_t* gu, const int32_t* m_indices, const Dropout& d,
                               const CastForms& dgu, const CastForms& h, int M, int I, const StreamArgs& s) {
  static bool done[64] = {};
  const cudaError_t e = allow_smem(swiglu_backward_kernel<UE, BLOCKS, SPLIT>, sizeof(GateShared<SPLIT>), done);
  if (e != cudaSuccess) return e;
  const int tiles = (M + 127) / 128 * (I / 128), most = s.limit.sms / SPLIT;
  return launch_plain(swiglu_backward_kernel<UE, BLOCKS, SPLIT>, (tiles < most ? tiles : most) * SPLIT, kGateThreads,
                      sizeof(GateShared<SPLIT>), s, dh, gu, m_indices, d, dgu, h, M, I, tiles);
}

}  // namespace

cudaError_t launch_cast(const uint16_t* x, const int32_t* m_indices, const CastForms& f, int G, int M, int N,
                        bool ue8m0, const StreamArgs& s) {
  return ue8m0 ? launch_cast_as<true>(x, m_indices, f, G, M, N, s) : launch_cast_as<false>(x, m_indices, f, G, M, N, s);
}

cudaError_t launch_swiglu_backward(const uint16_t* dh, const uint16_t* gu, const int32_t* m_indices,
                                   const Dropout& d, const CastForms& dgu, const CastForms& h, int M, int I,
                                   bool ue8m0, const StreamArgs& s) {
  auto go = [&](auto launch, const StreamArgs& with) { return launch(dh, gu, m_indices, d, dgu, h, M, I, with); };
  // few tiles: four CTAs on each, while every cluster gets SMs of its own
  const long long tiles = ((long long)M + 127) / 128 * (I / 128);
  if (4 * tiles <= s.limit.sms) {
    StreamArgs four = s;
    four.cluster = 4;
    if (h.q_blk) return ue8m0 ? go(launch_backward_as<true, true, 4>, four) : go(launch_backward_as<false, true, 4>, four);
    return ue8m0 ? go(launch_backward_as<true, false, 4>, four) : go(launch_backward_as<false, false, 4>, four);
  }
  if (h.q_blk) return ue8m0 ? go(launch_backward_as<true, true, 1>, s) : go(launch_backward_as<false, true, 1>, s);
  return ue8m0 ? go(launch_backward_as<true, false, 1>, s) : go(launch_backward_as<false, false, 1>, s);
}

}  // namespace dg
