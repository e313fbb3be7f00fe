// dg_norm.cu — the norms at a block's boundary, fused with the block's gate and residual scale, and their backward pass.
//
// Forward, one row m of N values (B, the gate, the scale and both norms are optional):
//     P = B·ra·w_after or B,   ra = 1/sqrt(mean(B²) + eps)        the norm after the block
//     R = X + gate[m]·scale·P                                     the stream behind it
//     Y = R·r·W,               r = 1/sqrt(mean(R²) + eps)         the norm before the next block
// FP32 throughout. R and Y are rounded once each, Y formed from the unrounded R; Y's E4M3 rows (the products' A, scales
// of 1x128 groups) are cast from the FP32 Y, as dg_cast_fp8 casts.
//
// Backward, from dY and the gradient dR that reaches the stream from behind (either may be absent), x̂ = R·r, b̂ = B·ra:
//     G  = dR + r·(dY·W − x̂·c),   c = mean(dY·W·x̂)               dX = G,  dW = Σ_m dY·x̂
//     dgate = Σ_n scale·P·G,  dscale = Σ_m gate·P·G,  Q = gate·scale·G
//     dB = ra·(Q·w_after − b̂·mean(Q·w_after·b̂)),  dw_after = Σ_m Q·b̂;   without the norm after the block dB = Q
// G is linear in c, so Σ scale·P·G = S2 − c·r·S3 with S2 = Σ scale·P·(dR + r·dY·W) and S3 = Σ scale·P·x̂, and the mean in
// dB is gate·dgate/N: three sums of one reduction give every scalar of a row.
//
// Both are bound by HBM. The columns' sums (dW, dscale, dw_after) are kept in FP32 registers over the rows of a CTA, one
// partial row a CTA goes to the workspace, and a second kernel adds them in order (no atomics: the same bits every time).
// Row m belongs to partial m % parts, and parts is a function of the sizes alone, not of dg_set_num_sms.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_scale.cuh"
#include "dg_vec.cuh"

namespace dg {

namespace {

// Sums of K values over the CTA, in a fixed order; every thread gets them. `red` holds 32 floats a value and is used by
// turns of two, so that one barrier a call is enough.
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float (*red)[32], int warps) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (warps == 1) return;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) red[k][warp] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? red[k][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}

// Eight elements from column c of a row of n; zeros past its end.
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16* row, int c, int n, float (&v)[8]) {
  if (VEC)
    unpack8(*reinterpret_cast<const uint4*>(row + c), v);
  else
    load8_part(row + c, n - c < 8 ? n - c : 8, v);
}
template <bool VEC>
__device__ __forceinline__ void load8(const float* row, int c, int n, float (&v)[8]) {
  if (VEC) {
    const float4 a = reinterpret_cast<const float4*>(row + c)[0], b = reinterpret_cast<const float4*>(row + c)[1];
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    load8_part(row + c, n - c < 8 ? n - c : 8, v);
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void put8(T* row, int c, int n, const float (&v)[8]) {
  if (VEC)
    store8(row + c, v);
  else
    store8_part(row + c, n - c < 8 ? n - c : 8, v);
}

// ---------------------------------------------------------------------------------------------
// Forward. A CTA takes one row, a thread V vectors of eight columns, in registers from the loads to the stores.
template <typename T, bool VEC, int V, bool UE>
__global__ void __launch_bounds__(128 * V) norm_kernel(const NormArgs a) {
  __shared__ float red[2][1][32];
  griddep_wait();
  griddep_launch_dependents();
  const int N = a.N, warps = blockDim.x / 32, tid = threadIdx.x;
  const float inv_n = 1.0f / (float)N;
  int turn = 0;
  for (int m = blockIdx.x; m < a.M; m += gridDim.x) {
    const size_t at = (size_t)m * N;
    const T* x = static_cast<const T*>(a.x) + at;
    float r[V][8];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * blockDim.x + tid) * 8;
      if (c < N)
        load8<VEC>(x, c, N, r[i]);
      else
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = 0.0f;
    }
    if (a.b) {
      const T* b = static_cast<const T*>(a.b) + at;
      float p[V][8];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * blockDim.x + tid) * 8;
        if (c < N)
          load8<VEC>(b, c, N, p[i]);
        else
#pragma unroll
          for (int j = 0; j < 8; ++j) p[i][j] = 0.0f;
      }
      float f = a.gate ? a.gate[m] : 1.0f;   // of the whole row
      if (a.w_after) {
        float s[1] = {0.0f};
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 8; ++j) s[0] = fmaf(p[i][j], p[i][j], s[0]);
        block_sum(s, red[turn], warps);
        turn ^= 1;
        const float ra = rsqrtf(fmaf(s[0], inv_n, a.eps));
        if (a.rstd_after && tid == 0) a.rstd_after[m] = ra;
        f *= ra;
      }
      T* out = a.r ? static_cast<T*>(a.r) + at : nullptr;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * blockDim.x + tid) * 8;
        if (c >= N) continue;
        if (a.w_after) {
          float w[8];
          load8<VEC>(a.w_after, c, N, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) p[i][j] *= w[j];
        }
        if (a.scale) {
          float w[8];
          load8<VEC>(a.scale, c, N, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) p[i][j] *= w[j];
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] = fmaf(p[i][j], f, r[i][j]);
        if (out) put8<VEC>(out, c, N, r[i]);
      }
    }
    if (!a.w) continue;
    float s[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) s[0] = fmaf(r[i][j], r[i][j], s[0]);
    block_sum(s, red[turn], warps);
    turn ^= 1;
    const float rs = rsqrtf(fmaf(s[0], inv_n, a.eps));
    if (a.rstd && tid == 0) a.rstd[m] = rs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * blockDim.x + tid) * 8;
      const bool live = c < N;
      if (live) {
        float w[8];
        load8<VEC>(a.w, c, N, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) r[i][j] *= rs * w[j];
        if (a.y) put8<VEC>(static_cast<T*>(a.y) + at, c, N, r[i]);
      }
      if (a.q) {   // sixteen lanes hold a group of 128; columns past N are zeros
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(r[i][j]));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (live) {
          float factor;
          uint32_t scale;
          group_scale<UE>(top, factor, scale);
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) q[j] = e4m3x2_satfinite(__fmul_rn(r[i][2 * j], factor), __fmul_rn(r[i][2 * j + 1], factor));
          *reinterpret_cast<uint2*>(a.q + at + c) = make_uint2(q[0] | (q[1] << 16), q[2] | (q[3] << 16));
          if (tid % 16 == 0) {
            const int groups = (N + 127) / 128, ld = (a.M + 3) / 4 * 4;
            put_scale_major<UE>(a.sq, 0, c / 128, groups, ld, m, scale);
            if (m == a.M - 1)   // the rows behind the last
              for (int pad = a.M; pad < ld; ++pad) put_scale_major<UE>(a.sq, 0, c / 128, groups, ld, pad, UE ? 127u : 0u);
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// Backward.
template <typename T>
__device__ __forceinline__ void copy_async(uint8_t* to, const T* from) {   // eight elements, to this thread's own place
#pragma unroll
  for (size_t o = 0; o < 8 * sizeof(T); o += 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + o)), "l"(reinterpret_cast<const uint8_t*>(from) + o)
                 : "memory");
}

// The inputs of `stages` rows are copied ahead into a ring in shared memory, each thread's columns to its own places (so no
// barrier guards them); with no stages (rows too long for it, or any alignment) they are read from the rows themselves.
template <typename T, bool VEC, int V>
__global__ void __launch_bounds__(512) norm_backward_kernel(const NormBackwardArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][3][32];
  griddep_wait();
  griddep_launch_dependents();
  const int N = a.N, TH = blockDim.x, tid = threadIdx.x, warps = TH / 32, stages = a.stages;
  const float inv_n = 1.0f / (float)N;
  const T *const dy = static_cast<const T*>(a.dy), *const dr = static_cast<const T*>(a.dr), *const r = static_cast<const T*>(a.r),
          *const b = static_cast<const T*>(a.b);
  // inputs of a stage one after another, each thread's vectors in its own places
  const size_t plane = (size_t)TH * V * 8 * sizeof(T);
  const int n_in = (dy ? 2 : 0) + (dr ? 1 : 0) + (b ? 1 : 0);   // (R only with dY)
  auto place = [&](int stage, int input, int i) { return ring + (size_t)(stage * n_in + input) * plane + ((size_t)i * TH + tid) * 8 * sizeof(T); };
  auto fetch = [&](int m, int stage) {
    if constexpr (VEC) {
      if (stages > 0 && m < a.M) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int c = (i * TH + tid) * 8;
          if (c >= N) continue;
          const size_t at = (size_t)m * N + c;
          int k = 0;
          if (dy) copy_async(place(stage, k++, i), dy + at), copy_async(place(stage, k++, i), r + at);
          if (dr) copy_async(place(stage, k++, i), dr + at);
          if (b) copy_async(place(stage, k, i), b + at);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  };
  auto get = [&](int stage, int input, int i, const T* from, int m, float (&v)[8]) {
    if (VEC && stages > 0)
      load8<true>(reinterpret_cast<const T*>(place(stage, input, i)), 0, 8, v);
    else
      load8<VEC>(from + (size_t)m * N, (i * TH + tid) * 8, N, v);
  };
  const int in_dr = dy ? 2 : 0, in_b = in_dr + (dr ? 1 : 0);

  for (int part = blockIdx.x; part < a.parts; part += gridDim.x) {   // (more than one only under dg_set_num_sms)
    float sw[V][8] = {}, ss[V][8] = {}, sa[V][8] = {};
    for (int s = 0; s < stages - 1; ++s) fetch(part + s * a.parts, s);
    int stage = 0, turn = 0;
    for (int m = part; m < a.M; m += a.parts, turn ^= 1) {
      {
        const int ahead = stage == 0 ? stages - 1 : stage - 1;   // the stage that the row before this one has left
        if (stages > 0) fetch(m + (stages - 1) * a.parts, stages == 1 ? 0 : ahead);
      }
      if constexpr (VEC) {
        if (stages <= 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
        else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 2;" ::: "memory");
      }
      const float rs = dy ? a.rstd[m] : 0.0f, ra = a.w_after ? a.rstd_after[m] : 1.0f, gate = a.gate ? a.gate[m] : 1.0f;
      float sums[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * TH + tid) * 8;
        if (c >= N) continue;
        float p[8], g[8] = {}, xh[8];
        if (b && (a.w_after || a.dgate)) {
          get(stage, in_b, i, b, m, p);
#pragma unroll
          for (int j = 0; j < 8; ++j) p[j] *= ra;
          float w[8];
          if (a.w_after) {
            load8<VEC>(a.w_after, c, N, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] *= w[j];
          }
          if (a.scale) {
            load8<VEC>(a.scale, c, N, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) p[j] *= w[j];
          }
          if (dr) get(stage, in_dr, i, dr, m, g);
        }
        if (dy) {
          float w[8], d[8];
          get(stage, 0, i, dy, m, d);
          get(stage, 1, i, r, m, xh);
          load8<VEC>(a.w, c, N, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float gw = d[j] * w[j];
            xh[j] *= rs;
            sums[0] = fmaf(gw, xh[j], sums[0]);
            g[j] = fmaf(rs, gw, g[j]);
          }
        }
        if (b && (a.w_after || a.dgate)) {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            sums[1] = fmaf(p[j], g[j], sums[1]);
            if (dy) sums[2] = fmaf(p[j], xh[j], sums[2]);
          }
        }
      }
      if (dy || a.w_after || a.dgate) block_sum(sums, red[turn], warps);
      const float c1 = sums[0] * inv_n, along = fmaf(-c1 * rs, sums[2], sums[1]);   // Σ scale·P·G
      if (a.dgate && tid == 0) a.dgate[m] = along;
      const float c2 = gate * along * inv_n;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = (i * TH + tid) * 8;
        if (c >= N) continue;
        const size_t at = (size_t)m * N;
        float g[8] = {};
        if (dr) get(stage, in_dr, i, dr, m, g);
        if (dy) {
          float w[8], d[8], xh[8];
          get(stage, 0, i, dy, m, d);
          get(stage, 1, i, r, m, xh);
          load8<VEC>(a.w, c, N, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            xh[j] *= rs;
            sw[i][j] = fmaf(d[j], xh[j], sw[i][j]);
            g[j] = fmaf(rs, fmaf(-xh[j], c1, d[j] * w[j]), g[j]);
          }
        }
        float q[8];
        if (b) {
          float bh[8], w[8], sc[8];
          get(stage, in_b, i, b, m, bh);
          if (a.w_after) load8<VEC>(a.w_after, c, N, w);
          if (a.scale) load8<VEC>(a.scale, c, N, sc);
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            bh[j] *= ra;
            const float t = gate * g[j];
            ss[i][j] = fmaf(t, a.w_after ? bh[j] * w[j] : bh[j], ss[i][j]);
            q[j] = a.scale ? t * sc[j] : t;
            if (a.w_after) {
              sa[i][j] = fmaf(q[j], bh[j], sa[i][j]);
              q[j] = ra * fmaf(-bh[j], c2, q[j] * w[j]);
            }
          }
        }
        if (a.dx) put8<VEC>(static_cast<T*>(a.dx) + at, c, N, g);
        if (a.db) put8<VEC>(static_cast<T*>(a.db) + at, c, N, q);
      }
      if (++stage >= stages) stage = 0;
    }
    if constexpr (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
    // the workspace: [parts][sums kept][N]
    float* out = a.partial + (size_t)part * a.sums * N;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (i * TH + tid) * 8;
      if (c >= N) continue;
      int k = 0;
      if (a.dw) put8<VEC>(out + (size_t)k++ * N, c, N, sw[i]);
      if (a.dscale) put8<VEC>(out + (size_t)k++ * N, c, N, ss[i]);
      if (a.dw_after) put8<VEC>(out + (size_t)k * N, c, N, sa[i]);
    }
    __syncthreads();   // red is free for the next part
  }
}

// Adds the partial rows: eight threads a column, each its share of the rows in order, then the eight in order.
constexpr int kSumCols = 32, kSumShares = 8;
__global__ void __launch_bounds__(kSumCols* kSumShares) norm_sum_kernel(const float* __restrict__ partial, int parts, int sums, int N,
                                                                         float* out0, float* out1, float* out2) {
  __shared__ float share[kSumShares][kSumCols];
  griddep_wait();
  griddep_launch_dependents();
  const int col = threadIdx.x % kSumCols, row = threadIdx.x / kSumCols, blocks = (N + kSumCols - 1) / kSumCols;
  for (int block = blockIdx.x; block < blocks * sums; block += gridDim.x) {
    const int k = block / blocks, n = (block % blocks) * kSumCols + col;
    float s = 0.0f;
    if (n < N) {
      const float* p = partial + (size_t)k * N + n;
#pragma unroll 8
      for (int i = row; i < parts; i += kSumShares) s += p[(size_t)i * sums * N];
    }
    share[row][col] = s;
    __syncthreads();
    if (row == 0 && n < N) {
#pragma unroll
      for (int i = 1; i < kSumShares; ++i) s += share[i][col];
      (k == 0 ? out0 : k == 1 ? out1 : out2)[n] = s;
    }
    __syncthreads();
  }
}

int threads_for(int N, int V) { return ((N + 8 * V - 1) / (8 * V) + 31) / 32 * 32; }

template <typename T, bool VEC, bool UE>
cudaError_t launch_forward(const NormArgs& a, const StreamArgs& s) {
  const int grid = (int)s.limit.all(a.M);
  if (a.N <= 1024) return launch_plain(norm_kernel<T, VEC, 1, UE>, grid, threads_for(a.N, 1), 0, s, a);
  if (a.N <= 4096) return launch_plain(norm_kernel<T, VEC, 2, UE>, grid, threads_for(a.N, 2), 0, s, a);
  return launch_plain(norm_kernel<T, VEC, 4, UE>, grid, threads_for(a.N, 4), 0, s, a);
}

bool all_aligned(std::initializer_list<const void*> ps) {
  uintptr_t bits = 0;
  for (const void* p : ps) bits |= reinterpret_cast<uintptr_t>(p);
  return bits % 16 == 0;
}

constexpr int kRingBytes = 216 << 10;   // of an SM, over its CTAs

struct BackwardPlan {
  int V, threads, per_sm, parts;
};
constexpr int kNormSms = 152;
BackwardPlan backward_plan(int M, int N) {
  const int V = N <= 4096 ? 1 : N <= 8192 ? 2 : 4, threads = threads_for(N, V);
  const int per_sm = threads <= 64 ? 8 : threads <= 128 ? 4 : threads <= 256 ? 2 : 1, parts = kNormSms * per_sm;
  return {V, threads, per_sm, M < parts ? M : parts};
}

}  // namespace

long long norm_backward_floats(int M, int N, int sums) {
  return (long long)backward_plan(M, N).parts * sums * N;
}

cudaError_t launch_norm(const NormArgs& a, bool f32, bool ue8m0, const StreamArgs& s) {
  const bool vec = a.N % 8 == 0 && all_aligned({a.x, a.b, a.r, a.y, a.w, a.w_after, a.scale});
  auto go = [&](auto one) {
    using T = decltype(one);
    if (a.q && ue8m0) return vec ? launch_forward<T, true, true>(a, s) : launch_forward<T, false, true>(a, s);
    return vec ? launch_forward<T, true, false>(a, s) : launch_forward<T, false, false>(a, s);
  };
  return f32 ? go(0.0f) : go(__nv_bfloat16{});
}

cudaError_t launch_norm_backward(NormBackwardArgs a, bool f32, const StreamArgs& s) {
  const bool vec = a.N % 8 == 0 && all_aligned({a.dy, a.dr, a.r, a.b, a.dx, a.db, a.w, a.w_after, a.scale, a.partial});
  const BackwardPlan plan = backward_plan(a.M, a.N);
  a.parts = plan.parts;
  auto go = [&](auto one, auto vector, auto v) -> cudaError_t {
    using T = decltype(one);
    constexpr bool VEC = decltype(vector)::value;
    constexpr int V = decltype(v)::value;
    auto kernel = norm_backward_kernel<T, VEC, V>;
    const size_t stage = (size_t)plan.threads * V * 8 * sizeof(T) * ((a.dy ? 2 : 0) + (a.dr ? 1 : 0) + (a.b ? 1 : 0));
    const size_t most = (size_t)kRingBytes / plan.per_sm;
    a.stages = !VEC ? 0 : 3 * stage <= most ? 3 : 2 * stage <= most ? 2 : stage <= most ? 1 : 0;
    const size_t smem = a.stages * stage;
    static bool configured[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev]) {
      if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes)) != cudaSuccess) return e;
      configured[dev] = true;
    }
    return launch_plain(kernel, (int)s.limit.all(plan.parts), plan.threads, smem, s, a);
  };
  auto pick = [&](auto one, auto vector) {
    return plan.V == 1 ? go(one, vector, std::integral_constant<int, 1>{})
                       : plan.V == 2 ? go(one, vector, std::integral_constant<int, 2>{}) : go(one, vector, std::integral_constant<int, 4>{});
  };
  auto type = [&](auto vector) { return f32 ? pick(0.0f, vector) : pick(__nv_bfloat16{}, vector); };
  cudaError_t e = vec ? type(std::true_type{}) : type(std::false_type{});
  if (e != cudaSuccess || a.sums == 0) return e;
  float* outs[3];
  int k = 0;
  for (float* o : {a.dw, a.dscale, a.dw_after})
    if (o) outs[k++] = o;
  for (; k < 3; ++k) outs[k] = nullptr;
  const int blocks = (a.N + kSumCols - 1) / kSumCols * a.sums;
  return launch_plain(norm_sum_kernel, (int)s.limit.all(blocks), kSumCols * kSumShares, 0, s, (const float*)a.partial, a.parts, a.sums,
                      a.N, outs[0], outs[1], outs[2]);
}

}  // namespace dg
