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
// Bound by HBM, with the issue slots half busy (us; floor at the measured copy rate): 8192x7168 BF16 with both norms, gate and scale 83
// (69), without the norm after, gate and scale 70 (69), the first one's backward pass 135 (104); 4099x2112 FP32 with E4M3 rows 16 (11.5);
// one row of 7168 4. Farther off where a row does not fit: the backward pass of FP32 rows has a ring of one row at 2112, 4096 and 7168
// columns (8192x7168 301 for 208, 8192x4096 148 for 119, 8192x2112 89 for 61; two rows at 5120, 184 for 149), so that nothing is asked
// for ahead, and above 8192 columns a thread's four vectors of column state spill (668 to 884 bytes a thread: 4096x16384 BF16 324 for 119,
// 4096x12288 281 for 89; forward, 52 to 104 bytes, 116 for 79 and 101 for 60). The columns' sums (dW, dscale, dw_after) are kept in FP32 registers over the rows of a CTA, one
// partial row a CTA goes to the workspace, and a second kernel adds them in order (no atomics: the same bits every time).
// Row m belongs to partial m % parts, and parts is a function of the sizes alone, not of dg_set_num_sms.
//
// Tried and not kept: the forward pass over three rows at once (one barrier a row, R formed again for Y) 83 to 90 us; in teams of 32 warps
// an SM with the columns' vectors in shared memory, 115; rings of four to six rows, 85 to 86; one vector a thread and twice the threads
// for rows of 7168, backward 164 to 220 (64 registers a thread, spilled).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_scale.cuh"
#include "dg_vec.cuh"

namespace dg {

namespace {

// Sums of K values over the CTA, in a fixed order; every thread gets them. `red` holds 32 floats a value and is used by
// turns of two, so that one barrier a call is enough. In two parts: each warp's sums go to `red`, then behind the barrier to everyone.
template <int K>
__device__ __forceinline__ void warp_part(float (&v)[K], float (*red)[32]) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (threadIdx.x % 32 == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) red[k][threadIdx.x / 32] = v[k];
}
template <int K>
__device__ __forceinline__ void block_part(float (&v)[K], float (*red)[32], int warps) {
  if (warps == 1) return;
  const int lane = threadIdx.x % 32;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lane < warps ? red[k][lane] : 0.0f;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
}
template <int K>
__device__ __forceinline__ void block_sum(float (&v)[K], float (*red)[32], int warps) {
  warp_part(v, red);
  block_part(v, red, warps);
}

// Eight elements from column c of a row of n, two a register pair (the arithmetic is on pairs); zeros past the row's end.
using Eight = float2[4];
__device__ __forceinline__ void unpack(const uint4& w, Eight& v) {
  v[0] = make_float2(bf16_lo(w.x), bf16_hi(w.x));
  v[1] = make_float2(bf16_lo(w.y), bf16_hi(w.y));
  v[2] = make_float2(bf16_lo(w.z), bf16_hi(w.z));
  v[3] = make_float2(bf16_lo(w.w), bf16_hi(w.w));
}
template <bool VEC, typename T>
__device__ __forceinline__ void load8(const T* row, int c, int n, Eight& v) {
  if constexpr (!VEC) {
    float e[8];
    load8_part(row + c, n - c < 8 ? n - c : 8, e);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = make_float2(e[2 * j], e[2 * j + 1]);
  } else if constexpr (sizeof(T) == 2) {
    unpack(*reinterpret_cast<const uint4*>(row + c), v);
  } else {
    const float4 a = reinterpret_cast<const float4*>(row + c)[0], b = reinterpret_cast<const float4*>(row + c)[1];
    v[0] = make_float2(a.x, a.y), v[1] = make_float2(a.z, a.w), v[2] = make_float2(b.x, b.y), v[3] = make_float2(b.z, b.w);
  }
}
template <bool VEC, typename T>
__device__ __forceinline__ void put8(T* row, int c, int n, const Eight& v) {
  const float e[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
  if constexpr (VEC)
    store8(row + c, e);
  else
    store8_part(row + c, n - c < 8 ? n - c : 8, e);
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// ---------------------------------------------------------------------------------------------
// The rows of a CTA. Its inputs are copied ahead into a ring of `stages` rows in shared memory, each thread's columns to its own
// places (so no barrier guards them); with no stages (rows too long for it, or any alignment) they are read from the rows
// themselves. A thread's V vectors of eight columns are the same in every row, so what belongs to the columns stays in registers.
template <typename T>
__device__ __forceinline__ void copy_async(uint8_t* to, const T* from) {   // eight elements
#pragma unroll
  for (size_t o = 0; o < 8 * sizeof(T); o += 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(to + o)), "l"(reinterpret_cast<const uint8_t*>(from) + o)
                 : "memory");
}

template <typename T, bool VEC, int V, int INPUTS>
struct RowRing {
  uint8_t* mine;                 // this thread's first place
  const T* in[INPUTS];           // the matrices at this thread's first column, null where absent (no places of the ring then)
  int off[INPUTS];               // of each input's places in a stage, in bytes
  int stage_bytes = 0, stages, M, N, column0, column_step;
  int head = 0;                  // the current row's stage, in bytes

  __device__ __forceinline__ RowRing(uint8_t* ring, int stages, int M, int N)
      : mine(ring + threadIdx.x * (int)(8 * sizeof(T))), stages(stages), M(M), N(N), column0(threadIdx.x * 8), column_step(blockDim.x * 8) {}
  __device__ __forceinline__ void add(int k, const void* p) {
    in[k] = static_cast<const T*>(p);
    off[k] = stage_bytes;
    if (p) stage_bytes += V * column_step * (int)sizeof(T);
  }
  __device__ __forceinline__ int column(int i) const { return column0 + i * column_step; }
  __device__ __forceinline__ void fetch(long long m, int at) {
    if constexpr (VEC) {
      if (stages > 0 && m < M) {
        const size_t row = (size_t)m * N + column0;
#pragma unroll
        for (int k = 0; k < INPUTS; ++k) {
          if (!in[k]) continue;
          const T* from = in[k] + row;
          uint8_t* to = mine + at + off[k];
#pragma unroll
          for (int i = 0; i < V; ++i)
            if (column(i) < N) copy_async(to + i * column_step * (int)sizeof(T), from + i * column_step);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    }
  }
  __device__ __forceinline__ void begin(long long m, long long step) {
    head = 0;
    for (int s = 0; s < stages - 1; ++s) fetch(m + s * step, s * stage_bytes);
  }
  // The current row m's inputs are there; the row stages - 1 further on is asked for, into the stage that the row before has left.
  __device__ __forceinline__ void arrive(long long m, long long step) {
    if constexpr (VEC) {
      if (stages == 0) return;
      fetch(m + (stages - 1) * step, (head == 0 ? stages * stage_bytes : head) - stage_bytes);
      if (stages == 1) asm volatile("cp.async.wait_group 0;" ::: "memory");
      else if (stages == 2) asm volatile("cp.async.wait_group 1;" ::: "memory");
      else asm volatile("cp.async.wait_group 2;" ::: "memory");
    }
  }
  // The same while the row before m keeps its stage (three stages): the row after m is asked for instead.
  __device__ __forceinline__ void arrive_keeping(long long m, long long step) {
    if constexpr (VEC) {
      const int past = head + stage_bytes >= stages * stage_bytes ? 0 : head + stage_bytes;
      fetch(m + step, past);
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    }
  }
  __device__ __forceinline__ void leave() {
    head += stage_bytes;
    if (head >= stages * stage_bytes) head = 0;
  }
  __device__ __forceinline__ void end() {
    if constexpr (VEC) asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  // (`at`: the row's stage)
  __device__ __forceinline__ void get(int k, int i, long long m, int at, Eight& v) const {
    if (VEC && stages > 0)
      load8<true>(reinterpret_cast<const T*>(mine + at + off[k] + i * column_step * (int)sizeof(T)), 0, 8, v);
    else
      load8<VEC>(in[k] + (size_t)m * N, column(i), N, v);
  }
};

// Eight columns of a vector that may be absent: ones then, and zeros past the row's end.
template <bool VEC>
__device__ __forceinline__ void columns_of(const float* p, int c, int n, Eight& v) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = make_float2(c + 2 * j < n ? 1.0f : 0.0f, c + 2 * j + 1 < n ? 1.0f : 0.0f);
  if (p && c < n) load8<VEC>(p, c, n, v);
}
__device__ __forceinline__ float sum_of(const float2& v) { return v.x + v.y; }

// Forward. A CTA takes one row at a time, a thread V vectors of eight columns.
template <typename T, bool VEC, int V, bool UE>
__global__ void __launch_bounds__(V == 1 ? 128 : 512, V == 1 ? 8 : 1) norm_kernel(const NormArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][1][32];
  const int N = a.N, warps = blockDim.x / 32, tid = threadIdx.x;
  const float inv_n = 1.0f / (float)N;
  griddep_wait();
  griddep_launch_dependents();
  RowRing<T, VEC, V, 2> rows(ring, a.stages, a.M, N);
  rows.add(0, a.x);
  rows.add(1, a.b);
  rows.begin(blockIdx.x, gridDim.x);
  Eight after[V], before[V];   // w_after·scale, W
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int c = rows.column(i);
    if (a.b) {
      Eight sc;
      columns_of<VEC>(a.w_after, c, N, after[i]);
      columns_of<VEC>(a.scale, c, N, sc);
#pragma unroll
      for (int j = 0; j < 4; ++j) after[i][j] = __fmul2_rn(after[i][j], sc[j]);
    }
    columns_of<VEC>(a.w, c, N, before[i]);
  }
  int turn = 0;
  const float* const gate = a.b ? a.gate : nullptr;
  float gate_ahead = gate && (int)blockIdx.x < a.M ? gate[blockIdx.x] : 1.0f;   // the next row's, from L2 or farther
  for (long long m = blockIdx.x; m < a.M; m += gridDim.x) {
    const size_t at = (size_t)m * N;
    float f = gate_ahead;   // of the whole row
    if (gate && m + gridDim.x < a.M) gate_ahead = gate[m + gridDim.x];
    rows.arrive(m, gridDim.x);
    Eight r[V] = {};
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (rows.column(i) < N) rows.get(0, i, m, rows.head, r[i]);
    if (a.b) {
      Eight p[V] = {};
#pragma unroll
      for (int i = 0; i < V; ++i)
        if (rows.column(i) < N) rows.get(1, i, m, rows.head, p[i]);
      if (a.w_after) {
        float2 sq = both(0.0f);
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) sq = __ffma2_rn(p[i][j], p[i][j], sq);
        float s[1] = {sum_of(sq)};
        block_sum(s, red[turn], warps);
        turn ^= 1;
        const float ra = rsqrtf(fmaf(s[0], inv_n, a.eps));
        if (a.rstd_after && tid == 0) a.rstd_after[m] = ra;
        f *= ra;
      }
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = rows.column(i);
        if (c >= N) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) r[i][j] = __ffma2_rn(__fmul2_rn(p[i][j], after[i][j]), both(f), r[i][j]);
        if (a.r) put8<VEC>(static_cast<T*>(a.r) + at, c, N, r[i]);
      }
    }
    rows.leave();
    if (!a.w) continue;
    float2 sq = both(0.0f);
#pragma unroll
    for (int i = 0; i < V; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) sq = __ffma2_rn(r[i][j], r[i][j], sq);
    float s[1] = {sum_of(sq)};
    block_sum(s, red[turn], warps);
    turn ^= 1;
    const float rs = rsqrtf(fmaf(s[0], inv_n, a.eps));
    if (a.rstd && tid == 0) a.rstd[m] = rs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = rows.column(i);
      const bool live = c < N;
#pragma unroll
      for (int j = 0; j < 4; ++j) r[i][j] = __fmul2_rn(r[i][j], __fmul2_rn(both(rs), before[i][j]));
      if (live && a.y) put8<VEC>(static_cast<T*>(a.y) + at, c, N, r[i]);
      if (a.q) {   // sixteen lanes hold a group of 128; columns past N are zeros
        float top = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(r[i][j].x), fabsf(r[i][j].y)));
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (live) {
          float factor;
          uint32_t scale;
          group_scale<UE>(top, factor, scale);
          uint32_t q[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 v = __fmul2_rn(r[i][j], both(factor));
            q[j] = e4m3x2_satfinite(v.x, v.y);
          }
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
  rows.end();
}

// ---------------------------------------------------------------------------------------------
// Backward. Both dscale = w_after·t and dw_after = scale·t come from t = Σ_m gate·G·b̂, so two columns' sums are kept.
template <typename T, bool VEC, int V>
__global__ void __launch_bounds__(V == 1 ? 128 : 512, V == 1 ? 4 : 1) norm_backward_kernel(const NormBackwardArgs a) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ float red[2][3][32];
  enum { kDY, kR, kDR, kB };
  const int N = a.N, tid = threadIdx.x, warps = blockDim.x / 32;
  const float inv_n = 1.0f / (float)N;
  const bool dy = a.dy, dr = a.dr, b = a.b, along_b = b && (a.w_after || a.dgate);
  griddep_wait();
  griddep_launch_dependents();
  RowRing<T, VEC, V, 4> rows(ring, a.stages, a.M, N);
  rows.add(kDY, a.dy);
  rows.add(kR, a.r);
  rows.add(kDR, a.dr);
  rows.add(kB, a.b);
  Eight w[V], ws[V];   // W, w_after·scale
  for (int part = blockIdx.x; part < a.parts; part += gridDim.x) {   // (more than one only under dg_set_num_sms)
    rows.begin(part, a.parts);
    if (part == (int)blockIdx.x) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        Eight sc;
        columns_of<VEC>(a.w, rows.column(i), N, w[i]);
        columns_of<VEC>(a.w_after, rows.column(i), N, ws[i]);
        columns_of<VEC>(a.scale, rows.column(i), N, sc);
#pragma unroll
        for (int j = 0; j < 4; ++j) ws[i][j] = __fmul2_rn(ws[i][j], sc[j]);
      }
    }
    Eight sw[V] = {}, st[V] = {};   // Σ dY·x̂, Σ gate·G·b̂
    // Σ dY·W·R, Σ scale·P·(dR + r·dY·W), Σ scale·P·R of row m (r, ra where a whole sum has them: in `scalars`), this thread's part
    auto row_sums = [&](long long m, int at, float rs, float (&sums)[3]) {
      float2 two[3] = {};
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (rows.column(i) >= N) continue;
        Eight g = {}, x = {};
        if (dr) rows.get(kDR, i, m, at, g);
        if (dy) {
          Eight d;
          rows.get(kDY, i, m, at, d);
          rows.get(kR, i, m, at, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 gw = __fmul2_rn(d[j], w[i][j]);
            two[0] = __ffma2_rn(gw, x[j], two[0]);
            g[j] = __ffma2_rn(both(rs), gw, g[j]);
          }
        }
        if (along_b) {
          Eight p;
          rows.get(kB, i, m, at, p);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            p[j] = __fmul2_rn(p[j], ws[i][j]);
            two[1] = __ffma2_rn(p[j], g[j], two[1]);
            two[2] = __ffma2_rn(p[j], x[j], two[2]);
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 3; ++k) sums[k] = sum_of(two[k]);
    };
    struct Row {   // the scalars of a row
      float rs, ra, gate;
    };
    auto row_of = [&](long long m) { return Row{dy ? a.rstd[m] : 0.0f, a.w_after ? a.rstd_after[m] : 1.0f, a.gate ? a.gate[m] : 1.0f}; };
    auto gradients = [&](long long m, int at, const Row& row, const float (&sums)[3]) {
      const float rs = row.rs, ra = row.ra;
      const float c1 = sums[0] * rs * inv_n;                                                // mean(dY·W·x̂)
      const float along = ra * fmaf(-c1 * rs * rs, sums[2], sums[1]);                       // Σ scale·P·G
      if (a.dgate && tid == 0) a.dgate[m] = along;
      const float c2 = a.w_after ? row.gate * along * inv_n * ra * ra : 0.0f, k1 = c1 * rs; // (of B, of R)
      const float gra = row.gate * ra;
      const size_t to = (size_t)m * N;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int c = rows.column(i);
        if (c >= N) continue;
        Eight g = {}, p;
        if (dr) rows.get(kDR, i, m, at, g);
        if (dy) {
          Eight d, x;
          rows.get(kDY, i, m, at, d);
          rows.get(kR, i, m, at, x);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sw[i][j] = __ffma2_rn(__fmul2_rn(d[j], both(rs)), x[j], sw[i][j]);
            g[j] = __ffma2_rn(both(rs), __ffma2_rn(x[j], both(-k1), __fmul2_rn(d[j], w[i][j])), g[j]);
          }
        }
        if (b) rows.get(kB, i, m, at, p);   // (dX may be B)
        if (a.dx) put8<VEC>(static_cast<T*>(a.dx) + to, c, N, g);
        if (b) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 t = __fmul2_rn(both(gra), g[j]);
            st[i][j] = __ffma2_rn(t, p[j], st[i][j]);
            g[j] = __ffma2_rn(t, ws[i][j], __fmul2_rn(p[j], both(-c2)));
          }
          if (a.db) put8<VEC>(static_cast<T*>(a.db) + to, c, N, g);
        }
      }
    };
    const bool reduce = dy || along_b;
    float sums[3] = {0.0f, 0.0f, 0.0f};
    int turn = 0;
    if (rows.stages >= 3) {
      // One row's sums are formed beside the gradients of the row before, so the reduction's latency is behind those.
      // (its scalars, from L2 or farther, are asked for a row earlier still)
      const auto ahead_of = [&](long long m) { return row_of(m < a.M ? m : part); };
      Row row = row_of(part), then = ahead_of(part + a.parts);
      asm volatile("cp.async.wait_group 1;" ::: "memory");   // (of the two rows asked for)
      if (reduce) {
        row_sums(part, rows.head, row.rs, sums);
        block_sum(sums, red[turn], warps);
      }
      for (long long m = part; m < a.M; m += a.parts) {
        const long long next = m + a.parts;
        const int at = rows.head;
        const bool more = next < a.M;
        const Row later = ahead_of(next + a.parts);
        float more_sums[3] = {0.0f, 0.0f, 0.0f};
        rows.leave();
        if (more) {
          rows.arrive_keeping(next, a.parts);
          if (reduce) {
            turn ^= 1;
            row_sums(next, rows.head, then.rs, more_sums);
            warp_part(more_sums, red[turn]);
          }
        }
        gradients(m, at, row, sums);
        if (more && reduce) block_part(more_sums, red[turn], warps);
        row = then;
        then = later;
#pragma unroll
        for (int k = 0; k < 3; ++k) sums[k] = more_sums[k];
      }
    } else {
      for (long long m = part; m < a.M; m += a.parts, turn ^= 1) {
        const Row row = row_of(m);
        rows.arrive(m, a.parts);
        if (reduce) {
          row_sums(m, rows.head, row.rs, sums);
          block_sum(sums, red[turn], warps);
        }
        gradients(m, rows.head, row, sums);
        rows.leave();
      }
    }
    rows.end();
    // the workspace: [parts][sums kept][N]
    float* out = a.partial + (size_t)part * a.sums * N;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = rows.column(i);
      if (c >= N) continue;
      if (a.dw) put8<VEC>(out, c, N, sw[i]);
      if (a.dscale || a.dw_after) put8<VEC>(out + (size_t)(a.dw ? N : 0), c, N, st[i]);
    }
    __syncthreads();   // red is free for the next part
  }
}

// Adds the partial rows: a thread takes four columns of each kSumShares-th row, then the shares are added in order.
constexpr int kSumCols = 32, kSumShares = 64;
__global__ void __launch_bounds__(kSumCols / 4 * kSumShares) norm_sum_kernel(const NormBackwardArgs a) {
  __shared__ float share[kSumShares][kSumCols + 1];
  griddep_wait();
  griddep_launch_dependents();
  const int N = a.N, quad = threadIdx.x % (kSumCols / 4) * 4, row = threadIdx.x / (kSumCols / 4), blocks = (N + kSumCols - 1) / kSumCols;
  for (int block = blockIdx.x; block < blocks * a.sums; block += gridDim.x) {
    const int k = block / blocks, n = (block % blocks) * kSumCols + quad;
    float s[4] = {};
    if (n < N) {
      const float* p = a.partial + (size_t)k * N + n;
      if (N % 4 == 0) {
#pragma unroll 4
        for (int i = row; i < a.parts; i += kSumShares) {
          const float4 v = *reinterpret_cast<const float4*>(p + (size_t)i * a.sums * N);
          s[0] += v.x, s[1] += v.y, s[2] += v.z, s[3] += v.w;
        }
      } else {
        for (int i = row; i < a.parts; i += kSumShares)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if (n + j < N) s[j] += p[(size_t)i * a.sums * N + j];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) share[row][quad + j] = s[j];
    __syncthreads();
    const int col = threadIdx.x, at = (block % blocks) * kSumCols + col;
    if (col < kSumCols && at < N) {
      float v = 0.0f;
#pragma unroll
      for (int i = 0; i < kSumShares; ++i) v += share[i][col];
      if (k == 0 && a.dw) {
        a.dw[at] = v;
      } else {
        if (a.dscale) a.dscale[at] = a.w_after ? v * a.w_after[at] : v;
        if (a.dw_after) a.dw_after[at] = a.scale ? v * a.scale[at] : v;
      }
    }
    __syncthreads();
  }
}

int threads_for(int N, int V) { return ((N + 8 * V - 1) / (8 * V) + 31) / 32 * 32; }

bool all_aligned(std::initializer_list<const void*> ps) {
  uintptr_t bits = 0;
  for (const void* p : ps) bits |= reinterpret_cast<uintptr_t>(p);
  return bits % 16 == 0;
}

// How rows of N are laid out: vectors and threads of a CTA, CTAs an SM, and how many of them take the rows by turns.
// (152 SMs: those of the GPU that this is for; the sums' order depends on it, and so not on dg_set_num_sms.)
constexpr int kNormSms = 152, kRingBytes = 216 << 10;   // (the ring: of an SM, over its CTAs)
struct RowPlan {
  int V, threads, per_sm, parts;
};
// Two vectors a thread above 1024 columns: with one, 4099x2112 FP32 takes 20 us for 16 and the backward pass of 8192x2112 79 for 60.
RowPlan row_plan(int M, int N) {
  const int V = N <= 1024 ? 1 : N <= 8192 ? 2 : 4, threads = threads_for(N, V);
  const int fit = 512 / threads, per_sm = fit > 8 ? 8 : fit, parts = kNormSms * per_sm;
  return {V, threads, per_sm, M < parts ? M : parts};
}
int ring_stages(const RowPlan& p, bool vec, int inputs, size_t size, size_t* bytes) {
  const size_t stage = (size_t)p.threads * p.V * 8 * size * inputs, most = (size_t)kRingBytes / p.per_sm;
  const int stages = !vec ? 0 : 3 * stage <= most ? 3 : 2 * stage <= most ? 2 : stage <= most ? 1 : 0;
  *bytes = stages * stage;
  return stages;
}

// Launches a kernel of the plan's V, its shared-memory limit set on first use per device.
template <typename Kernel, typename Args>
cudaError_t launch_rows(Kernel kernel, bool (&configured)[64], const RowPlan& p, size_t smem, const StreamArgs& s, const Args& a) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes)) != cudaSuccess) return e;
    configured[dev] = true;
  }
  return launch_plain(kernel, (int)s.limit.all(p.parts), p.threads, smem, s, a);
}

template <typename F>
cudaError_t with_vectors(int V, F f) {
  return V == 1 ? f(std::integral_constant<int, 1>{}) : V == 2 ? f(std::integral_constant<int, 2>{}) : f(std::integral_constant<int, 4>{});
}

}  // namespace

long long norm_backward_floats(int M, int N, int sums) { return (long long)row_plan(M, N).parts * sums * N; }

cudaError_t launch_norm(NormArgs a, bool f32, bool ue8m0, const StreamArgs& s) {
  const bool vec = a.N % 8 == 0 && all_aligned({a.x, a.b, a.r, a.y, a.w, a.w_after, a.scale});
  const RowPlan plan = row_plan(a.M, a.N);
  size_t smem;
  a.stages = ring_stages(plan, vec, a.b ? 2 : 1, f32 ? 4 : 2, &smem);
  return with_vectors(plan.V, [&](auto v) {
    auto go = [&](auto one, auto vector, auto ue) {
      constexpr int V = decltype(v)::value;
      static bool configured[64] = {};
      return launch_rows(norm_kernel<decltype(one), decltype(vector)::value, V, decltype(ue)::value>, configured, plan, smem, s, a);
    };
    auto scales = [&](auto one, auto vector) { return a.q && ue8m0 ? go(one, vector, std::true_type{}) : go(one, vector, std::false_type{}); };
    auto type = [&](auto vector) { return f32 ? scales(0.0f, vector) : scales(__nv_bfloat16{}, vector); };
    return vec ? type(std::true_type{}) : type(std::false_type{});
  });
}

cudaError_t launch_norm_backward(NormBackwardArgs a, bool f32, const StreamArgs& s) {
  const bool vec = a.N % 8 == 0 && all_aligned({a.dy, a.dr, a.r, a.b, a.dx, a.db, a.w, a.w_after, a.scale, a.partial});
  const RowPlan plan = row_plan(a.M, a.N);
  size_t smem;
  a.stages = ring_stages(plan, vec, (a.dy ? 2 : 0) + (a.dr ? 1 : 0) + (a.b ? 1 : 0), f32 ? 4 : 2, &smem);
  a.parts = plan.parts;
  a.sums = (a.dw ? 1 : 0) + (a.dscale || a.dw_after ? 1 : 0);
  cudaError_t e = with_vectors(plan.V, [&](auto v) {
    auto go = [&](auto one, auto vector) {
      constexpr int V = decltype(v)::value;
      static bool configured[64] = {};
      return launch_rows(norm_backward_kernel<decltype(one), decltype(vector)::value, V>, configured, plan, smem, s, a);
    };
    auto type = [&](auto vector) { return f32 ? go(0.0f, vector) : go(__nv_bfloat16{}, vector); };
    return vec ? type(std::true_type{}) : type(std::false_type{});
  });
  if (e != cudaSuccess || a.sums == 0) return e;
  const int blocks = (a.N + kSumCols - 1) / kSumCols * a.sums;
  return launch_plain(norm_sum_kernel, (int)s.limit.all(blocks), kSumCols / 4 * kSumShares, 0, s, a);
}

}  // namespace dg
