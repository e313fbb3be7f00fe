// dg_dropout.cu — dropout from a counter-based generator, with the residual sum.
//
//   Y[i] = R[i] + (kept(i) ? X[i] / q : 0),   q = 1 - T / 65536 the exact keep probability
//
// computed in FP32 (product, then sum) and rounded once. R may be absent. The mask (dg_philox.cuh)
// is a function of the seed, the offset and i, so the backward pass is the same call on dY without R.
//
// One counter serves eight consecutive elements (16 bytes of BF16, 32 of FP32). Bound by HBM, in one pass of the grid: a
// resident grid that loops takes 118 us where one pass takes 106 (117M BF16 elements with a residual, 6.7 TB/s), and 82 where it
// takes 67 (59M FP32 without). A large tensor takes GROUPS such eights a thread, all loads ahead of the generator's
// arithmetic, except BF16 with a residual, whose two loads a group are enough in flight (us at 1 group and at
// several; 117M BF16 and 59M FP32 elements): BF16 without a residual 80 and 73, with one 106 and 112; FP32 67.8 and 67.4, with
// one 98.9 and 97.9.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_vec.cuh"

namespace dg {

namespace {

constexpr int kThreads = 256;

// Eight elements as they are in memory.
template <typename T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 a;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { a = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float (&v)[8]) const { unpack8(a, v); }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};

template <bool RES>
__device__ __forceinline__ void drop_and_add(float (&v)[8], const float (&add)[8], const Philox& gen, long long i, const Dropout& d) {
  if (d.threshold) dropout8(v, gen((uint64_t)i), d.threshold, d.scale);
  if constexpr (RES) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(add[j], v[j]);
  }
}

// VEC: X, R and Y are 16-byte aligned; otherwise every access is one element (any alignment that the
// element type allows). CAPPED: a grid of fewer CTAs (dg_set_num_sms) that loops.
template <typename T, bool VEC, bool RES, int GROUPS, bool CAPPED>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const T* x, const T* r, T* y, const Dropout d, long long n) {
  griddep_wait();
  griddep_launch_dependents();
  const Philox gen = d.threshold ? Philox(d.rng) : Philox();
  auto pass = [&](long long first) {
    Eight<T> xs[GROUPS], rs[GROUPS];
    if constexpr (VEC) {
#pragma unroll
      for (int k = 0; k < GROUPS; ++k) {
        const long long i = first + k * kThreads;
        if (i * 8 + 8 > n) continue;
        xs[k].load(x + i * 8);
        if constexpr (RES) rs[k].load(r + i * 8);
      }
    }
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const long long i = first + k * kThreads;
      if (i * 8 >= n) return;
      float v[8], add[8];
      if (VEC && i * 8 + 8 <= n) {
        xs[k].values(v);
        if constexpr (RES) rs[k].values(add);
        drop_and_add<RES>(v, add, gen, i, d);
        store8(y + i * 8, v);
      } else {   // unaligned tensors, and the last, partial eight
        const int live = (int)(n - i * 8 < 8 ? n - i * 8 : 8);
        load8_part(x + i * 8, live, v);
        if constexpr (RES) load8_part(r + i * 8, live, add);
        drop_and_add<RES>(v, add, gen, i, d);
        store8_part(y + i * 8, live, v);
      }
    }
  };
  const long long first = (long long)blockIdx.x * (kThreads * GROUPS) + threadIdx.x;
  if constexpr (CAPPED) {
    for (long long i = first; i * 8 < n; i += (long long)gridDim.x * (kThreads * GROUPS)) pass(i);
  } else {
    pass(first);
  }
}

template <typename T, bool VEC, bool RES>
cudaError_t launch_shape(const T* x, const T* r, T* y, const Dropout& d, long long n, const StreamArgs& s) {
  // several groups a thread once they still fill every SM four times over (BF16 with a residual: one, see above)
  constexpr int kGroups = sizeof(T) == 2 ? 4 : 2;
  const long long eights = (n + 7) / 8;
  auto go = [&](auto kernel, auto capped, int groups) {
    const long long per = (long long)kThreads * groups, blocks = (eights + per - 1) / per, grid = s.limit.all(blocks);
    return launch_plain(grid < blocks ? capped : kernel, (int)grid, kThreads, 0, s, x, r, y, d, n);
  };
  if constexpr (VEC && !(RES && sizeof(T) == 2))
    if (eights >= 4LL * s.limit.sms * kThreads * kGroups)
      return go(dropout_kernel<T, VEC, RES, kGroups, false>, dropout_kernel<T, VEC, RES, kGroups, true>, kGroups);
  return go(dropout_kernel<T, VEC, RES, 1, false>, dropout_kernel<T, VEC, RES, 1, true>, 1);
}

template <typename T>
cudaError_t launch_typed(const void* x, const void* r, void* y, const Dropout& d, long long n, const StreamArgs& s) {
  const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(r) | reinterpret_cast<uintptr_t>(y)) % 16) == 0;
  auto go = [&](auto launch) { return launch(static_cast<const T*>(x), static_cast<const T*>(r), static_cast<T*>(y), d, n, s); };
  if (r) return vec ? go(launch_shape<T, true, true>) : go(launch_shape<T, false, true>);
  return vec ? go(launch_shape<T, true, false>) : go(launch_shape<T, false, false>);
}

}  // namespace

cudaError_t launch_dropout(const void* x, const void* r, void* y, bool f32, const Dropout& d, long long n, const StreamArgs& s) {
  return f32 ? launch_typed<float>(x, r, y, d, n, s) : launch_typed<__nv_bfloat16>(x, r, y, d, n, s);
}

}  // namespace dg
