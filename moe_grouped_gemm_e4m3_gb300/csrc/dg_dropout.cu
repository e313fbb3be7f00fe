// dg_dropout.cu — dropout from a counter-based generator, with the residual sum.
//
//   Y[i] = R[i] + (kept(i) ? X[i] / q : 0),   q = 1 - T / 65536 the exact keep probability
//
// computed in FP32 (product, then sum) and rounded once. R may be absent. The mask (dg_philox.cuh)
// is a function of the seed, the offset and i, so the backward pass is the same call on dY without R.
//
// One thread takes eight consecutive elements (16 bytes of BF16, 32 of FP32) per counter.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_vec.cuh"

namespace dg {

namespace {

constexpr int kThreads = 256;

// VEC: X, R and Y are 16-byte aligned; otherwise every access is one element (any alignment that the
// element type allows).
template <typename T, bool VEC, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const T* x, const T* r, T* y, const Dropout d, long long n) {
  griddep_wait();
  griddep_launch_dependents();
  const long long groups = (n + 7) / 8;
  const long long step = (long long)gridDim.x * kThreads;
  const bool drop = d.threshold != 0;
  const Philox gen = drop ? Philox(d.rng) : Philox();
  for (long long i = (long long)blockIdx.x * kThreads + threadIdx.x; i < groups; i += step) {
    float v[8], add[8];
    const int live = (int)(n - i * 8 < 8 ? n - i * 8 : 8);
    const bool whole = VEC && live == 8;
    if (whole) {
      load8(x + i * 8, v);
      if constexpr (RES) load8(r + i * 8, add);
    } else {
      load8_part(x + i * 8, live, v);
      if constexpr (RES) load8_part(r + i * 8, live, add);
    }
    if (drop) dropout8(v, gen((uint64_t)i), d.threshold, d.scale);
    if constexpr (RES) {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fadd_rn(add[j], v[j]);
    }
    if (whole)
      store8(y + i * 8, v);
    else
      store8_part(y + i * 8, live, v);
  }
}

template <typename T>
cudaError_t launch_typed(const void* x, const void* r, void* y, const Dropout& d, long long n, const StreamArgs& s) {
  const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(r) | reinterpret_cast<uintptr_t>(y)) % 16) == 0;
  const long long blocks = ((n + 7) / 8 + kThreads - 1) / kThreads, most = 8LL * s.sms;
  const int grid = (int)(blocks < most ? blocks : most);
  auto go = [&](auto kernel) {
    return launch_plain(kernel, grid, kThreads, 0, s, static_cast<const T*>(x), static_cast<const T*>(r), static_cast<T*>(y), d, n);
  };
  if (r) return vec ? go(dropout_kernel<T, true, true>) : go(dropout_kernel<T, false, true>);
  return vec ? go(dropout_kernel<T, true, false>) : go(dropout_kernel<T, false, false>);
}

}  // namespace

cudaError_t launch_dropout(const void* x, const void* r, void* y, bool f32, const Dropout& d, long long n, const StreamArgs& s) {
  return f32 ? launch_typed<float>(x, r, y, d, n, s) : launch_typed<__nv_bfloat16>(x, r, y, d, n, s);
}

}  // namespace dg
