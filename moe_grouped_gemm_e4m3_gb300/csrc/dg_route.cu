// dg_route.cu — the router: k experts of each token from its E logits, and the gradient of their weights.
//
// Scores s: softmax over the E logits, or the sigmoid of each. Selected are the k largest of s + bias (without a bias: of
// the logits themselves, which order the same way and have no rounding), ties to the lowest index, in descending order.
//     w_i = f·s_i                     or, normalised again,  w_i = f·s_i / S,  S = Σ_selected s + 1e-20
// Backward, with dw' = f·dw:  ds_i = dw'_i   or   (dw'_i − Σ_j dw'_j s_j / S) / S,  zero elsewhere;
//     dl_e = s_e (ds_e − Σ s ds)  (softmax)   or   ds_e s_e (1 − s_e)  (sigmoid).
//
// A score next to the border of the k-th is settled in FP64: FP32 scores within 4e-6 of a round's best are within their
// rounding of it, so those candidates (rarely any) are computed again, and the selection is that of the exact scores
// whatever exp's last bits are. Logits that are NaN or -inf, and biases of -inf, are never selected; a token
// with fewer than k others gets the index -1 and the weight 0 in the places left.
//
// One warp a token, E/32 logits a lane in registers. A round of the selection is two warp reductions (the largest key as an
// ordered integer, the lowest index that has it).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_vec.cuh"

namespace dg {

namespace {

constexpr int kWarps = 4;
constexpr float kNear = 4e-6f;

// Larger floats have larger integers; what is never selected has 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  if (!(x > -INFINITY)) return 0;
  const uint32_t b = __float_as_uint(x);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The scores of a lane's logits (index j·32 + lane), NaN and -inf scoring 0. Softmax: also the row's largest logit and sum.
template <int VPL>
__device__ __forceinline__ void scores(const float (&l)[VPL], bool sigmoid, float (&s)[VPL], float& top) {
  if (sigmoid) {
    top = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) s[j] = l[j] > -INFINITY ? 1.0f / (1.0f + expf(-l[j])) : 0.0f;
    return;
  }
  uint32_t best = 0;
#pragma unroll
  for (int j = 0; j < VPL; ++j) best = max(best, ordered(l[j]));
  top = unordered(__reduce_max_sync(0xffffffffu, best));
  float sum = 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    s[j] = l[j] > -INFINITY ? expf(l[j] - top) : 0.0f;
    sum += s[j];
  }
  sum = warp_sum(sum);
  const float f = sum > 0.0f ? 1.0f / sum : 0.0f;
#pragma unroll
  for (int j = 0; j < VPL; ++j) s[j] *= f;
}

template <int VPL, typename T>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, float (&l)[VPL]) {
#pragma unroll
  for (int j = 0; j < VPL; ++j) l[j] = j * 32 + lane < E ? to_f32(row[j * 32 + lane]) : -INFINITY;
}

// The best of the candidates (bit j of a lane: index j·32 + lane) by their exact scores. `total` is the softmax's exact sum,
// or 0 while no round of this token has asked for it. Rare, so out of line and with the logits read again.
template <typename T>
__device__ __noinline__ int settle(const T* row, const float* bias, int E, uint32_t near, int lane, bool sigmoid, float top, double& total) {
  if (!sigmoid && total == 0.0) {
    double part = 0.0;
    for (int e = lane; e < E; e += 32)
      if (to_f32(row[e]) > -INFINITY) part += exp((double)to_f32(row[e]) - (double)top);
    total = warp_sum(part);
  }
  double most = -INFINITY;
  int winner = INT32_MAX;
  for (; near; near &= near - 1) {
    const int e = (__ffs(near) - 1) * 32 + lane;
    const double l = (double)to_f32(row[e]), v = (sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / total) + (double)bias[e];
    if (v > most || winner == INT32_MAX) most = v, winner = e;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double v = __shfl_xor_sync(0xffffffffu, most, o);
    const int e = __shfl_xor_sync(0xffffffffu, winner, o);
    if (e != INT32_MAX && (winner == INT32_MAX || v > most || (v == most && e < winner))) most = v, winner = e;
  }
  return winner;
}

template <typename T, int VPL>
__global__ void __launch_bounds__(32 * kWarps) route_kernel(const RouteArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  for (long long t = (long long)blockIdx.x * kWarps + threadIdx.x / 32; t < a.T; t += (long long)gridDim.x * kWarps) {
    float l[VPL], s[VPL], top;
    const T* row = static_cast<const T*>(a.logits) + t * a.E;
    load_logits(row, a.E, lane, l);
    scores(l, a.sigmoid, s, top);
    uint32_t key[VPL];
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
      const int e = j * 32 + lane;
      key[j] = ordered(!a.bias ? l[j] : e < a.E && l[j] > -INFINITY ? s[j] + a.bias[e] : -INFINITY);
    }
    double total = 0.0;   // softmax: the exact sum, once a near tie asks for it
    int mine = -1;        // lane i keeps the i-th choice
    float weight = 0.0f;
    for (int i = 0; i < a.k; ++i) {
      uint32_t best = 0;
#pragma unroll
      for (int j = 0; j < VPL; ++j) best = max(best, key[j]);
      best = __reduce_max_sync(0xffffffffu, best);
      if (best == 0) break;
      int winner = INT32_MAX;
#pragma unroll
      for (int j = VPL - 1; j >= 0; --j)
        if (key[j] == best) winner = j * 32 + lane;
      winner = (int)__reduce_min_sync(0xffffffffu, (unsigned)winner);
      if (a.bias) {
        const float b = unordered(best);
        const uint32_t border = max(1u, ordered(b - kNear * fmaxf(1.0f, fabsf(b))));
        uint32_t near = 0;   // bit j
#pragma unroll
        for (int j = 0; j < VPL; ++j) near |= (key[j] >= border ? 1u : 0u) << j;
        const int others = __popc(near) - (winner % 32 == lane ? 1 : 0);
        if (__any_sync(0xffffffffu, others > 0)) winner = settle(row, a.bias, a.E, near, lane, a.sigmoid, top, total);
      }
      float w = 0.0f;
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j * 32 + lane == winner) {
          w = s[j];
          key[j] = 0;
        }
      w = __shfl_sync(0xffffffffu, w, winner % 32);
      if (lane == i) mine = winner, weight = w;
    }
    if (a.renorm) weight = weight / (warp_sum(weight) + 1e-20f);
    if (lane < a.k) {
      a.ids[t * a.k + lane] = mine;
      a.weights[t * a.k + lane] = weight * a.factor;
    }
  }
}

template <typename T, int VPL>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(const RouteArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  for (long long t = (long long)blockIdx.x * kWarps + threadIdx.x / 32; t < a.T; t += (long long)gridDim.x * kWarps) {
    float l[VPL], s[VPL], top;
    load_logits(static_cast<const T*>(a.logits) + t * a.E, a.E, lane, l);
    int e = lane < a.k ? a.ids[t * a.k + lane] : -1;
    if (e >= a.E) e = -1;
    float d = e >= 0 ? a.factor * a.dweights[t * a.k + lane] : 0.0f;
    scores(l, a.sigmoid, s, top);
    float ds[VPL] = {};
    if (a.renorm) {
      float sel = 0.0f;   // the score of this lane's choice
      for (int i = 0; i < a.k; ++i) {
        const int at = __shfl_sync(0xffffffffu, e, i);
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
          if (at == j * 32 + lane) v = s[j];
        v = __shfl_sync(0xffffffffu, v, at & 31);
        if (lane == i && at >= 0) sel = v;
      }
      const float total = warp_sum(sel) + 1e-20f, mean = warp_sum(d * sel) / total;
      d = e >= 0 ? (d - mean) / total : 0.0f;
    }
    for (int i = 0; i < a.k; ++i) {
      const int at = __shfl_sync(0xffffffffu, e, i);
      const float v = __shfl_sync(0xffffffffu, d, i);
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (at == j * 32 + lane) ds[j] += v;
    }
    float along = 0.0f;
    if (!a.sigmoid) {
#pragma unroll
      for (int j = 0; j < VPL; ++j) along = fmaf(s[j], ds[j], along);
      along = warp_sum(along);
    }
    T* out = static_cast<T*>(a.dlogits) + t * a.E;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (j * 32 + lane < a.E) store_f32(out + j * 32 + lane, a.sigmoid ? ds[j] * s[j] * (1.0f - s[j]) : s[j] * (ds[j] - along));
  }
}

template <typename T, int VPL>
cudaError_t launch_one(const RouteArgs& a, bool backward, const StreamArgs& s) {
  const int grid = (int)s.limit.all((a.T + kWarps - 1) / kWarps);
  return launch_plain(backward ? route_backward_kernel<T, VPL> : route_kernel<T, VPL>, grid, 32 * kWarps, 0, s, a);
}

template <typename T>
cudaError_t launch_typed(const RouteArgs& a, bool backward, const StreamArgs& s) {
  if (a.E <= 64) return launch_one<T, 2>(a, backward, s);
  if (a.E <= 128) return launch_one<T, 4>(a, backward, s);
  if (a.E <= 256) return launch_one<T, 8>(a, backward, s);
  if (a.E <= 512) return launch_one<T, 16>(a, backward, s);
  return launch_one<T, 32>(a, backward, s);
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, bool bf16, bool backward, const StreamArgs& s) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, backward, s) : launch_typed<float>(a, backward, s);
}

}  // namespace dg
