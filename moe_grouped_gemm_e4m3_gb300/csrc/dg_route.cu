// dg_route.cu — the router: k experts of each token from its E logits, and the gradient of their weights.
//
// Scores s: softmax over the E logits, or the sigmoid of each. Selected are the k largest of s + bias (without a bias: of
// the logits themselves, which order the same way and have no rounding), ties to the lowest index, in descending order.
//     w_i = f·s_i                     or, normalised again,  w_i = f·s_i / S,  S = Σ_selected s + 1e-20
// Backward, with dw' = f·dw:  ds_i = dw'_i   or   (dw'_i − Σ_j dw'_j s_j / S) / S,  zero elsewhere;
//     dl_e = s_e (ds_e − Σ s ds)  (softmax)   or   ds_e s_e (1 − s_e)  (sigmoid; 1 − s(l) = s(−l)).
//
// The selection is that of the exact scores: choices that FP32 does not tell apart are compared in FP64, so it does not depend on
// whatever exp's last bits are. Logits that are NaN or -inf, and biases of -inf, are never selected; a token
// with fewer than k others gets the index -1 and the weight 0 in the places left.
//
// One warp a token, E/32 logits a lane in registers. The selection runs on keys as ordered integers whose last bits are cut off
// for the index, so that one number tells both: a lane sorts its own, and a round is one warp-wide maximum of the lanes' first
// and a step of the lane that had it (four times fewer instructions than keys and indexes by themselves). It goes one round
// further than k, so that wherever the cut bits (or a bias's rounding) could matter two neighbours of the sorted k + 1 are near each
// other. Then (1 to 3% of the tokens) the rounds go on until the last one is near no other, the lanes form their choices' whole keys and
// change places; what those do not tell apart is compared exactly. A warp that is late is what the whole call waits for, so this way is
// short: with the rounds made again from whole keys instead, which only lists longer than a warp get now, 16384x256 took 17.3 us for 13.6,
// 8192x512 (softmax) 38.6 for 23.3 (six sets of inputs in turn). The weights are computed from the selected logits by one lane each. In the
// backward pass every logit's gradient but the selected ones' is −s·Σ s ds (or zero), so these are stored as if none were selected, and
// the k lanes of the selected store theirs behind them.
//
// Bound by its instructions (667 a token of 256 experts with a bias, 537 without): 16384x256 sigmoid scores with a bias 12.5 us,
// where the read takes 2.6; backward of 16381x160 softmax scores 7 to 9 us (3.2).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_vec.cuh"

namespace dg {

namespace {

constexpr int kWarps = 4;
// How near keys may be in FP32 and be told apart. A sigmoid by the fast exponential and division is within 4e-7 of itself, one by expf and
// a division within 1.8e-7 (3.6e-7 of its value). A softmax's scores have one sum of exponentials (up to ten additions one behind the
// other, expf's 2.4e-7, a division, and the distances' rounding below, at most 2.6e-7 of the sum of 1024: 1.2e-6 of the score, in both
// alike, so of their difference). Each has an expf and a product (3.1e-7), and its logit's distance to the largest is rounded before
// (6e-8 of the distance, which is so much of the score: scores 18 below the largest were told apart that were not so). No score is larger
// than that of the largest logit, 1 / Σ exp(l - largest), and what is d below it e^d smaller. A sum with a bias rounds by 6e-8 of it.
constexpr float kNearFastSigmoid = 1.2e-6f, kNearSoftmax = 2e-6f, kNearSum = 1.3e-7f;   // of two keys, and of the larger one
// Of each score, of a softmax's with its distance to the largest logit; of each bias (a step of FP64: where the sums tie there, they tie,
// although FP32 may know which score is the larger one: equal biases of scores below 1e-16 of them); of the two scores' and their biases'
// differences; and where scores have no FP32 numbers.
constexpr float kNearOwn = 3.8e-7f, kNearDistance = 6e-8f, kNearBias = 2.3e-16f, kNearDifference = 1.4e-6f, kNearBiases = 1.3e-7f, kNearTiny = 1e-38f;

// Larger floats have larger integers, from 2^23 on; what is never selected (NaN, -inf, not `some`) has 0.
__device__ __forceinline__ uint32_t ordered(float x, bool some = true) {
  const uint32_t b = __float_as_uint(x);
  return some && x > -INFINITY ? b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u) : 0u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

template <typename V>
__device__ __forceinline__ V warp_sum(V v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ float sigmoid(float x) { return x > -INFINITY ? 1.0f / (1.0f + expf(-x)) : 0.0f; }   // (NaN: 0 too)

// A lane's logits: of every 128 four neighbours (QUADS: E a multiple of four, rows that start on 16 bytes, BF16 on 8), or every 32nd.
template <bool QUADS>
__device__ __forceinline__ int expert_of(int j, int lane) {
  return QUADS ? (j >> 2) * 128 + lane * 4 + (j & 3) : j * 32 + lane;
}
template <bool QUADS, int VPL, typename T>
__device__ __forceinline__ void load_logits(const T* row, int E, int lane, float (&l)[VPL]) {
  if constexpr (QUADS) {
#pragma unroll
    for (int j = 0; j < VPL; j += 4) {
      const int e = expert_of<true>(j, lane);
      if (e < E) {
        if constexpr (sizeof(T) == 4) {
          const float4 v = *reinterpret_cast<const float4*>(row + e);
          l[j] = v.x, l[j + 1] = v.y, l[j + 2] = v.z, l[j + 3] = v.w;
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(row + e);
          l[j] = bf16_lo(v.x), l[j + 1] = bf16_hi(v.x), l[j + 2] = bf16_lo(v.y), l[j + 3] = bf16_hi(v.y);
        }
      } else {
        l[j] = l[j + 1] = l[j + 2] = l[j + 3] = -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < VPL; ++j) l[j] = j * 32 + lane < E ? to_f32(row[j * 32 + lane]) : -INFINITY;
  }
}

// The softmax of a row: its largest logit and 1 / Σ exp(l - largest) (0 where there is none); NaN and -inf count as nothing.
struct Softmax {
  float top, inverse;
  __device__ __forceinline__ float operator()(float l) const { return l > -INFINITY ? expf(l - top) * inverse : 0.0f; }
};
// (exps: those of the lane's logits, for whoever wants them all)
template <int VPL>
__device__ __forceinline__ Softmax softmax_of(const float (&l)[VPL], float (&exps)[VPL]) {
  float best = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPL; ++j) best = fmaxf(best, l[j]);   // (a NaN is passed over)
  Softmax s;
  s.top = unordered(__reduce_max_sync(0xffffffffu, ordered(best)));
  float part[VPL];
#pragma unroll
  for (int j = 0; j < VPL; ++j) part[j] = exps[j] = l[j] > -INFINITY ? expf(l[j] - s.top) : 0.0f;
#pragma unroll
  for (int w = VPL / 2; w > 0; w /= 2)
#pragma unroll
    for (int j = 0; j < w; ++j) part[j] += part[j + w];
  const float sum = warp_sum(part[0]);
  s.inverse = sum == 0.0f ? 0.0f : 1.0f / sum;
  return s;
}

// The keys of a lane's logits, as ordered integers; 0 for what is never selected. (Their errors are far below the near ones'
// distance: the fast exponential's counts by s(1 - s), the reciprocal's by s.)
template <bool QUADS, int VPL>
__device__ __forceinline__ void keys_of(const RouteArgs& a, const Softmax& soft, const float (&l)[VPL], const float (&exps)[VPL], int lane,
                                        uint32_t (&key)[VPL]) {
  if (!a.bias) {
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = ordered(l[j] + 0.0f);   // (-0 ties with 0)
    return;
  }
  float b[VPL];
  load_logits<QUADS>(a.bias, a.E, lane, b);   // (-inf past the end)
#pragma unroll
  for (int j = 0; j < VPL; ++j) {
    float s;
    if (a.sigmoid)
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.0f + __expf(-l[j])));
    else
      s = exps[j] * soft.inverse;
    key[j] = ordered(s + b[j], l[j] > -INFINITY);
  }
}

// Sorts a lane's numbers, the largest first (odd-even merge: Batcher, "Sorting networks and their applications", 1968).
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&v)[N]) {
#pragma unroll
  for (int p = 1; p < N; p <<= 1)
#pragma unroll
    for (int k = p; k >= 1; k >>= 1)
#pragma unroll
      for (int j = k % p; j + k < N; j += 2 * k)
#pragma unroll
        for (int i = 0; i < k; ++i)
          if (i + j + k < N && (i + j) / (2 * p) == (i + j + k) / (2 * p)) {
            const uint32_t hi = max(v[i + j], v[i + j + k]), lo = min(v[i + j], v[i + j + k]);
            v[i + j] = hi, v[i + j + k] = lo;
          }
}

// The best of the candidates (bit j of a lane) by their exact scores. `total` is the softmax's exact sum, or 0 while no round of
// this token has asked for it. Rare, so out of line and with the logits read again.
template <bool QUADS, typename T>
__device__ __noinline__ int settle(const T* row, const float* bias, int E, uint32_t near, int lane, bool is_sigmoid, float top, double& total) {
  if (!is_sigmoid && total == 0.0) {
    double part = 0.0;
    for (int e = lane; e < E; e += 32)
      if (to_f32(row[e]) > -INFINITY) part += exp((double)to_f32(row[e]) - (double)top);
    total = warp_sum(part);
  }
  double most = -INFINITY;
  int winner = INT32_MAX;
  for (; near; near &= near - 1) {
    const int e = expert_of<QUADS>(__ffs(near) - 1, lane);
    const double l = (double)to_f32(row[e]), v = (is_sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)top) / total) + (double)bias[e];
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

// The exact score of each lane's choice.
template <typename T>
__device__ __noinline__ double exact_score(const T* row, int E, int choice, int lane, bool is_sigmoid, float top) {
  const double l = choice >= 0 ? (double)to_f32(row[choice]) : 0.0;
  if (is_sigmoid) return 1.0 / (1.0 + exp(-l));
  double total = 0.0;
  for (int e = lane; e < E; e += 32)
    if (to_f32(row[e]) > -INFINITY) total += exp((double)to_f32(row[e]) - (double)top);
  return exp(l - (double)top) / warp_sum(total);
}

// The selection with whole keys, for tokens with more near ones than lanes: lane i's choice. Out of line; the logits are read again.
template <int VPL, bool QUADS, typename T>
__device__ __noinline__ int select_carefully(const RouteArgs& a, const T* row, const Softmax& soft, int lane) {
  const float near = a.sigmoid ? kNearFastSigmoid : kNearSoftmax * soft.inverse;
  float l[VPL], exps[VPL] = {};
  load_logits<QUADS>(row, a.E, lane, l);
  if (!a.sigmoid)
#pragma unroll
    for (int j = 0; j < VPL; ++j) exps[j] = l[j] > -INFINITY ? expf(l[j] - soft.top) : 0.0f;
  uint32_t key[VPL];
  keys_of<QUADS>(a, soft, l, exps, lane, key);
  double total = 0.0;
  int mine = -1;
  for (int i = 0; i < a.k; ++i) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) best = max(best, key[j]);
    best = __reduce_max_sync(0xffffffffu, best);
    if (best == 0) break;
    const float c = unordered(best);
    const uint32_t border = a.bias ? max(1u, ordered(c - fmaf(kNearSum, fabsf(c), near))) : best;
    uint32_t candidates = 0;
#pragma unroll
    for (int j = 0; j < VPL; ++j) candidates |= (key[j] >= border ? 1u : 0u) << j;
    // (a lane's experts ascend with j, so its first candidate is its lowest)
    int winner = (int)__reduce_min_sync(0xffffffffu, candidates ? (unsigned)expert_of<QUADS>(__ffs(candidates) - 1, lane) : (unsigned)INT32_MAX);
    const uint32_t lanes = __ballot_sync(0xffffffffu, candidates != 0);
    if (a.bias && ((lanes & (lanes - 1)) || __any_sync(0xffffffffu, candidates & (candidates - 1))))
      winner = settle<QUADS>(row, a.bias, a.E, candidates, lane, a.sigmoid, soft.top, total);
#pragma unroll
    for (int j = 0; j < VPL; ++j)
      if (expert_of<QUADS>(j, lane) == winner) key[j] = 0;
    if (lane == i) mine = winner;
  }
  return mine;
}

template <typename T, int VPL, bool QUADS>
__global__ void __launch_bounds__(32 * kWarps, VPL <= 8 ? 8 : 1) route_kernel(const RouteArgs a) {
  constexpr uint32_t kIndex = VPL * 32 - 1;   // the bits of a key that its index takes
  const int rounds = a.k < a.E ? a.k + 1 : a.k;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  for (unsigned t = blockIdx.x * kWarps + threadIdx.x / 32; t < (unsigned)a.T; t += gridDim.x * kWarps) {   // (T and the step: below 2^31 each)
    const T* row = static_cast<const T*>(a.logits) + (size_t)t * (unsigned)a.E;
    const size_t to = (size_t)t * (unsigned)a.k + lane;
    float l[VPL];
    load_logits<QUADS>(row, a.E, lane, l);
    Softmax soft{};
    float exps[VPL] = {};
    if (!a.sigmoid) soft = softmax_of(l, exps);
    uint32_t key[VPL];
    keys_of<QUADS>(a, soft, l, exps, lane, key);
#pragma unroll
    for (int j = 0; j < VPL; ++j) key[j] = (key[j] & ~kIndex) | (kIndex - expert_of<QUADS>(j, lane));   // (the lower index is the larger number; of none, up to kIndex)
    sort_descending(key);
    uint32_t mine = 0, top = 0;   // lane i keeps the i-th
    auto round = [&](int i) {
      top = __reduce_max_sync(0xffffffffu, key[0]);
      if (key[0] == top) {
#pragma unroll
        for (int j = 0; j + 1 < VPL; ++j) key[j] = key[j + 1];
        key[VPL - 1] = 0;
      }
      if (lane == i) mine = top;
    };
    for (int i = 0; i < rounds; ++i) round(i);
    // Whether one and the one behind it could change places: the same but for the cut bits (BF16 logits have none there), or (bias)
    // within the rounding.
    auto is_near = [&](uint32_t one, uint32_t behind) {
      if (behind <= kIndex) return false;   // none
      if (!a.bias) return sizeof(T) == 4 && (one ^ behind) <= kIndex;
      const float x = unordered(one & ~kIndex), y = unordered(behind | kIndex), apart = a.sigmoid ? kNearFastSigmoid : kNearSoftmax * soft.inverse;
      return (one ^ behind) <= kIndex || x - y <= fmaf(kNearSum, fmaxf(fabsf(unordered(one | kIndex)), fabsf(unordered(behind & ~kIndex))), apart);
    };
    const uint32_t behind = __shfl_down_sync(0xffffffffu, mine, 1);
    bool near = is_near(mine, lane < 31 ? behind : rounds == 33 ? top : 0u);   // (the 33rd has no lane)
    uint32_t nears = __ballot_sync(0xffffffffu, near);
    auto choice_of = [&]() { return mine > kIndex ? (int)(kIndex - (mine & kIndex)) : -1; };
    int choice = choice_of();
    if (nears) {
      // The list goes on until its last one is near no other, then whole keys tell the order of two near ones (exact ones where those
      // are near too).
      int listed = min(rounds, 32);
      for (; listed < 32 && listed > 1 && (nears >> (listed - 2) & 1); ++listed) {
        round(listed);
        if (lane == listed - 1) near = is_near(mine, top);
        nears = __ballot_sync(0xffffffffu, near);
      }
      choice = choice_of();
      if (nears >> 31 || (listed == 32 && a.k < 32 && nears >> 30)) {   // a list that does not end
        choice = select_carefully<VPL, QUADS>(a, row, soft, lane);
      } else {
        float score = choice >= 0 ? to_f32(row[choice]) : 0.0f, own = kNearOwn;
        const float b = a.bias && choice >= 0 ? a.bias[choice] : 0.0f;
        if (a.bias) {
          if (!a.sigmoid) own = fmaf(kNearDistance, soft.top - score, own);
          score = a.sigmoid ? sigmoid(score) : soft(score);
          own = fmaf(own, score, kNearBias * fabsf(b));
        }
        double exact = 0.0;
        bool exactly = false, unclear = false;
        auto before = [&](int i, bool ask) {   // whether lane i's choice comes before this lane's
          const int its = __shfl_sync(0xffffffffu, choice, i);
          if (exactly) {
            const double other = __shfl_sync(0xffffffffu, exact, i);
            return ask && (other > exact || (other == exact && its < choice));
          }
          const float other = __shfl_sync(0xffffffffu, score, i), ds = other - score, db = __shfl_sync(0xffffffffu, b, i) - b, d = ds + db;
          const float owns = own + __shfl_sync(0xffffffffu, own, i) + kNearTiny;
          unclear |= ask && a.bias && !(fabsf(d) > owns + kNearDifference * fabsf(ds) + kNearBiases * fabsf(db));
          return ask && (d > 0.0f || (!(d < 0.0f) && its < choice));   // (two infinite logits are equal)
        };
        int from = lane;
        for (;;) {
          if ((nears & (nears << 1)) == 0) {   // only neighbours can change places
            const uint32_t swaps = __ballot_sync(0xffffffffu, before((lane + 1) & 31, near));
            from = lane + (int)(swaps >> lane & 1) - (int)((swaps << 1) >> lane & 1);
          } else {
            int place = 0;
            for (int i = 0; i < listed; ++i) {
              const int its = __shfl_sync(0xffffffffu, choice, i);
              place += before(i, its >= 0 && choice >= 0 && i != lane);
            }
            for (int i = 0; i < listed; ++i)
              if (__shfl_sync(0xffffffffu, choice >= 0 ? place : -1, i) == lane) from = i;
          }
          if (exactly || !__any_sync(0xffffffffu, unclear)) break;
          exact = exact_score(row, a.E, choice, lane, a.sigmoid, soft.top) + (double)b;
          exactly = true;
        }
        choice = __shfl_sync(0xffffffffu, choice, from);
      }
    }
    if (lane >= a.k) choice = -1;
    float weight = 0.0f;
    if (choice >= 0) {
      const float x = to_f32(row[choice]);
      weight = a.sigmoid ? sigmoid(x) : soft(x);
    }
    if (a.renorm) weight = __fdiv_rn(weight, warp_sum(weight) + 1e-20f);
    if (lane < a.k) {
      a.ids[to] = choice;
      a.weights[to] = weight * a.factor;
    }
  }
}

template <typename T, int VPL, bool QUADS>
__global__ void __launch_bounds__(32 * kWarps) route_backward_kernel(const RouteArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32;
  for (unsigned t = blockIdx.x * kWarps + threadIdx.x / 32; t < (unsigned)a.T; t += gridDim.x * kWarps) {   // (T and the step: below 2^31 each)
    const T* row = static_cast<const T*>(a.logits) + (size_t)t * (unsigned)a.E;
    const size_t to = (size_t)t * (unsigned)a.k + lane;
    T* out = static_cast<T*>(a.dlogits) + (size_t)t * (unsigned)a.E;
    int e = lane < a.k ? a.ids[to] : -1;
    float d = lane < a.k ? a.dweights[to] : 0.0f;
    float l[VPL];
    if (!a.sigmoid) load_logits<QUADS>(row, a.E, lane, l);
    if (e < 0 || e >= a.E) e = -1, d = 0.0f;
    d *= a.factor;
    const float x = e >= 0 ? to_f32(row[e]) : 0.0f;   // (behind the row's own loads: in L1 then)
    Softmax soft{};
    if (!a.sigmoid) soft = softmax_of(l, l);
    const float s = e < 0 ? 0.0f : a.sigmoid ? sigmoid(x) : soft(x);
    if (a.renorm) {
      const float total = warp_sum(s) + 1e-20f, mean = warp_sum(d * s) / total;
      d = e >= 0 ? (d - mean) / total : 0.0f;
    }
    const float along = a.sigmoid ? 0.0f : warp_sum(s * d);
    // an expert chosen twice: each of its lanes has the sum
    const uint32_t same = __match_any_sync(0xffffffffu, e);
    float all = d;
    if (__any_sync(0xffffffffu, e >= 0 && (same & (same - 1)))) {
      all = 0.0f;
      for (int i = 0; i < 32; ++i) {
        const float v = __shfl_sync(0xffffffffu, d, i);
        if (same >> i & 1) all += v;
      }
    }
    __syncwarp();   // dlogits may be logits: every lane has read what it needs
    if constexpr (QUADS) {
#pragma unroll
      for (int j = 0; j < VPL; j += 4) {
        const int c = expert_of<true>(j, lane);
        if (c >= a.E) continue;
        float v[4] = {};
        if (!a.sigmoid)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = -along * (l[j + i] * soft.inverse);   // (exponentials by now)
        if constexpr (sizeof(T) == 4)
          *reinterpret_cast<float4*>(out + c) = make_float4(v[0], v[1], v[2], v[3]);
        else
          *reinterpret_cast<uint2*>(out + c) = make_uint2(round_bf16x2(v[0], v[1]), round_bf16x2(v[2], v[3]));
      }
    } else {
#pragma unroll
      for (int j = 0; j < VPL; ++j)
        if (j * 32 + lane < a.E) store_f32(out + j * 32 + lane, a.sigmoid ? 0.0f : -along * (l[j] * soft.inverse));
    }
    __syncwarp();   // (the selected ones' stores come behind)
    if (e >= 0) store_f32(out + e, a.sigmoid ? all * s * sigmoid(-x) : s * (all - along));   // (1 - s without its cancellation)
  }
}

template <typename T, int VPL, bool QUADS>
cudaError_t launch_one(const RouteArgs& a, bool backward, const StreamArgs& s) {
  const int grid = (int)s.limit.all((a.T + kWarps - 1) / kWarps);
  return launch_plain(backward ? route_backward_kernel<T, VPL, QUADS> : route_kernel<T, VPL, QUADS>, grid, 32 * kWarps, 0, s, a);
}

template <typename T>
cudaError_t launch_typed(const RouteArgs& a, bool backward, const StreamArgs& s) {
  const uintptr_t places = reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits), bias = reinterpret_cast<uintptr_t>(a.bias);
  auto pick = [&](auto vpl) {
    constexpr int VPL = decltype(vpl)::value;
    return a.E % 4 == 0 && places % (4 * sizeof(T)) == 0 && bias % 16 == 0 ? launch_one<T, VPL, true>(a, backward, s) : launch_one<T, VPL, false>(a, backward, s);
  };
  if (a.E <= 64) return launch_one<T, 2, false>(a, backward, s);
  if (a.E <= 128) return pick(std::integral_constant<int, 4>{});
  if (a.E <= 256) return pick(std::integral_constant<int, 8>{});
  if (a.E <= 512) return pick(std::integral_constant<int, 16>{});
  return pick(std::integral_constant<int, 32>{});
}

}  // namespace

cudaError_t launch_route(const RouteArgs& a, bool bf16, bool backward, const StreamArgs& s) {
  return bf16 ? launch_typed<__nv_bfloat16>(a, backward, s) : launch_typed<float>(a, backward, s);
}

}  // namespace dg
