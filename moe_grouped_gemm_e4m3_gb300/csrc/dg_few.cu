// dg_few.cu — products of a few tokens with streamed weights: the experts' feed-forward layer (two products and the
// cast between them), and the dense product with four-bit weights.
//
//   layer: for each token t and each of its k experts e = ids[t, j]
//     d = x_t·W1[e]ᵀ (2I rows: I gate rows, then I up rows),  h = silu(d[:I])·d[I:]       stream kernel, kStreamUp
//     q, s = E4M3 cast of h in groups of 128                                              h_cast_kernel
//     y_t = Σ_j weights[t, j]·(q·s)·W2[e]ᵀ                                                stream kernel, kStreamDown
//   dense: D = A·Bᵀ                                                                       stream kernel, kStreamDense
//
// All of it is a read of weights: with a token or two an expert each weight byte meets two to four operations. So the
// kernel is built around the read. A warp streams units of 16 weight rows x 128 bytes (128 E4M3 or 256 E2M1 values of each
// row) through a ring of its own in shared memory, by asynchronous copies that run ahead over units, items and experts alike; nothing
// but the warp itself waits for them. (A read alone through such rings reaches 6.6 to 7.1 TB/s, 352 MB to 1 GB.) The warps
// of a CTA take an item's units in turn (K split over them) and add their sums through shared memory in warp order: no atomics.
//
// Arithmetic: mma.sync m16n8k16 in FP16 with FP32 accumulators. The 16 rows are weights (kStreamUp: 8 gate rows and the 8 up
// rows of the same columns, so a thread ends up with both), the 8 columns tokens. E4M3 and E2M1 values are exact in FP16, and
// converting them costs one instruction for two (mma.sync on E4M3 itself takes twice as long here: 13.8 ns a k32 against
// 2 x 4.2 in FP16). The order of k inside a scale's group is free as long as both operands use the same one, so a lane's
// operands are consecutive bytes. A group's partial sum meets its scales in FP32: E4M3 weights every 128 values, E2M1 every 32.
// Tokens that an expert does not serve are columns of zeros; a token keeps its column, so kStreamDown adds up a token's
// experts in the accumulators.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_scale.cuh"
#include "dg_vec.cuh"

namespace dg {

namespace {

enum Kind { kStreamUp, kStreamDown, kStreamDense };

constexpr int kRows = 16, kUnitBytes = 128;                 // of a unit: weight rows, bytes of each
constexpr int kStage = kRows * kUnitBytes + kRows * 12;     // codes, then scales (E2M1: 12 bytes a row; E4M3: two words)

struct FewArgs {
  const uint8_t* x;        // E4M3 rows: tokens (kStreamUp, kStreamDense) or the cast h of each (token, choice) (kStreamDown)
  const void* sx;          // their scales: MN-major [K groups][align4(T)] (kStreamUp, kStreamDense), [row][I/128] FP32 (kStreamDown)
  const uint8_t* w;        // codes
  const void* sw;
  const int32_t* ids;
  const float* weights;
  void* out;               // kStreamUp: h [T·k, I] FP32
  int* status;
  int T, k, E;
  int K;                   // contraction
  int rows;                // weight rows an expert (kStreamUp: 2I)
};

__device__ __forceinline__ void mma_16x8x16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two E4M3 codes (the low or high half of a word) as FP16.
__device__ __forceinline__ uint32_t e4m3_lo(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, a;}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_hi(uint32_t w) {
  uint32_t r;
  asm("{.reg .b16 a, b; mov.b32 {a, b}, %1; cvt.rn.f16x2.e4m3x2 %0, b;}" : "=r"(r) : "r"(w));
  return r;
}
// The eight E2M1 codes of a word as FP16, two a register, the low half of a byte first.
__device__ __forceinline__ void e2m1_x8(uint32_t w, uint32_t (&r)[4]) {
  asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %4; cvt.rn.f16x2.e2m1x2 %0, a; cvt.rn.f16x2.e2m1x2 %1, b; "
      "cvt.rn.f16x2.e2m1x2 %2, c; cvt.rn.f16x2.e2m1x2 %3, d;}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(w));
}

__device__ __forceinline__ void copy_16(uint32_t to, const uint8_t* from, bool live) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy_4(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ uint4 load_x(const uint8_t* p, bool live) {
  return live ? __ldg(reinterpret_cast<const uint4*>(p)) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ uint2 load_x8(const uint8_t* p, bool live) {
  return live ? __ldg(reinterpret_cast<const uint2*>(p)) : make_uint2(0, 0);
}

// The tokens of one pass (at most 32 of them): which experts they use, and where each (expert, token) pair's h row is.
struct Routing {
  uint32_t* mask;      // [E] tokens of each expert
  float* weight;       // of a pair: its weight (an expert chosen twice: their sum)
  uint16_t* active;    // [E] the active experts, ascending
  uint16_t* first;     // [E] of each active expert: its first pair
  uint16_t* row;       // of a pair: the choice t·k + j (within the pass) whose h row it uses
  int* count;          // of active experts
  __host__ __device__ static size_t bytes(int E, int pairs) { return (size_t)E * 8 + (size_t)pairs * 8 + 16; }
  __device__ Routing(uint8_t* at, int E, int pairs) {
    mask = reinterpret_cast<uint32_t*>(at);
    weight = reinterpret_cast<float*>(mask + E);
    active = reinterpret_cast<uint16_t*>(weight + pairs);
    first = active + E;
    row = first + E;
    count = reinterpret_cast<int*>(at + (bytes(E, pairs) - 16));
  }
};

__device__ void build_routing(const Routing& r, const FewArgs& a, int t0, int tokens, bool with_weights) {
  const int tid = threadIdx.x, n = tokens * a.k;
  __syncthreads();   // the last pass is done with it
  for (int e = tid; e < a.E; e += blockDim.x) r.mask[e] = 0;
  __syncthreads();
  const int32_t* ids = a.ids + (size_t)t0 * a.k;
  for (int i = tid; i < n; i += blockDim.x) {
    const int e = ids[i];
    if (e >= 0 && e < a.E)
      atomicOr(&r.mask[e], 1u << (i / a.k));
    else if (e != -1 && blockIdx.x == 0)
      atomicOr(a.status, kStatusBadGroup);
  }
  __syncthreads();
  if (tid < 32) {   // active experts and their pairs, by prefix sums over 32 experts at a time
    int count = 0, pairs = 0;
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + tid;
      const uint32_t mask = e < a.E ? r.mask[e] : 0;
      const uint32_t some = __ballot_sync(0xffffffffu, mask != 0);
      int before = __popc(mask);
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, before, o);
        if (tid >= o) before += v;
      }
      const int all = __shfl_sync(0xffffffffu, before, 31);
      before -= __popc(mask);
      if (mask) {
        const int at = count + __popc(some & ((1u << tid) - 1));
        r.active[at] = (uint16_t)e;
        r.first[at] = (uint16_t)(pairs + before);
      }
      count += __popc(some);
      pairs += all;
    }
    if (tid == 0) *r.count = count;
  }
  __syncthreads();
  // each expert's pairs
  for (int at = tid / 32; at < *r.count; at += blockDim.x / 32) {
    const int e = r.active[at], t = tid % 32;
    const uint32_t mask = r.mask[e];
    if (mask >> t & 1) {
      const int pair = r.first[at] + __popc(mask & ((1u << t) - 1));
      int first = -1;
      float w = 0.0f;
      for (int j = 0; j < a.k; ++j)
        if (ids[t * a.k + j] == e) {
          if (first < 0) first = j;
          if (with_weights) w += a.weights[(size_t)(t0 + t) * a.k + j];
        }
      r.row[pair] = (uint16_t)(t * a.k + first);
      r.weight[pair] = w;
    }
  }
  __syncthreads();
}

template <Kind KIND, WeightForm FORM, int NT, bool OUT_F32>
__global__ void __launch_bounds__(512, 1) stream_kernel(const FewArgs a, const int stages) {
  extern __shared__ __align__(16) uint8_t ring_of_all[];
  constexpr bool kRouted = KIND != kStreamDense, kFour = FORM == kMxfp4;
  constexpr int kUnitK = kFour ? 256 : 128;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, W = blockDim.x / 32, g = lane / 4, t4 = lane % 4;
  float* const sums = reinterpret_cast<float*>(ring_of_all + (size_t)W * stages * kStage);   // [2][W][NT][4][32]
  const Routing route(reinterpret_cast<uint8_t*>(sums + 2 * W * NT * 128), a.E, (a.T < 8 * NT ? a.T : 8 * NT) * a.k);
  const uint32_t ring = smem_u32(ring_of_all) + warp * stages * kStage;
  const uint8_t* const ring_at = ring_of_all + (size_t)warp * stages * kStage;
  if constexpr (KIND != kStreamDown) griddep_wait();   // (kStreamDown reads weights and ids first: see launch_moe)
  griddep_launch_dependents();

  const int units_k = (a.K + kUnitK - 1) / kUnitK, groups_k = (a.K + 127) / 128;
  const int row_bytes = kFour ? a.K / 2 : a.K, row_scales = a.K / 32;
  const int blocks = KIND == kStreamUp ? a.rows / 16 : (a.rows + 15) / 16;   // items an expert (kStreamDown: in all)
  const int ldx = (a.T + 3) / 4 * 4;
  bool waited = KIND != kStreamDown;

  for (int t0 = 0; t0 < a.T; t0 += 8 * NT) {
    const int tokens = a.T - t0 < 8 * NT ? a.T - t0 : 8 * NT;
    if constexpr (kRouted) build_routing(route, a, t0, tokens, KIND == kStreamDown);
    const int active = kRouted ? *route.count : 1;
    const int items = KIND == kStreamUp ? active * blocks : blocks, per = KIND == kStreamDown ? active * units_k : units_k;

    // The copies' place: an item and one of its units (the expert, and the unit along K).
    int p_item = blockIdx.x, p_at = 0, p_u = warp, p_stage = 0;
    auto settle = [&](int& item, int& at, int& u) {   // to the next unit that there is, when u has run past the row
      if constexpr (KIND == kStreamDown) {
        while (u >= units_k) {
          u -= units_k;
          if (++at >= active) {
            at = 0, u = warp, item += gridDim.x;
            while (u >= units_k && at < active) u -= units_k, ++at;
            if (at >= active) item = items, at = 0, u = 0;   // this warp has no unit of any item
            break;
          }
        }
      } else if (u >= units_k) {
        u = warp, item += gridDim.x;
        if (u >= units_k) item = items;
      }
    };
    auto first = [&](int& item, int& at, int& u) {
      item = blockIdx.x, at = 0, u = warp;
      if constexpr (KIND == kStreamDown) {
        while (u >= units_k && at < active) u -= units_k, ++at;
        if (at >= active) item = items;
      } else if (u >= units_k) {
        item = items;
      }
    };
    first(p_item, p_at, p_u);
    auto issue = [&]() {
      if (p_item < items) {
        const int expert = KIND == kStreamUp ? route.active[p_item / blocks] : KIND == kStreamDown ? route.active[p_at] : 0;
        const int block = KIND == kStreamUp ? p_item % blocks : p_item;
        const uint32_t to = ring + p_stage * kStage;
        // rows 0..7 and 8..15 of the unit start here in the expert's matrix
        const int lo = KIND == kStreamUp ? block * 8 : block * 16, hi = KIND == kStreamUp ? a.rows / 2 + lo : lo + 8;
        const int r = lane / 8, c = lane % 8;
        const int byte = p_u * kUnitBytes + c * 16;
        const bool live = byte < row_bytes;
        const size_t first_row = (size_t)expert * a.rows;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int local = r + 4 * j, row = j < 2 ? lo + local : hi + local - 8;
          const bool there = live && (KIND != kStreamDense || row < a.rows);
          copy_16(to + local * kUnitBytes + ((c ^ (local & 7)) * 16), there ? a.w + (first_row + row) * row_bytes + byte : a.w, there);
        }
        if constexpr (kFour) {
          // eight scale bytes of each row from any place: the three aligned words that hold them
          for (int q = lane; q < kRows * 3; q += 32) {
            const int local = q / 3, row = local < 8 ? lo + local : hi + local - 8;
            if (KIND != kStreamDense || row < a.rows) {
              const size_t at = (first_row + row) * row_scales + p_u * 8, word = (at & ~(size_t)3) + (q % 3) * 4;
              const size_t end = (size_t)(kRouted ? a.E : 1) * a.rows * row_scales;
              const int bytes = word >= end ? 0 : end - word < 4 ? (int)(end - word) : 4;
              copy_4(to + kRows * kUnitBytes + local * 12 + (q % 3) * 4, static_cast<const uint8_t*>(a.sw) + (bytes ? word : 0), bytes);
            }
          }
        } else {
          // the scales of both halves' 128-row blocks: an FP32 value each, or the packed word with this K-block's byte
          if (lane < 2) {
            const int ns = FORM == kFp8Packed ? (groups_k + 3) / 4 : groups_k, kq = FORM == kFp8Packed ? p_u / 4 : p_u;
            const int nb = (lane == 0 ? lo : hi) / 128;
            copy_4(to + kRows * kUnitBytes + lane * 4,
                   static_cast<const uint32_t*>(a.sw) + ((size_t)expert * ((a.rows + 127) / 128) + nb) * ns + kq, 4);
          }
        }
        p_u += W;
        settle(p_item, p_at, p_u);
        if (++p_stage == stages) p_stage = 0;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int s = 0; s < stages - 1; ++s) issue();
    if constexpr (KIND == kStreamDown) {
      if (!waited) griddep_wait(), waited = true;
    }

    int stage = 0, buffer = 0;
    for (int item = blockIdx.x; item < items; item += gridDim.x, buffer ^= 1) {
      float acc[NT][4] = {};
      int at = KIND == kStreamUp ? item / blocks : 0, u = warp;
      if constexpr (KIND == kStreamDown)
        while (u >= units_k && at < active) u -= units_k, ++at;
      for (int n = warp; n < per; n += W) {
        const uint32_t mask = kRouted ? route.mask[route.active[at]] : 0xffffffffu;
        // the tokens' operands: column n·8 + g of this lane
        const uint8_t* xs[NT];
        bool live[NT];
        float sx[NT][kFour ? 2 : 1][2];
        bool on[NT][2];
#pragma unroll
        for (int i = 0; i < NT; ++i) {
          const int t = i * 8 + g;
          live[i] = t < tokens && (mask >> t & 1);
          size_t row = (size_t)(t0 + t);
          if (KIND == kStreamDown && live[i]) row = (size_t)t0 * a.k + route.row[route.first[at] + __popc(mask & ((1u << t) - 1))];
          xs[i] = a.x + (live[i] ? row : 0) * a.K;
#pragma unroll
          for (int c = 0; c < 2; ++c) {   // the scales of the tokens of this lane's accumulators
            const int tc = i * 8 + 2 * t4 + c;
            const bool there = tc < tokens && (mask >> tc & 1);
            on[i][c] = there;
#pragma unroll
            for (int b = 0; b < (kFour ? 2 : 1); ++b) {
              const int kb = kFour ? 2 * u + b : u;
              float s = 0.0f;
              if (there && kb < groups_k) {
                if constexpr (KIND == kStreamDown) {
                  const int pair = route.first[at] + __popc(mask & ((1u << tc) - 1));
                  s = static_cast<const float*>(a.sx)[((size_t)t0 * a.k + route.row[pair]) * groups_k + kb] * route.weight[pair];
                } else if constexpr (FORM == kFp8Packed) {
                  s = ue8m0_value(__ldg(static_cast<const uint32_t*>(a.sx) + (size_t)(kb / 4) * ldx + t0 + tc) >> (8 * (kb & 3)));
                } else {
                  s = __ldg(static_cast<const float*>(a.sx) + (size_t)kb * ldx + t0 + tc);
                }
              }
              sx[i][b][c] = s;
            }
          }
        }
        if (stages == 4) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else if (stages == 3) asm volatile("cp.async.wait_group 1;" ::: "memory");
        else asm volatile("cp.async.wait_group 0;" ::: "memory");   // (two stages)
        __syncwarp();
        issue();
        const uint8_t* unit = ring_at + stage * kStage;
        if constexpr (kFour) {
          // 8 groups of 32: a lane has word t4 of chunk j of its rows
          const uint8_t* sc = unit + kRows * kUnitBytes;
          uint32_t scales[2][2];   // of rows g and g + 8: eight bytes
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int local = g + 8 * h;
            const int row = KIND == kStreamUp ? (item % blocks) * 8 + g + h * (a.rows / 2) : item * 16 + local;
            const int expert = kRouted ? route.active[at] : 0;
            const uint32_t shift = (uint32_t)(((size_t)expert * a.rows + row) * row_scales + u * 8) & 3;
            const uint32_t* w = reinterpret_cast<const uint32_t*>(sc + local * 12);
            const uint32_t w0 = w[0], w1 = w[1], w2 = w[2];
            scales[h][0] = __funnelshift_r(w0, w1, 8 * shift);
            scales[h][1] = __funnelshift_r(w1, w2, 8 * shift);
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            float part[NT][4] = {};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int chunk = b * 4 + j, k = u * 256 + chunk * 32 + t4 * 8;
              const bool in = u * 256 + chunk * 32 < a.K;
              uint32_t lo[4], hi[4];
              e2m1_x8(*reinterpret_cast<const uint32_t*>(unit + g * kUnitBytes + ((chunk ^ g) * 16) + t4 * 4), lo);
              e2m1_x8(*reinterpret_cast<const uint32_t*>(unit + (g + 8) * kUnitBytes + ((chunk ^ g) * 16) + t4 * 4), hi);
              const float s0 = in ? ue8m0_value(scales[0][b] >> (8 * j)) : 0.0f, s1 = in ? ue8m0_value(scales[1][b] >> (8 * j)) : 0.0f;
              const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
              for (int i = 0; i < NT; ++i) {
                const uint2 x = load_x8(xs[i] + k, live[i] && in);
                float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                mma_16x8x16(c, a0, e4m3_lo(x.x), e4m3_hi(x.x));
                mma_16x8x16(c, a1, e4m3_lo(x.y), e4m3_hi(x.y));
                part[i][0] = fmaf(c[0], s0, part[i][0]);
                part[i][1] = fmaf(c[1], s0, part[i][1]);
                part[i][2] = fmaf(c[2], s1, part[i][2]);
                part[i][3] = fmaf(c[3], s1, part[i][3]);
              }
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
              for (int q = 0; q < 4; ++q)
                if (on[i][q & 1]) acc[i][q] = fmaf(part[i][q], sx[i][b][q & 1], acc[i][q]);   // (0·NaN of another token's expert)
          }
        } else {
          // one group of 128: a lane has 32 consecutive bytes of its rows
          const int k = u * 128 + t4 * 32;
          uint4 x[NT][2];
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) x[i][h] = load_x(xs[i] + k + 16 * h, live[i] && k + 16 * h < a.K);
          float part[NT][4] = {};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 w0 = *reinterpret_cast<const uint4*>(unit + g * kUnitBytes + (((2 * t4 + h) ^ g) * 16));
            const uint4 w1 = *reinterpret_cast<const uint4*>(unit + (g + 8) * kUnitBytes + (((2 * t4 + h) ^ g) * 16));
            auto word = [&](uint32_t lo, uint32_t hi, auto of) {
              const uint32_t f[4] = {e4m3_lo(lo), e4m3_lo(hi), e4m3_hi(lo), e4m3_hi(hi)};
#pragma unroll
              for (int i = 0; i < NT; ++i) mma_16x8x16(part[i], f, e4m3_lo(of(x[i][h])), e4m3_hi(of(x[i][h])));
            };
            word(w0.x, w1.x, [](const uint4& v) { return v.x; });
            word(w0.y, w1.y, [](const uint4& v) { return v.y; });
            word(w0.z, w1.z, [](const uint4& v) { return v.z; });
            word(w0.w, w1.w, [](const uint4& v) { return v.w; });
          }
          const uint32_t* sc = reinterpret_cast<const uint32_t*>(unit + kRows * kUnitBytes);
          float s0, s1;
          if constexpr (FORM == kFp8Packed)
            s0 = ue8m0_value(sc[0] >> (8 * (u & 3))), s1 = ue8m0_value(sc[1] >> (8 * (u & 3)));
          else
            s0 = __uint_as_float(sc[0]), s1 = __uint_as_float(sc[1]);
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q)
              if (on[i][q & 1]) acc[i][q] = fmaf(part[i][q], (q < 2 ? s0 : s1) * sx[i][0][q & 1], acc[i][q]);   // (0·NaN, see above)
        }
        __syncwarp();   // the stage is free for the copies of the next turn
        if (++stage == stages) stage = 0;
        u += W;
        if constexpr (KIND == kStreamDown)
          while (u >= units_k && at < active) u -= units_k, ++at;
      }

      // the warps' sums, in warp order (two buffers by turns: one barrier an item)
      float* const mine = sums + (size_t)buffer * W * NT * 128;
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int q = 0; q < 4; ++q) mine[((warp * NT + i) * 4 + q) * 32 + lane] = acc[i][q];
      __syncthreads();
      auto sum = [&](int m, int row) {   // token m, row of the 16
        const int q = (row / 8) * 2 + m % 2, from = ((m / 8) * 4 + q) * 32 + (row % 8) * 4 + (m % 8) / 2;
        float s = 0.0f;
        for (int w = 0; w < W; ++w) s += mine[w * NT * 128 + from];
        return s;
      };
      if constexpr (KIND == kStreamUp) {
        const int act = item / blocks, j0 = (item % blocks) * 8;
        const uint32_t mask = route.mask[route.active[act]];
        for (int o = threadIdx.x; o < 8 * tokens; o += blockDim.x) {
          const int m = o / 8, j = o % 8;
          if (!(mask >> m & 1)) continue;
          const size_t row = (size_t)t0 * a.k + route.row[route.first[act] + __popc(mask & ((1u << m) - 1))];
          const float gate = sum(m, j), up = sum(m, 8 + j);
          static_cast<float*>(a.out)[row * (a.rows / 2) + j0 + j] = silu_f32(gate) * up;
        }
      } else {
        for (int o = threadIdx.x; o < 16 * tokens; o += blockDim.x) {
          const int m = o / 16, j = o % 16, n = item * 16 + j;
          if (n >= a.rows) continue;
          const float v = sum(m, j);
          const size_t to = (size_t)(t0 + m) * a.rows + n;
          if constexpr (OUT_F32)
            static_cast<float*>(a.out)[to] = v;
          else
            static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(v);
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if constexpr (KIND == kStreamDown) {
    if (!waited) griddep_wait();
  }
}

// The cast of h [rows, I] in FP32: E4M3 codes and one FP32 scale per group of 128 (UE: a power of two). A warp a group.
template <bool UE>
__global__ void __launch_bounds__(256) h_cast_kernel(const float* __restrict__ h, const int32_t* __restrict__ ids, uint8_t* __restrict__ q,
                                                     float* __restrict__ s, long long groups, int per_row) {
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % 32;
  for (long long i = (long long)blockIdx.x * 8 + threadIdx.x / 32; i < groups; i += (long long)gridDim.x * 8) {
    if (ids[i / per_row] < 0) continue;   // no expert: no h
    const float4 v = reinterpret_cast<const float4*>(h)[i * 32 + lane];
    float top = fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    float f;
    uint32_t scale;
    group_scale<UE>(top, f, scale);
    const uint32_t lo = e4m3x2_satfinite(__fmul_rn(v.x, f), __fmul_rn(v.y, f)), hi = e4m3x2_satfinite(__fmul_rn(v.z, f), __fmul_rn(v.w, f));
    reinterpret_cast<uint32_t*>(q)[i * 32 + lane] = lo | (hi << 16);
    if (lane == 0) s[i] = UE ? ue8m0_value(scale) : __uint_as_float(scale);
  }
}

// Warps a CTA: the number among which an item's units divide best. Sixteen warps an SM in all, with as many stages as fit.
struct FewPlan {
  int warps, ctas, stages;
  size_t smem;
};
FewPlan few_plan(int units, int NT, size_t routing, const SmLimit& limit) {
  FewPlan p{8, 0, 0, 0};
  double least = 1e9;
  for (int w : {8, 4, 16}) {
    const double turns = (double)((units + w - 1) / w) * w / units;
    if (turns < least - 0.02) least = turns, p.warps = w;
  }
  for (p.ctas = limit.capped ? 1 : 16 / p.warps;; --p.ctas)
    for (p.stages = 4; p.stages >= (p.ctas == 1 ? 2 : 3); --p.stages) {
      p.smem = (size_t)p.warps * (p.stages * kStage + 2 * NT * 128 * sizeof(float)) + routing;
      if (p.ctas * (p.smem + 1024) <= (size_t)227 << 10) return p;
    }
}

template <Kind KIND, WeightForm FORM, int NT, bool OUT_F32>
cudaError_t launch_stream_nt(const FewArgs& a, int items, int units, const StreamArgs& s) {
  auto kernel = stream_kernel<KIND, FORM, NT, OUT_F32>;
  const int pairs = (a.T < 8 * NT ? a.T : 8 * NT) * a.k;
  const FewPlan plan = few_plan(units, NT, Routing::bytes(a.E, pairs), s.limit);
  static bool configured[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!configured[dev]) {
    if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 226 << 10)) != cudaSuccess) return e;
    configured[dev] = true;
  }
  const long long most = (long long)s.limit.sms * plan.ctas;
  return launch_plain(kernel, (int)(items < most ? items : most), plan.warps * 32, plan.smem, s, a, plan.stages);
}

template <Kind KIND, WeightForm FORM, bool OUT_F32>
cudaError_t launch_stream(const FewArgs& a, int items, int units, const StreamArgs& s) {
  if (a.T <= 8) return launch_stream_nt<KIND, FORM, 1, OUT_F32>(a, items, units, s);
  if (a.T <= 16) return launch_stream_nt<KIND, FORM, 2, OUT_F32>(a, items, units, s);
  return launch_stream_nt<KIND, FORM, 4, OUT_F32>(a, items, units, s);
}

size_t align16(size_t n) { return (n + 15) / 16 * 16; }

template <WeightForm FORM>
cudaError_t launch_moe_form(const MoeArgs& m, bool out_f32, const StreamArgs& s) {
  const size_t rows = (size_t)m.T * m.k;
  float* h = static_cast<float*>(m.workspace);
  uint8_t* q = reinterpret_cast<uint8_t*>(h) + align16(rows * m.I * sizeof(float));
  float* sq = reinterpret_cast<float*>(q + align16(rows * m.I));
  constexpr int unit_k = FORM == kMxfp4 ? 256 : 128;
  const int most = (int)((long long)m.T * m.k < m.E ? (long long)m.T * m.k : m.E);   // experts that can be active
  FewArgs up{m.A, m.sA, m.w1, m.s1, m.ids, m.weights, h, m.status, m.T, m.k, m.E, m.K, 2 * m.I};
  cudaError_t e = launch_stream<kStreamUp, FORM, true>(up, most * (m.I / 8), (m.K + unit_k - 1) / unit_k, s);
  if (e != cudaSuccess) return e;
  const long long groups = (long long)rows * (m.I / 128);
  e = launch_plain(FORM == kFp8Packed ? h_cast_kernel<true> : h_cast_kernel<false>, (int)s.limit.all((groups + 7) / 8), 256, 0, s,
                   (const float*)h, m.ids, q, sq, groups, m.I / 128);
  if (e != cudaSuccess) return e;
  FewArgs down{q, sq, m.w2, m.s2, m.ids, m.weights, m.y, m.status, m.T, m.k, m.E, m.I, m.N};
  const int units = (m.I + unit_k - 1) / unit_k * most, items = (m.N + 15) / 16;
  return out_f32 ? launch_stream<kStreamDown, FORM, true>(down, items, units, s) : launch_stream<kStreamDown, FORM, false>(down, items, units, s);
}

}  // namespace

long long moe_workspace_bytes(int T, int k, int I) {
  const size_t rows = (size_t)T * k;
  return (long long)(align16(rows * I * sizeof(float)) + align16(rows * I) + rows * (I / 128) * sizeof(float));
}

cudaError_t launch_moe(const MoeArgs& m, WeightForm form, bool out_f32, const StreamArgs& s) {
  if (form == kMxfp4) return launch_moe_form<kMxfp4>(m, out_f32, s);
  return form == kFp8Packed ? launch_moe_form<kFp8Packed>(m, out_f32, s) : launch_moe_form<kFp8Scaled>(m, out_f32, s);
}

cudaError_t launch_mxfp4_gemm(const uint8_t* A, const float* sA, const uint8_t* B, const uint8_t* sB, void* D, bool out_f32, int M,
                              int N, int K, const StreamArgs& s) {
  FewArgs a{A, sA, B, sB, nullptr, nullptr, D, nullptr, M, 0, 1, K, N};
  const int items = (N + 15) / 16, units = (K + 255) / 256;
  return out_f32 ? launch_stream<kStreamDense, kMxfp4, true>(a, items, units, s) : launch_stream<kStreamDense, kMxfp4, false>(a, items, units, s);
}

}  // namespace dg
