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
//
// Measured (us; floor: the weights read once at the measured copy rate): one token through 8 of 32 experts of 7168x2048, E4M3, 60
// (52); through 64 such, packed scales, 4 tokens 151, 16 tokens 320 (at most 367: uneven choices read fewer experts), 32 tokens 551 (410).
// Four bits: 1x7168x16384 16.2 (9.2), 16x24576x1536 11.4 to 13.1 (3.1; the upper one with six sets of inputs in turn, more than L2 holds),
// through 8 of 32 experts of 7168x2048 2 tokens 68 (48) and 16 tokens 212 (110), 32 tokens through 4 of 32 of 4096x2048 216 (62).
// With E4M3 and up to 16 tokens the read bounds it (5.8 to 7 TB/s). The four-bit products saturate nothing: 1x7168x16384 has 40% of the
// issue slots in use, 40% of the ALU pipe, 23% of the tensor pipe and 41% of the DRAM cycles, with 2.2 warps a scheduler that wait for
// loads (20 to 25% of a warp's time), fixed latencies (17%) and the pipe of the conversions (9%), and its 224 items are one or two an SM
// (18 to 54% of the issue slots); 16x24576x1536 has 35%, 28% and 18%, and waits for L1, its queues and shared memory (24%), fixed latencies
// (21%), loads (14%) and the barrier after every six units (7%). 438 instructions a unit of 32x256 (one column tile), 160 of them
// conversions. Not kept: more warps (24 for 16) and the tokens' operands staged as FP16 in shared memory, at most 4% off; batches of items
// whose units the warps share as ranges (fewer turns, one joining of sums a batch), 66 us for 60 and 17 for 15: the warps' pieces of a row
// lie apart then, and the joining is not hidden. E2M1 kernels of four column tiles spill (360 to 690 bytes a thread).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "dg_few_plan.h"
#include "dg_launch.h"
#include "dg_scale.cuh"
#include "dg_vec.cuh"

namespace dg {

namespace {

enum Kind { kStreamUp, kStreamDown, kStreamDense };

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

// (With no bytes the address is not read, and zeros are written.)
__device__ __forceinline__ void copy_16(uint32_t to, const uint8_t* from, int bytes) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_4(uint32_t to, const void* from, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
}

__device__ __forceinline__ void copy_8(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(to), "l"(from) : "memory");
}

// The tokens of one pass (at most 32 of them): which experts they use, and where each (expert, token) pair's h row is.
struct Routing {
  uint32_t* mask;      // [E] tokens of each expert
  float* chosen;       // [pairs] the choices' weights as given
  float* weight;       // of a pair: its weight (an expert chosen twice: their sum)
  uint16_t* choice;    // [pairs] the choices as given, kNone for no expert
  uint16_t* active;    // [E] the active experts, ascending
  uint16_t* first;     // [E] of each active expert: its first pair
  uint16_t* row;       // of a pair: the choice t·k + j (within the pass) whose h row it uses
  uint16_t* token;     // of a pair
  int* count;          // of active experts
  static constexpr uint16_t kNone = 0xFFFF;
  __device__ Routing(uint8_t* at, int E, int pairs) {
    mask = reinterpret_cast<uint32_t*>(at);
    chosen = reinterpret_cast<float*>(mask + E);
    weight = chosen + pairs;
    choice = reinterpret_cast<uint16_t*>(weight + pairs);
    active = choice + pairs;
    first = active + E;
    row = first + E;
    token = row + pairs;
    count = reinterpret_cast<int*>(at + (routing_bytes(E, pairs) - 16));
  }
};

// The active experts of a pass: all that the copies of weights need to begin.
__device__ void find_active(const Routing& r, const FewArgs& a, int t0, int tokens, bool with_weights) {
  const int tid = threadIdx.x, n = tokens * a.k;
  __syncthreads();   // the last pass is done with it
  for (int e = tid; e < a.E; e += blockDim.x) r.mask[e] = 0;
  __syncthreads();
  for (int i = tid; i < n; i += blockDim.x) {
    const int e = a.ids[(size_t)t0 * a.k + i];
    const bool some = e >= 0 && e < a.E;
    if (with_weights) r.chosen[i] = a.weights[(size_t)t0 * a.k + i];
    r.choice[i] = some ? (uint16_t)e : Routing::kNone;
    if (some)
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
      if (some == 0) continue;
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
}

// Each active expert's pairs (beside the first copies).
__device__ void find_pairs(const Routing& r, const FewArgs& a, bool with_weights) {
  for (int at = threadIdx.x / 32; at < *r.count; at += blockDim.x / 32) {
    const int e = r.active[at], t = threadIdx.x % 32;
    const uint32_t mask = r.mask[e];
    if (mask >> t & 1) {
      const int pair = r.first[at] + __popc(mask & ((1u << t) - 1));
      int first = -1;
      float w = 0.0f;
      for (int j = 0; j < a.k; ++j)
        if (r.choice[t * a.k + j] == e) {
          if (first < 0) first = j;
          if (with_weights) w += r.chosen[t * a.k + j];
        }
      r.row[pair] = (uint16_t)(t * a.k + first);
      r.token[pair] = (uint16_t)t;
      r.weight[pair] = w;
    }
  }
  __syncthreads();
}

// A place in a warp's sequence of units: an item of the CTA (kStreamUp: block `block` of the expert number `at`), for kStreamDown one of
// the active experts (`at`, a walk over them inside the item), and a unit along K. A warp takes each W-th unit of every item of
// its CTA. What depends on the item and the expert alone is computed where those change, so a step along K is a few additions.
template <Kind KIND>
struct Cursor {
  int at, block, u;
  __device__ __forceinline__ void start_item(int warp, int units_k, int active) {
    u = warp;
    if constexpr (KIND == kStreamDown) {
      at = 0;
      while (u >= units_k && at < active) u -= units_k, ++at;
    }
  }
  __device__ __forceinline__ void start(int warp, int units_k, int active, int blocks) {
    at = 0, block = blockIdx.x;
    if constexpr (KIND == kStreamUp)
      while (block >= blocks) block -= blocks, ++at;
    start_item(warp, units_k, active);
  }
  __device__ __forceinline__ bool in_item(int units_k, int active) const { return KIND == kStreamDown ? at < active : u < units_k; }
  __device__ __forceinline__ bool item_left(int active, int blocks) const { return KIND == kStreamUp ? at < active : block < blocks; }
  __device__ __forceinline__ void next_item(int warp, int units_k, int active, int blocks) {
    block += gridDim.x;
    if constexpr (KIND == kStreamUp)
      while (block >= blocks) block -= blocks, ++at;
    start_item(warp, units_k, active);
  }
  // One unit on, within the item; whether the expert has changed.
  __device__ __forceinline__ bool step(int W, int units_k, int active) {
    u += W;
    bool changed = false;
    if constexpr (KIND == kStreamDown)
      while (u >= units_k && at < active) u -= units_k, ++at, changed = true;
    return changed;
  }
};

// The tokens' side of a unit: this lane's bytes of its column's token, and the scales of the two tokens of its accumulators.
template <int NT, bool FOUR>
struct Operands {
  static constexpr int tiles = NT;
  uint32_t x[NT][FOUR ? 16 : 8];
  float2 s[NT][FOUR ? 2 : 1];
};

__device__ __forceinline__ void mma_16x8x16(float2 (&c)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0].x), "+f"(c[0].y), "+f"(c[1].x), "+f"(c[1].y)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from zero.
__device__ __forceinline__ void mma_16x8x16_zero(float2 (&c)[2], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(c[0].x), "=f"(c[0].y), "=f"(c[1].x), "=f"(c[1].y)
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four E8M0 codes of a word as FP32, two a conversion (code 0 is a subnormal, 255 NaN).
__device__ __forceinline__ void e8m0_x4(uint32_t w, float (&v)[4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const __nv_bfloat162_raw b = __nv_cvt_e8m0x2_to_bf162raw((__nv_fp8x2_storage_t)(w >> (16 * h)));
    v[2 * h] = __uint_as_float((uint32_t)b.x << 16);
    v[2 * h + 1] = __uint_as_float((uint32_t)b.y << 16);
  }
}

// WHOLE: E2M1 weights whose rows are whole units, with scales that start on eight bytes in every row.
template <Kind KIND, WeightForm FORM, int NT, int R, bool OUT_F32, bool WHOLE>
__global__ void __launch_bounds__(R == 2 ? 384 : 512, 1) stream_kernel(const FewArgs a, const int stages) {
  extern __shared__ __align__(16) uint8_t ring_of_all[];
  constexpr bool kRouted = KIND != kStreamDense, kFour = FORM == kMxfp4;
  // A token keeps its column whatever the expert, and kStreamDown's sums go from one expert to the next in registers (kCarries). Or an
  // expert has only its own tokens in columns, one after another, so that mostly one tile of columns is computed (kCompact), and kStreamDown
  // adds an expert's sums to its tokens' in shared memory: where the columns' work counts, with four tiles of them or E2M1 weights (32
  // tokens, us, compact and carried: 8 of 64 experts 551 and 666, four bits 4 of 32 216 and 333; 16 tokens, four bits 212 and 221, but E4M3
  // 377 and 325).
  constexpr bool kCompact = kRouted && (NT > 2 || (NT == 2 && kFour)), kCarries = KIND == kStreamDown && !kCompact;
  constexpr int kUnitK = kFour ? 256 : 128, kRows = 16 * R, kStage = stage_bytes(R);
  constexpr int kScaleCopies = (kRows * 3 + 31) / 32;   // E2M1: three words a row, unless they start on eight bytes
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, W = blockDim.x / 32, g = lane / 4, t4 = lane % 4;
  float* const sums = reinterpret_cast<float*>(ring_of_all + (size_t)W * stages * kStage);   // [2][W][R][NT][4][32]
  const Routing route(reinterpret_cast<uint8_t*>(sums + 2 * W * R * NT * 128), a.E, (a.T < 8 * NT ? a.T : 8 * NT) * a.k);
  const uint32_t ring = smem_u32(ring_of_all) + warp * stages * kStage;
  const uint8_t* const ring_at = ring_of_all + (size_t)warp * stages * kStage;
  if constexpr (KIND != kStreamDown) griddep_wait();   // (kStreamDown reads weights and ids first: see launch_moe_form)
  griddep_launch_dependents();

  const int units_k = (a.K + kUnitK - 1) / kUnitK, groups_k = (a.K + 127) / 128;
  const int row_bytes = kFour ? a.K / 2 : a.K, row_scales = a.K / 32, half = a.rows / 2;
  const int blocks = (a.rows + kRows - 1) / kRows;   // of an expert's rows
  const int ldx = (a.T + 3) / 4 * 4;
  // Row l of a block: gate and up rows by turns of eight (kStreamUp), or one after another.
  auto row_of = [&](int block, int l) {
    return KIND == kStreamUp ? block * 8 * R + (l >> 4) * 8 + (l & 7) + ((l & 8) ? half : 0) : block * kRows + l;
  };
  const int word_steps = FORM == kFp8Packed ? (groups_k + 3) / 4 : groups_k;   // E4M3 weights' scales along K
  const uint8_t* const scales_end = static_cast<const uint8_t*>(a.sw) + (size_t)(kRouted ? a.E : 1) * a.rows * row_scales;
  constexpr bool eights = WHOLE;   // a unit's scales of a row in one piece
  // where this lane copies to in a stage: chunk lane % 8 of rows lane / 8 + 4j
  const int copy_row = lane / 8, copy_byte = (lane % 8) * 16;
  const uint32_t to_even = copy_row * kUnitBytes + ((lane % 8) ^ copy_row) * 16, to_odd = (copy_row + 4) * kUnitBytes + ((lane % 8) ^ (copy_row + 4)) * 16;
  const size_t four_rows = (size_t)4 * row_bytes, eight_rows = 2 * four_rows, half_rows = (size_t)half * row_bytes;
  bool waited = KIND != kStreamDown;
  int buffer = 0;   // of the sums: by turns over the items of all passes, so that none is written while the item before is still added up

  for (int t0 = 0; t0 < a.T; t0 += 8 * NT) {
    const int tokens = a.T - t0 < 8 * NT ? a.T - t0 : 8 * NT;
    if constexpr (kRouted) find_active(route, a, t0, tokens, KIND == kStreamDown);
    const int active = kRouted ? *route.count : 1;

    // ---- copies
    Cursor<KIND> p{};
    const uint8_t* p_from = a.w;                 // this lane's bytes of the unit's row `copy_row`
    const uint8_t* p_scales[kFour ? kScaleCopies : 1];
    int p_stage = 0;
    auto copy_enter = [&]() {   // at another item or expert
      const int expert = !kRouted ? 0 : route.active[p.at];
      const size_t first_row = (size_t)expert * a.rows;
      p_from = a.w + (first_row + row_of(p.block, copy_row)) * row_bytes + p.u * kUnitBytes + copy_byte;
      if constexpr (kFour) {
#pragma unroll
        for (int i = 0; i < kScaleCopies; ++i) {
          const int q = lane + 32 * i, l = eights ? q : q / 3, row = row_of(p.block, l);
          const bool there = l < kRows && (KIND == kStreamUp || row < a.rows);
          const size_t at = ((first_row + row) * row_scales & ~(size_t)3) + p.u * 8 + (eights ? 0 : (q % 3) * 4);
          p_scales[i] = there ? static_cast<const uint8_t*>(a.sw) + at : scales_end;
        }
      } else {
        const int nb = row_of(p.block, (lane & 1) * 8) / 128;
        p_scales[0] = static_cast<const uint8_t*>(a.sw) + (((size_t)expert * ((a.rows + 127) / 128) + nb) * word_steps) * 4;
      }
    };
    auto issue = [&]() {
      if (p.item_left(active, blocks)) {
        const uint32_t to = ring + p_stage * kStage;
        // rows copy_row + 4j, which kStreamUp takes from the gate half, the up half, and so on; zeros behind the end of K
        const int bytes = WHOLE || p.u * kUnitBytes + copy_byte < row_bytes ? 16 : 0;
        auto copy = [&](int j, int bytes) {
          const size_t more = KIND == kStreamUp ? (j >> 2) * eight_rows + (j & 1) * four_rows + (j & 2 ? half_rows : 0) : j * four_rows;
          copy_16(to + (j >> 1) * 8 * kUnitBytes + (j & 1 ? to_odd : to_even), p_from + more, bytes);
        };
        if (KIND == kStreamUp || (p.block + 1) * kRows <= a.rows) {
#pragma unroll
          for (int j = 0; j < 4 * R; ++j) copy(j, bytes);
        } else {   // the last block of a number of rows that is no multiple
#pragma unroll
          for (int j = 0; j < 4 * R; ++j)
            if (p.block * kRows + copy_row + 4 * j < a.rows) copy(j, bytes);
        }
        if constexpr (kFour) {
          // eight scale bytes of each row: in one piece, or from any place the three aligned words that hold them, as far as there are any
          if constexpr (eights) {
            if (lane < kRows && p_scales[0] != scales_end) {   // (kRows is at most 32)
              copy_8(to + kRows * kUnitBytes + lane * 16, p_scales[0]);
              p_scales[0] += 8 * W;
            }
          } else {
#pragma unroll
            for (int i = 0; i < kScaleCopies; ++i) {
              const ptrdiff_t left = scales_end - p_scales[i];
              const int bytes = left >= 4 ? 4 : left > 0 ? (int)left : 0, q = lane + 32 * i;
              if (q < kRows * 3) copy_4(to + kRows * kUnitBytes + (q / 3) * 16 + (q % 3) * 4, bytes ? p_scales[i] : static_cast<const uint8_t*>(a.sw), bytes);
              p_scales[i] += 8 * W;
            }
          }
        } else if (lane < (KIND == kStreamUp ? 2 : 1)) {
          // the scale of the rows' 128-row block (gate and up: two): an FP32 value, or the packed word with this K-block's byte
          copy_4(to + kRows * kUnitBytes + lane * 4, p_scales[0] + (FORM == kFp8Packed ? p.u / 4 : p.u) * 4, 4);
        }
        p_from += W * kUnitBytes;
        if (++p_stage == stages) p_stage = 0;
        const bool changed = p.step(W, units_k, active);
        if (!p.in_item(units_k, active)) {
          p.next_item(warp, units_k, active, blocks);
          if (!p.in_item(units_k, active)) p.at = active, p.block = blocks;   // this warp has no unit of any item
          if (p.item_left(active, blocks)) copy_enter();
        } else if (changed) {
          copy_enter();
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    p.start(warp, units_k, active, blocks);
    if (!p.in_item(units_k, active)) p.at = active, p.block = blocks;
    if (p.item_left(active, blocks)) copy_enter();

    // ---- the tokens' operands. Columns without a token, or whose token does not use the expert, read some row there is: their
    // sums are dropped (`on`, or at the end of the item). Chunks behind the end of K, whose weights are zeros, read the row's last one.
    const uint8_t* x_of[NT];     // this lane's bytes of its tokens' rows
    uint32_t on = 0;             // bit 2i + c: token i·8 + 2·t4 + c has the expert
    int columns = tokens;        // that the expert has (kCompact)
    auto tiles = [&]() { return columns <= 8 ? 1 : columns <= 16 ? 2 : 4; };
    const float* s_of[NT][2];    // those tokens' scales, and (kStreamDown) weights
    float weight_of[NT][2];
    auto enter = [&](const Cursor<KIND>& c) {   // at another item or expert
      const uint32_t mask = kRouted ? route.mask[route.active[c.at]] : 0xffffffffu;
      const int first = kRouted ? route.first[c.at] : 0;
      on = 0;
      if constexpr (kCompact) columns = __popc(mask);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        if (kCompact && i >= tiles()) continue;
        auto pair_of = [&](int column) {   // (kRouted; some pair there is where the column has none)
          if constexpr (kCompact) return first + min(column, columns - 1);
          return column < tokens && (mask >> column & 1) ? first + __popc(mask & ((1u << column) - 1)) : first;
        };
        auto token_of = [&](int column) {
          if constexpr (kCompact) return (int)route.token[pair_of(column)];
          return column < tokens && (mask >> column & 1) ? column : 0;
        };
        const size_t row = KIND == kStreamDown ? (size_t)t0 * a.k + route.row[pair_of(i * 8 + g)] : (size_t)(t0 + token_of(i * 8 + g));
        x_of[i] = a.x + row * a.K;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int tc = i * 8 + 2 * t4 + h;
          if (kCarries && tc < tokens && (mask >> tc & 1)) on |= 1u << (2 * i + h);
          if constexpr (KIND == kStreamDown) {
            s_of[i][h] = static_cast<const float*>(a.sx) + ((size_t)t0 * a.k + route.row[pair_of(tc)]) * groups_k;
            weight_of[i][h] = route.weight[pair_of(tc)];
          } else {
            s_of[i][h] = static_cast<const float*>(a.sx) + t0 + token_of(tc);
          }
        }
      }
    };
    // Plain loads: the read-only path is for data that nobody writes while the kernel lives, and a kernel that starts early lives beside
    // the one that writes its tokens (kStreamDown: beside the cast; the others: beside whatever came before the call).
    auto load = [&](const Cursor<KIND>& c, auto& o) {
#pragma unroll
      for (int i = 0; i < o.tiles; ++i) {
        if constexpr (kFour) {   // word t4 of each chunk of 32: eight consecutive values
          const uint8_t* x = x_of[i] + c.u * 256 + t4 * 8;
          if (WHOLE || c.u * 256 + 256 <= a.K) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint2 v = *reinterpret_cast<const uint2*>(x + j * 32);
              o.x[i][2 * j] = v.x, o.x[i][2 * j + 1] = v.y;
            }
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint2 v = *reinterpret_cast<const uint2*>(x_of[i] + min(c.u * 256 + j * 32, a.K - 32) + t4 * 8);
              o.x[i][2 * j] = v.x, o.x[i][2 * j + 1] = v.y;
            }
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 v = *reinterpret_cast<const uint4*>(x_of[i] + min(c.u * 128 + t4 * 32 + h * 16, a.K - 16));
            o.x[i][4 * h] = v.x, o.x[i][4 * h + 1] = v.y, o.x[i][4 * h + 2] = v.z, o.x[i][4 * h + 3] = v.w;
          }
        }
#pragma unroll
        for (int b = 0; b < (kFour ? 2 : 1); ++b) {
          const int kb = kFour ? WHOLE ? 2 * c.u + b : min(2 * c.u + b, groups_k - 1) : c.u;
          float s[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (KIND == kStreamDown)
              s[h] = s_of[i][h][kb] * weight_of[i][h];
            else if constexpr (FORM == kFp8Packed)
              s[h] = ue8m0_value(reinterpret_cast<const uint32_t*>(s_of[i][h])[(size_t)(kb >> 2) * ldx] >> (8 * (kb & 3)));
            else
              s[h] = s_of[i][h][(size_t)kb * ldx];
          }
          o.s[i][b] = make_float2(s[0], s[1]);
        }
      }
    };

    for (int s = 0; s < stages - 1; ++s) issue();
    if constexpr (kRouted) find_pairs(route, a, KIND == kStreamDown);
    if constexpr (KIND == kStreamDown) {
      if (!waited) griddep_wait(), waited = true;
    }
    Cursor<KIND> c;
    c.start(warp, units_k, active, blocks);
    int stage = 0;
    for (; c.item_left(active, blocks); buffer ^= 1) {
      const int item_at = c.at, item_block = c.block;
      float2 acc[R][NT][2] = {};
      uint32_t shift[kFour ? R : 1][2];   // E2M1: where the scale bytes of this lane's rows start in their words
      auto shifts = [&]() {
        if constexpr (kFour && !WHOLE) {
          const size_t first_row = (size_t)(kRouted ? route.active[c.at] : 0) * a.rows;
#pragma unroll
          for (int r = 0; r < R; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) shift[r][h] = 8 * ((uint32_t)((first_row + row_of(c.block, r * 16 + h * 8 + g)) * row_scales) & 3);
        }
      };
      float* const mine = sums + ((size_t)buffer * W + warp) * R * NT * 128;   // this warp's sums of the item
      if constexpr (kCompact && KIND == kStreamDown) {
        for (int i = lane; i < R * NT * 128; i += 32) mine[i] = 0.0f;
        __syncwarp();
      }
      auto unit_of = [&](auto some) {   // the unit at c, by so many tiles of columns
        constexpr int TILES = decltype(some)::value;
        Operands<TILES, kFour> o;
        load(c, o);    // (from L1 or L2: behind the copies' addresses and the wait)
        if constexpr (!kCompact) issue();
        if (stages == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
        else if (stages == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
        else asm volatile("cp.async.wait_group 1;" ::: "memory");   // (two stages)
        __syncwarp();
        const uint8_t* unit = ring_at + stage * kStage;
        [[maybe_unused]] const int u = c.u;
        if constexpr (kFour) {
          // 8 groups of 32: a lane has word t4 of chunk j of its rows
#pragma unroll
          for (int r = 0; r < R; ++r) {
            const uint8_t* rows = unit + (r * 16 + g) * kUnitBytes + t4 * 4;
            const uint8_t* sc = unit + kRows * kUnitBytes + (r * 16 + g) * 16;
            uint2 c0 = *reinterpret_cast<const uint2*>(sc), c1 = *reinterpret_cast<const uint2*>(sc + 128);   // of rows g and g + 8
            if constexpr (!eights) {
              const uint32_t b0 = reinterpret_cast<const uint32_t*>(sc)[2], b1 = reinterpret_cast<const uint32_t*>(sc + 128)[2];
              c0 = make_uint2(__funnelshift_r(c0.x, c0.y, shift[r][0]), __funnelshift_r(c0.y, b0, shift[r][0]));
              c1 = make_uint2(__funnelshift_r(c1.x, c1.y, shift[r][1]), __funnelshift_r(c1.y, b1, shift[r][1]));
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              float s0[4], s1[4];
              uint32_t e0 = b ? c0.y : c0.x, e1 = b ? c1.y : c1.x;
              if constexpr (!eights) {   // groups behind the end of K have bytes of another row: none, so that no NaN meets the zeros there
                const int left = a.K / 32 - u * 8 - b * 4;
                const uint32_t there = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1;
                e0 &= there, e1 &= there;
              }
              e8m0_x4(e0, s0);
              e8m0_x4(e1, s1);
              float2 part[TILES][2];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int chunk = b * 4 + j;
                uint32_t lo[4], hi[4];
                e2m1_x8(*reinterpret_cast<const uint32_t*>(rows + ((chunk ^ g) * 16)), lo);
                e2m1_x8(*reinterpret_cast<const uint32_t*>(rows + 8 * kUnitBytes + ((chunk ^ g) * 16)), hi);
                const uint32_t a0[4] = {lo[0], hi[0], lo[1], hi[1]}, a1[4] = {lo[2], hi[2], lo[3], hi[3]};
#pragma unroll
                for (int i = 0; i < TILES; ++i) {
                  const uint32_t x0 = o.x[i][2 * chunk], x1 = o.x[i][2 * chunk + 1];
                  float2 m[2];
                  mma_16x8x16_zero(m, a0, e4m3_lo(x0), e4m3_hi(x0));
                  mma_16x8x16(m, a1, e4m3_lo(x1), e4m3_hi(x1));
                  part[i][0] = j ? __ffma2_rn(m[0], make_float2(s0[j], s0[j]), part[i][0]) : __fmul2_rn(m[0], make_float2(s0[j], s0[j]));
                  part[i][1] = j ? __ffma2_rn(m[1], make_float2(s1[j], s1[j]), part[i][1]) : __fmul2_rn(m[1], make_float2(s1[j], s1[j]));
                }
              }
#pragma unroll
              for (int i = 0; i < TILES; ++i)   // (the bits: 0·NaN of another token's expert)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  if constexpr (!kCarries) {
                    acc[r][i][h] = __ffma2_rn(part[i][h], o.s[i][b], acc[r][i][h]);
                  } else {
                    if (on >> (2 * i) & 1) acc[r][i][h].x = fmaf(part[i][h].x, o.s[i][b].x, acc[r][i][h].x);
                    if (on >> (2 * i + 1) & 1) acc[r][i][h].y = fmaf(part[i][h].y, o.s[i][b].y, acc[r][i][h].y);
                  }
                }
            }
          }
        } else {
          // one group of 128: a lane has 32 consecutive bytes of its rows
          const uint32_t* sc = reinterpret_cast<const uint32_t*>(unit + kRows * kUnitBytes);
          const uint32_t c0 = sc[0], c1 = KIND == kStreamUp ? sc[1] : c0;
          const float s0 = FORM == kFp8Packed ? ue8m0_value(c0 >> (8 * (u & 3))) : __uint_as_float(c0);
          const float s1 = FORM == kFp8Packed ? ue8m0_value(c1 >> (8 * (u & 3))) : __uint_as_float(c1);
          float2 part[R][TILES][2] = {};
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int r = 0; r < R; ++r) {
              const uint8_t* rows = unit + (r * 16 + g) * kUnitBytes + (((2 * t4 + h) ^ g) * 16);
              const uint4 w0 = *reinterpret_cast<const uint4*>(rows), w1 = *reinterpret_cast<const uint4*>(rows + 8 * kUnitBytes);
              const uint32_t lo[4] = {w0.x, w0.y, w0.z, w0.w}, hi[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t f[4] = {e4m3_lo(lo[j]), e4m3_lo(hi[j]), e4m3_hi(lo[j]), e4m3_hi(hi[j])};
#pragma unroll
                for (int i = 0; i < TILES; ++i) mma_16x8x16(part[r][i], f, e4m3_lo(o.x[i][4 * h + j]), e4m3_hi(o.x[i][4 * h + j]));
              }
            }
#pragma unroll
          for (int i = 0; i < TILES; ++i) {
            const float2 f0 = __fmul2_rn(o.s[i][0], make_float2(s0, s0)), f1 = __fmul2_rn(o.s[i][0], make_float2(s1, s1));
#pragma unroll
            for (int r = 0; r < R; ++r) {   // (the bits: see above)
              if (!kCarries || (on >> (2 * i) & 1)) {
                acc[r][i][0].x = fmaf(part[r][i][0].x, f0.x, acc[r][i][0].x);
                acc[r][i][1].x = fmaf(part[r][i][1].x, f1.x, acc[r][i][1].x);
              }
              if (!kCarries || (on >> (2 * i + 1) & 1)) {
                acc[r][i][0].y = fmaf(part[r][i][0].y, f0.y, acc[r][i][0].y);
                acc[r][i][1].y = fmaf(part[r][i][1].y, f1.y, acc[r][i][1].y);
              }
            }
          }
        }
      };
      auto flush = [&](int at) {   // (kStreamDown, kCompact) the expert's sums to its tokens'
        const int first = route.first[at];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int column = i * 8 + 2 * t4 + h;
            if (column < columns) {
              const int t = route.token[first + column];
              float* const to = mine + ((t >> 3) * 4 + (t & 1)) * 32 + g * 4 + ((t & 7) >> 1);
#pragma unroll
              for (int r = 0; r < R; ++r)
#pragma unroll
                for (int q = 0; q < 2; ++q) to[(r * NT * 4 + q * 2) * 32] += h ? acc[r][i][q].y : acc[r][i][q].x;
            }
          }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < NT; ++i) acc[r][i][0] = acc[r][i][1] = make_float2(0.0f, 0.0f);
        __syncwarp();   // (another lane may have the next expert's column of the token)
      };
      if (c.in_item(units_k, active)) shifts(), enter(c);
      while (c.in_item(units_k, active)) {
        if constexpr (kCompact) {
          issue();
          const int used = tiles();
          if (used == 1)
            unit_of(std::integral_constant<int, 1>{});
          else if (NT == 2 || used == 2)
            unit_of(std::integral_constant<int, 2>{});
          else
            unit_of(std::integral_constant<int, NT>{});
        } else {
          unit_of(std::integral_constant<int, NT>{});
        }
        __syncwarp();   // the stage is free for the copies of the next turn
        if (++stage == stages) stage = 0;
        const int at = c.at;
        if (c.step(W, units_k, active)) {
          if constexpr (kCompact && KIND == kStreamDown) flush(at);
          if (c.in_item(units_k, active)) shifts(), enter(c);
        }
      }

      // the warps' sums, in warp order (two buffers by turns: one barrier an item)
      if constexpr (!(kCompact && KIND == kStreamDown)) {
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) mine[((r * NT + i) * 4 + q) * 32 + lane] = q & 1 ? acc[r][i][q >> 1].y : acc[r][i][q >> 1].x;
      }
      __syncthreads();
      const float* const all = sums + (size_t)buffer * W * R * NT * 128;
      auto sum = [&](int m, int l) {   // column m, row l
        const int q = ((l >> 3) & 1) * 2 + m % 2, from = (((l >> 4) * NT + m / 8) * 4 + q) * 32 + (l % 8) * 4 + (m % 8) / 2;
        float s = 0.0f;
        for (int w = 0; w < W; ++w) s += all[w * R * NT * 128 + from];
        return s;
      };
      if constexpr (KIND == kStreamUp) {
        const uint32_t mask = route.mask[route.active[item_at]];
        const int first = route.first[item_at], count = kCompact ? __popc(mask) : tokens;
        for (int o = threadIdx.x; o < 8 * R * count; o += blockDim.x) {
          const int m = o / (8 * R), j = o % (8 * R);
          if (!kCompact && !(mask >> m & 1)) continue;
          const size_t row = (size_t)t0 * a.k + route.row[first + (kCompact ? m : __popc(mask & ((1u << m) - 1)))];
          const int l = (j >> 3) * 16 + (j & 7);
          const float gate = sum(m, l), up = sum(m, l + 8);
          static_cast<float*>(a.out)[row * half + item_block * 8 * R + j] = silu_f32(gate) * up;
        }
      } else {
        for (int o = threadIdx.x; o < kRows * tokens; o += blockDim.x) {
          const int m = o / kRows, j = o % kRows, col = item_block * kRows + j;
          if (col >= a.rows) continue;
          const float v = sum(m, j);
          const size_t to = (size_t)(t0 + m) * a.rows + col;
          if constexpr (OUT_F32)
            static_cast<float*>(a.out)[to] = v;
          else
            static_cast<__nv_bfloat16*>(a.out)[to] = __float2bfloat16_rn(v);
        }
      }
      c.at = item_at;
      c.next_item(warp, units_k, active, blocks);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
  }
  if constexpr (KIND == kStreamDown) {
    if (!waited) griddep_wait();
  }
}

// The cast of h [rows, I] in FP32: E4M3 codes and one FP32 scale per group of 128 (UE: a power of two). A warp a group.
// (No __restrict__: h is written while this kernel may live already, which a read-only load would not allow.)
template <bool UE>
__global__ void __launch_bounds__(256) h_cast_kernel(const float* h, const int32_t* ids, uint8_t* q, float* s, long long groups, int per_row) {
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

template <Kind KIND, WeightForm FORM, int NT, int R, bool OUT_F32, bool WHOLE>
cudaError_t launch_stream_kernel(const FewArgs& a, int rows, const FewPlan& plan, const StreamArgs& s) {
  auto kernel = stream_kernel<KIND, FORM, NT, R, OUT_F32, WHOLE>;
  const int items = (rows + 16 * R - 1) / (16 * R);
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

bool whole_units(const FewArgs& a) { return a.K % 256 == 0 && reinterpret_cast<uintptr_t>(a.sw) % 8 == 0; }

template <Kind KIND, WeightForm FORM, int NT, int R, bool OUT_F32>
cudaError_t launch_stream_nt(const FewArgs& a, int rows, const FewPlan& plan, const StreamArgs& s) {
  constexpr bool kWholeAlone = FORM == kMxfp4 && R == 2;   // (see few_choice)
  if constexpr (FORM == kMxfp4)
    if (kWholeAlone || whole_units(a)) return launch_stream_kernel<KIND, FORM, NT, R, OUT_F32, true>(a, rows, plan, s);
  if constexpr (!kWholeAlone) return launch_stream_kernel<KIND, FORM, NT, R, OUT_F32, false>(a, rows, plan, s);
}

// (rows, units: see few_choice)
template <Kind KIND, WeightForm FORM, int NT, bool OUT_F32>
cudaError_t launch_stream_tokens(const FewArgs& a, int rows, int units, const StreamArgs& s) {
  const FewChoice c = few_choice(a.T, a.k, a.E, rows, units, FORM == kMxfp4, whole_units(a), s.limit.capped);
  if constexpr (few_two_tiles(NT, FORM == kMxfp4))
    if (c.R == 2) return launch_stream_nt<KIND, FORM, NT, 2, OUT_F32>(a, rows, c.plan, s);
  return launch_stream_nt<KIND, FORM, NT, 1, OUT_F32>(a, rows, c.plan, s);
}

template <Kind KIND, WeightForm FORM, bool OUT_F32>
cudaError_t launch_stream(const FewArgs& a, int rows, int units, const StreamArgs& s) {
  const int tiles = few_tiles(a.T);
  if (tiles == 1) return launch_stream_tokens<KIND, FORM, 1, OUT_F32>(a, rows, units, s);
  if (tiles == 2) return launch_stream_tokens<KIND, FORM, 2, OUT_F32>(a, rows, units, s);
  return launch_stream_tokens<KIND, FORM, 4, OUT_F32>(a, rows, units, s);
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
  cudaError_t e = launch_stream<kStreamUp, FORM, true>(up, most * 2 * m.I, (m.K + unit_k - 1) / unit_k, s);
  if (e != cudaSuccess) return e;
  // The cast starts the down product before it waits itself, so that product begins while the up product still runs (as its CTAs leave
  // the SMs): it sets up its routing and fills its rings with weights, and waits only before it reads h. What it reads before (ids,
  // weights, W2 and its scales) was there before the up product, which has waited for all that came ahead of it.
  const long long groups = (long long)rows * (m.I / 128);
  e = launch_plain(FORM == kFp8Packed ? h_cast_kernel<true> : h_cast_kernel<false>, (int)s.limit.all((groups + 7) / 8), 256, 0, s,
                   (const float*)h, m.ids, q, sq, groups, m.I / 128);
  if (e != cudaSuccess) return e;
  FewArgs down{q, sq, m.w2, m.s2, m.ids, m.weights, m.y, m.status, m.T, m.k, m.E, m.I, m.N};
  const int units = (m.I + unit_k - 1) / unit_k * most;
  return out_f32 ? launch_stream<kStreamDown, FORM, true>(down, m.N, units, s) : launch_stream<kStreamDown, FORM, false>(down, m.N, units, s);
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
  const int units = (K + 255) / 256;
  return out_f32 ? launch_stream<kStreamDense, kMxfp4, true>(a, N, units, s) : launch_stream<kStreamDense, kMxfp4, false>(a, N, units, s);
}

}  // namespace dg
