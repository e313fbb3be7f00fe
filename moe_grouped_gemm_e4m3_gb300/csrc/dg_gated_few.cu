// dg_gated_few.cu — the dense gated projection for a few tokens (serving's decode step).
//
// With M tokens of at most 8·NT the product is a read of the weights: 2·I·K bytes, against M·4·I·K
// operations. The tiled kernel spends 128-row tiles, a cluster exchange and their barriers on it
// (the read of 1x4096x7168 is 4.4 us). Here nothing is staged: one CTA owns 8 columns of H,
// i.e. 8 gate rows and the matching 8 up rows, the 16 rows of one mma.sync m16n8k32 (E4M3, FP32
// accumulation) whose 8 columns are tokens, so each thread ends up with the gate and the up value of the
// same (token, column). The CTA's warps take every WARPS-th K-block; a lane loads 16 bytes of its row at a
// time, straight into operand registers (the order of k inside a K-block is free as long as both operands
// use the same one). The K-block's partial is scaled by sA·sB into FP32
// accumulators, as in the tiled kernels; the warps' sums are added in warp order through shared
// memory (deterministic). mma.sync is below tcgen05's rate by far, but the tensor pipe idles here
// either way: the bound is the weights' read. 1x4096x7168: 7.8 us, 3.8 TB/s, about 2 us of it the launch; the tiled
// kernel 12.9. Measured (us, here / tiled; 2I = 4096, K = 7168 and 2I = K = 2048): FP32 scales 8 tokens 7.9 / 12.8 and 2.7 / 6.3,
// 16 tokens 10.3 / 13.7 and 3.0 / 6.3; packed scales 8 tokens 7.8 / 12.1 and 2.5 / 6.1, 16 tokens 10.6 / 12.2 and 3.0 / 6.3.
// Each further 8 tokens read the activations once more per 16 weight rows and take as many accumulators again, so the tiled
// kernel has the rest (17 tokens 12.9 and 6.3, packed 12.4 and 6.4).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "dg_launch.h"
#include "dg_vec.cuh"

namespace dg {

namespace {

// Warps a CTA and K-blocks in flight a warp, two CTAs an SM. Measured at 2I = 4096, K = 7168 and 2I = 2048, K = 2048
// (us, FP32 scales; weights from HBM): M = 1: 16 warps x 1 K-block 7.8 and 2.5, 8 x 4 7.7 and 3.0, 8 x 2 8.1 and
// 2.7, 8 x 1 (4 CTAs an SM) 9.7 and 3.2, 4 x 4 9.5 and 3.0; M = 16: 8 x 2 10.3 and 3.4, 16 x 1 13.4 and 4.3.
template <int NT>
struct FewPlan {
  static constexpr int kWarps = NT == 1 ? 16 : 8, kBatch = NT == 1 ? 1 : 2, kThreads = kWarps * 32;
};

// The loads of a batch, volatile so that all of them are issued before its first product (left free, the
// compiler sank the scales' loads to their uses, each a round trip to L2).
__device__ __forceinline__ uint4 load_16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t load_4(const uint32_t* p) {
  uint32_t v;
  asm volatile("ld.global.u32 %0, [%1];" : "=r"(v) : "l"(p));
  return v;
}

__device__ __forceinline__ uint4 load_stream(const uint8_t* p) {   // read once: not kept in L1
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

__device__ __forceinline__ void mma_16x8x32(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                            uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3]) : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The scale of K-block kb from its 32 bits: FP32, or byte kb % 4 of a packed word.
template <bool UE>
__device__ __forceinline__ float scale_value(uint32_t bits, int kb) {
  if constexpr (!UE) return __uint_as_float(bits);
  return ue8m0_value(bits >> (8 * (kb & 3)));
}

// CAPPED: fewer CTAs than groups of 8 columns (dg_set_num_sms), each taking several; a loop in the other form spills.
template <bool UE, bool OUT_F32, int NT, bool CAPPED>
__global__ void __launch_bounds__(FewPlan<NT>::kThreads, 2)
    gated_few_kernel(const uint8_t* A, const void* sA, const uint8_t* B, const void* sB, void* H, uint16_t* GU, const Dropout drop, int M, int I, int K) {
  constexpr int kWarps = FewPlan<NT>::kWarps, kBatch = FewPlan<NT>::kBatch;
  __shared__ float sums[kWarps][NT][4][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int nkb = (K + 127) / 128, nkq = (nkb + 3) / 4, ldsa = (M + 3) / 4 * 4;
  auto columns = [&](int j0) {   // 8 columns of H
    const int nb_gate = j0 / 128, nb_up = I / 128 + nb_gate;
    const uint8_t* gate = B + (size_t)(j0 + g) * K;
    const uint8_t* up = gate + (size_t)I * K;

    float acc[NT][4] = {};
    for (int kb0 = warp; kb0 < nkb; kb0 += kWarps * kBatch) {
      uint4 w[kBatch][4], x[kBatch][NT][2];   // w: gate and up, 64-byte halves 0 and 1
      uint32_t sg[kBatch], su[kBatch], sx[kBatch][NT][2];
      const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int kb = kb0 + i * kWarps;
        const bool some = kb < nkb;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int k = kb * 128 + c * 64 + t * 16;
          const bool live = some && k < K;
          w[i][c] = live ? load_stream(gate + k) : zero;
          w[i][2 + c] = live ? load_stream(up + k) : zero;
#pragma unroll
          for (int n = 0; n < NT; ++n)
            x[i][n][c] = live && n * 8 + g < M ? load_16(A + (size_t)(n * 8 + g) * K + k) : zero;
        }
        // (FP32 scales one a K-block, packed words one a four)
        const int kq = UE ? kb / 4 : kb, ns = UE ? nkq : nkb;
        const uint32_t *a = static_cast<const uint32_t*>(sA), *b = static_cast<const uint32_t*>(sB);
        sg[i] = some ? load_4(b + (size_t)nb_gate * ns + kq) : 0u;
        su[i] = some ? load_4(b + (size_t)nb_up * ns + kq) : 0u;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const int m = n * 8 + 2 * t + c;
            sx[i][n][c] = some && m < M ? load_4(a + (size_t)kq * ldsa + m) : 0u;
          }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int kb = kb0 + i * kWarps;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint4 &a = w[i][c], &b = w[i][2 + c], &v = x[i][n][c];
            mma_16x8x32(part, a.x, b.x, a.y, b.y, v.x, v.y);
            mma_16x8x32(part, a.z, b.z, a.w, b.w, v.z, v.w);
          }
#pragma unroll
          for (int q = 0; q < 4; ++q) {   // rows g (gate: q = 0, 1) and g + 8 (up), tokens 2t and 2t + 1
            const float s = scale_value<UE>(q < 2 ? sg[i] : su[i], kb), m = scale_value<UE>(sx[i][n][q & 1], kb);
            acc[n][q] = fmaf(part[q], m * s, acc[n][q]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int q = 0; q < 4; ++q) sums[warp][n][q][lane] = acc[n][q];
    __syncthreads();
    // thread -> (token, column): the column fastest, so that a token's 8 columns are stored together
    for (int o = threadIdx.x; o < 8 * M; o += kWarps * 32) {
      const int m = o / 8, j = o % 8, n = m / 8, from = j * 4 + (m % 8) / 2, q = m % 2;
      float gs = 0.0f, us = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        gs += sums[w][n][q][from];
        us += sums[w][n][2 + q][from];
      }
      if (GU) {
        __nv_bfloat16* row = reinterpret_cast<__nv_bfloat16*>(GU) + (size_t)m * 2 * I;
        row[j0 + j] = __float2bfloat16_rn(gs);
        row[I + j0 + j] = __float2bfloat16_rn(us);
      }
      float h = silu_f32(gs) * us;
      if (drop.threshold) h = dropout1(h, Philox(drop.rng)(((size_t)m * I + j0) / 8), j, drop.threshold, drop.scale);
      if constexpr (OUT_F32)
        static_cast<float*>(H)[(size_t)m * I + j0 + j] = h;
      else
        static_cast<__nv_bfloat16*>(H)[(size_t)m * I + j0 + j] = __float2bfloat16_rn(h);
    }
  };
  if constexpr (CAPPED) {
    for (int j0 = blockIdx.x * 8; j0 < I; j0 += gridDim.x * 8) {
      columns(j0);
      __syncthreads();   // the sums have been read
    }
  } else {
    columns(blockIdx.x * 8);
  }
}

}  // namespace

cudaError_t launch_gated_few(const uint8_t* A, const void* sA, const uint8_t* B, const void* sB, void* H, uint16_t* GU,
                             const Dropout& drop, int M, int I, int K, bool out_f32, bool ue8m0, const StreamArgs& s) {
  const int grid = (int)s.limit.all(I / 8);
  auto pick = [&](auto nt, auto capped) {
    constexpr int NT = decltype(nt)::value;
    constexpr bool CAPPED = decltype(capped)::value;
    auto go = [&](auto kernel) {
      return launch_plain(kernel, grid, FewPlan<NT>::kThreads, 0, s, A, sA, B, sB, H, GU, drop, M, I, K);
    };
    if (ue8m0) return out_f32 ? go(gated_few_kernel<true, true, NT, CAPPED>) : go(gated_few_kernel<true, false, NT, CAPPED>);
    return out_f32 ? go(gated_few_kernel<false, true, NT, CAPPED>) : go(gated_few_kernel<false, false, NT, CAPPED>);
  };
  auto pick_tokens = [&](auto capped) {
    return M <= 8 ? pick(std::integral_constant<int, 1>{}, capped) : pick(std::integral_constant<int, 2>{}, capped);
  };
  return grid < I / 8 ? pick_tokens(std::true_type{}) : pick_tokens(std::false_type{});
}

}  // namespace dg
