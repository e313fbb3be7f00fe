// dg_gated.cuh — the epilogue of the gated projection H = dropout(silu(X·Wgᵀ) · (X·Wuᵀ)) in the dense
// and contiguous forms, shared by the FP32-scale and the block-scaled kernel.
//
// A tile covers 128 (BN = 256) or 64 (BN = 128) columns of H: as many gate rows and the matching up rows of
// the weights. Each epilogue warp holds, for its 32 rows, HC = 64 or 32 gate columns (acc[0..]) and the same
// up columns (acc[HC..]), so silu(g)·u needs no exchange between warps. On request it also stores the pre-activations, rounded to
// BF16, at columns [j] (gate) and [I + j] (up) of GU, for the backward pass. H is formed from the FP32
// values. Whole 32-row slabs leave through TMA (64-byte boxes, two staging buffers a warp);
// slabs with rows that must stay untouched use predicated 16-byte stores.
#pragma once

#include <cuda.h>

#include <cstdint>
#include <type_traits>

#include "dg_philox.cuh"
#include "dg_ptx.cuh"
#include "dg_vec.cuh"

namespace dg {

// What the gated kernels take beside GemmParams.
struct GatedExt {
  CUtensorMap tmGU;   // GU, BF16 [rows, 2I]: boxes of 32 rows x 32 columns (valid, unused where gu is null)
  uint16_t* gu;       // the saved pre-activations, or null
  Dropout drop;
};
struct NoExt {};

// silu(x) = x / (1 + e^-x), the gate function of SwiGLU, with the fast exponential and division
// (relative error ~1e-6). For x below about -87 the denominator overflows and the quotient is -0, the
// function's limit. (An IEEE-rounded division or reciprocal there takes a slow special-case path:
// it made the fused kernel 50% slower than the GEMM alone on decode-sized outputs.)
__device__ __forceinline__ float silu_f32(float x) { return __fdividef(x, 1.0f + __expf(-x)); }

// Four columns of one row (col a multiple of 4), from the summed pre-activations: h and (on request) g and
// u to memory. The path of the rows that a cluster split reduces.
template <bool OUT_F32>
__device__ __forceinline__ void gated_store4(const GatedExt& e, void* H, int I, size_t row, int col, const float4& g,
                                             const float4& u) {
  if (e.gu) {
    uint16_t* to = e.gu + row * 2 * I + col;
    *reinterpret_cast<uint2*>(to) = make_uint2(round_bf16x2(g.x, g.y), round_bf16x2(g.z, g.w));
    *reinterpret_cast<uint2*>(to + I) = make_uint2(round_bf16x2(u.x, u.y), round_bf16x2(u.z, u.w));
  }
  float4 h = make_float4(silu_f32(g.x) * u.x, silu_f32(g.y) * u.y, silu_f32(g.z) * u.z, silu_f32(g.w) * u.w);
  if (e.drop.threshold) {
    const uint4 w = Philox(e.drop.rng)((row * I + col) / 8);
    const int j = col & 4;
    h.x = dropout1(h.x, w, j, e.drop.threshold, e.drop.scale);
    h.y = dropout1(h.y, w, j + 1, e.drop.threshold, e.drop.scale);
    h.z = dropout1(h.z, w, j + 2, e.drop.threshold, e.drop.scale);
    h.w = dropout1(h.w, w, j + 3, e.drop.threshold, e.drop.scale);
  }
  if constexpr (OUT_F32)
    *reinterpret_cast<float4*>(static_cast<float*>(H) + row * I + col) = h;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(H) + row * I + col) =
        make_uint2(round_bf16x2(h.x, h.y), round_bf16x2(h.z, h.w));
}

// One 32-row x 64-byte box (32 BF16 or 16 FP32 columns, v[0..]) through the warp's staging buffers.
template <bool F32>
__device__ __forceinline__ void gated_box(const CUtensorMap* tm, uint8_t* staging, uint32_t box_bytes, uint32_t& count,
                                          const float* v, int col, int row, int lane) {
  const uint32_t sel = count & 1;
  if (count >= 2) {
    if (lane == 0) tma_store_wait_read_1();   // the box that used this buffer has been read
    __syncwarp();
  }
  uint8_t* buf = staging + sel * box_bytes;
#pragma unroll
  for (int j = 0; j < 4; ++j) {   // four 16-byte pieces per 64-byte row, 64-byte swizzle
    const uint32_t phys = (uint32_t)(j ^ ((lane >> 1) & 3));
    uint4 w;
    if constexpr (F32)
      w = make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]), __float_as_uint(v[4 * j + 2]),
                     __float_as_uint(v[4 * j + 3]));
    else
      w = make_uint4(round_bf16x2(v[8 * j], v[8 * j + 1]), round_bf16x2(v[8 * j + 2], v[8 * j + 3]),
                     round_bf16x2(v[8 * j + 4], v[8 * j + 5]), round_bf16x2(v[8 * j + 6], v[8 * j + 7]));
    *reinterpret_cast<uint4*>(buf + lane * 64 + phys * 16) = w;
  }
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_2d(tm, buf, col, row);
    tma_store_commit();
  }
  ++count;
  __syncwarp();
}

// The epilogue of one warp's 32 rows x HC columns of H. row0: its first row of H; write_row: whether this
// lane's row is stored; all_rows: whether TMA may store the slab (rows past the matrix are clipped there).
// Boxes go out in the order G, U, H of each 32 columns, so that the staging buffers drain while h is formed.
template <bool OUT_F32, int HC>
__device__ __forceinline__ void gated_epilogue(const GatedExt& e, const CUtensorMap* tmH, void* H, int I, float* acc,
                                               int row0, int col0, bool write_row, bool all_rows, uint8_t* staging,
                                               uint32_t box_bytes, uint32_t& count, int lane) {
  const size_t row = (size_t)row0 + lane;
  auto form_h = [&](int b) {   // columns 32·b .. of H, in place of their gate values
#pragma unroll
    for (int j = 32 * b; j < 32 * b + 32; ++j) acc[j] = silu_f32(acc[j]) * acc[HC + j];
    if (e.drop.threshold) {
      const Philox gen(e.drop.rng);
      const uint64_t index = (row * I + col0) / 8;
#pragma unroll
      for (int j = 32 * b; j < 32 * b + 32; j += 8)
        dropout8(*reinterpret_cast<float(*)[8]>(acc + j), gen(index + j / 8), e.drop.threshold, e.drop.scale);
    }
  };
  if (all_rows) {
#pragma unroll
    for (int b = 0; b < HC / 32; ++b) {
      if (e.gu) {
        gated_box<false>(&e.tmGU, staging, box_bytes, count, acc + 32 * b, col0 + 32 * b, row0, lane);
        gated_box<false>(&e.tmGU, staging, box_bytes, count, acc + HC + 32 * b, I + col0 + 32 * b, row0, lane);
      }
      form_h(b);
      constexpr int kCols = OUT_F32 ? 16 : 32;
#pragma unroll
      for (int c = 32 * b; c < 32 * b + 32; c += kCols)
        gated_box<OUT_F32>(tmH, staging, box_bytes, count, acc + c, col0 + c, row0, lane);
    }
  } else if (write_row) {
    if (e.gu) {
      __nv_bfloat16* dst = reinterpret_cast<__nv_bfloat16*>(e.gu) + row * 2 * I + col0;
#pragma unroll
      for (int j = 0; j < 2 * HC; j += 8)
        store8(dst + (j >= HC ? I - HC : 0) + j, *reinterpret_cast<float(*)[8]>(acc + j));
    }
#pragma unroll
    for (int b = 0; b < HC / 32; ++b) form_h(b);
#pragma unroll
    for (int j = 0; j < HC; j += 8) {
      if constexpr (OUT_F32)
        store8(static_cast<float*>(H) + row * I + col0 + j, *reinterpret_cast<float(*)[8]>(acc + j));
      else
        store8(static_cast<__nv_bfloat16*>(H) + row * I + col0 + j, *reinterpret_cast<float(*)[8]>(acc + j));
    }
  }
}

// Cluster split-K: sums the rows r = rank (mod S) of the S partial tiles of a cluster in range order and
// stores them. `part`: this CTA's partial tile in shared memory, rows of `row_bytes`, tile columns as
// the epilogue warps hold them: [HC gate | HC up] for columns 0..HC-1 of H, then for the next HC.
// m_indices: the contiguous form's rows (null: dense); g: the tile's group.
template <bool OUT_F32, int HC>
__device__ __forceinline__ void gated_cluster_reduce(const GatedExt& e, void* H, int I, uint32_t part, uint32_t row_bytes,
                                                     int S, int rank, int threads, int a_row, int rows, int n_blk, int g,
                                                     const int32_t* m_indices, int* status, int bad_group_bit) {
  // Neighbouring lanes read neighbouring float4, HC/4 of them side by side. (Lanes of 8 columns, 32 bytes
  // apart, cost 4 us a tile more: 64x4096x7168 16.4 us instead of 12.3.)
  constexpr int kLanes = HC / 2;                                    // lanes a row
  const int c = (threadIdx.x % kLanes) * 4;                         // first of four columns of H in the tile
  const uint32_t off = (uint32_t)((c / HC) * 2 * HC + c % HC) * 4;  // their gate partials; up HC columns on
  for (int r = rank + (int)(threadIdx.x / kLanes) * S; r < rows; r += threads / kLanes * S) {
    const uint32_t at = part + r * row_bytes + off;
    // every peer's two float4 are requested before the first add
    float4 gs[kMaxClusterCtas], us[kMaxClusterCtas];
#pragma unroll
    for (int s = 0; s < kMaxClusterCtas; ++s)
      if (s < S) {
        const uint32_t peer = cluster_map(at, (uint32_t)s);
        gs[s] = ld_cluster_v4(peer);
        us[s] = ld_cluster_v4(peer + HC * 4);
      }
    float4 g4 = make_float4(0.0f, 0.0f, 0.0f, 0.0f), u4 = g4;
#pragma unroll
    for (int s = 0; s < kMaxClusterCtas; ++s)
      if (s < S) {
        g4.x += gs[s].x; g4.y += gs[s].y; g4.z += gs[s].z; g4.w += gs[s].w;
        u4.x += us[s].x; u4.y += us[s].y; u4.z += us[s].z; u4.w += us[s].w;
      }
    if (m_indices) {
      const int idx = __ldg(m_indices + a_row + r);
      if (idx != g) {
        if (idx != -1 && c == 0) atomicOr(status, bad_group_bit);
        continue;   // a padding row (or another group's): left untouched
      }
    }
    gated_store4<OUT_F32>(e, H, I, (size_t)a_row + r, n_blk * 2 * HC + c, g4, u4);
  }
}

}  // namespace dg
