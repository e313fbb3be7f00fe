// dg_scale.cuh — the scale of a group of 128 values that are cast to E4M3, and its place among A's scales.
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

namespace dg {

// The factor to codes and the scale of a group: FP32 bits, or a UE8M0 code.
template <bool UE>
__device__ __forceinline__ void group_scale(float amax, float& factor, uint32_t& scale) {
  const float a = fmaxf(amax, 0x1p-100f);
  if constexpr (UE) {
    const uint32_t bits = __float_as_uint(a), e = bits >> 23;
    uint32_t code = e - 8u + ((bits & 0x7FFFFFu) > 0x600000u ? 1u : 0u);   // 448 = 1.75 · 2^8
    if (amax == 0.0f) code = 127u;
    factor = __uint_as_float((254u - code) << 23);
    if (e == 255u) { code = 255u; factor = 0.0f; }
    scale = code;
  } else {
    factor = amax == 0.0f ? 1.0f : __fdiv_rn(448.0f, a);
    scale = __float_as_uint(amax == 0.0f ? 1.0f : __fdiv_rn(a, 448.0f));
  }
}

// Puts the scale of group `kb` (of nkb along the contraction) of line `i`: FP32 at [kb][i] of lines of
// `stride`, or byte kb % 4 of word [kb / 4][i]; the last group also fills its word's unused bytes.
template <bool UE>
__device__ __forceinline__ void put_scale_major(void* base, size_t first_kb, int kb, int nkb, size_t stride, size_t i,
                                                uint32_t scale) {
  if constexpr (UE) {
    uint8_t* p = static_cast<uint8_t*>(base) + ((first_kb + kb / 4) * stride + i) * 4;
    p[kb & 3] = (uint8_t)scale;
    if (kb == nkb - 1)
      for (int j = (kb & 3) + 1; j < 4; ++j) p[j] = 127;
  } else {
    static_cast<uint32_t*>(base)[(first_kb + kb) * stride + i] = scale;
  }
}

}  // namespace dg
