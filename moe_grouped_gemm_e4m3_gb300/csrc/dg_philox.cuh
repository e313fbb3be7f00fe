// dg_philox.cuh — the counter-based generator behind dropout, and its element mask.
//
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy as 1, 2, 3", SC'11):
// ten rounds over a 128-bit counter under a 64-bit key give four 32-bit words. One counter serves
// eight consecutive elements, 16 bits each: element i of a tensor (row-major flat index) takes half
// i % 2 (0: low) of word (i % 8) / 2 of the counter {i / 8 (64 bits), offset (64 bits)} under the key
// `seed`. It is kept when those 16 bits are at least the threshold T = round(65536 p), and then scaled
// by 65536 / (65536 - T), the inverse of the exact keep probability. So a mask is a function of
// (seed, offset, i, T) and is never stored.
#pragma once

#include <cstdint>

#include "dg_ptx.cuh"

namespace dg {

struct Dropout {
  const uint64_t* rng;   // device: {seed, offset}; read by the kernels, never by the host
  uint32_t threshold;    // T; 0: no dropout (rng is not read)
  float scale;           // 65536 / (65536 - T)
};

// The state of one thread: the key and the constant half of the counter.
struct Philox {
  uint32_t k0 = 0, k1 = 0, c2 = 0, c3 = 0;
  __device__ __forceinline__ Philox() {}
  __device__ __forceinline__ explicit Philox(const uint64_t* rng) {
    // (in place: loads that the compiler gathers cost the few-token gated projection registers, which it then spills)
    const uint64_t seed = load_here(rng), offset = load_here(rng + 1);
    k0 = (uint32_t)seed;
    k1 = (uint32_t)(seed >> 32);
    c2 = (uint32_t)offset;
    c3 = (uint32_t)(offset >> 32);
  }
  // The four words of counter `index`.
  __device__ __forceinline__ uint4 operator()(uint64_t index) const {
    uint32_t x0 = (uint32_t)index, x1 = (uint32_t)(index >> 32), x2 = c2, x3 = c3, a = k0, b = k1;
#pragma unroll
    for (int r = 0; r < 10; ++r) {
      const uint64_t p = (uint64_t)0xD2511F53u * x0, q = (uint64_t)0xCD9E8D57u * x2;
      x0 = (uint32_t)(q >> 32) ^ x1 ^ a;
      x1 = (uint32_t)q;
      x2 = (uint32_t)(p >> 32) ^ x3 ^ b;
      x3 = (uint32_t)p;
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    return make_uint4(x0, x1, x2, x3);
  }
};

// Dropout of the eight elements of one counter: dropped elements become 0, whatever they were (a NaN
// or an infinity too); kept ones are multiplied by `scale`.
__device__ __forceinline__ void dropout8(float (&v)[8], const uint4& w, uint32_t threshold, float scale) {
  const uint32_t t = threshold << 16;   // threshold <= 65535
  const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = (words[j] << 16) >= t ? __fmul_rn(v[2 * j], scale) : 0.0f;
    v[2 * j + 1] = words[j] >= t ? __fmul_rn(v[2 * j + 1], scale) : 0.0f;
  }
}

// The same for element j (of eight) alone.
__device__ __forceinline__ float dropout1(float v, const uint4& w, int j, uint32_t threshold, float scale) {
  const uint32_t word = j < 4 ? (j < 2 ? w.x : w.y) : (j < 6 ? w.z : w.w);
  return ((word >> (16 * (j & 1))) & 0xFFFFu) >= threshold ? __fmul_rn(v, scale) : 0.0f;
}

}  // namespace dg
