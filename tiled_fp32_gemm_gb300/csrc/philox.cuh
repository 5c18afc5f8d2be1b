// Dropout's random words: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011), the counter-based
// generator of ten rounds of two 32 x 32 -> 64-bit products.  A word depends on
// key and counter alone, so the mask of any element is computed where it is
// needed, forwards and backwards, and is never stored.
//
// Cost: 20 wide products, 40 three-input logic operations and the key's
// additions (the same for every thread) for four words.  Beside 4 to 10 bytes
// an element of memory traffic that is the smaller part of a pass as long as
// every word is used, so threads that hold single columns share the blocks
// (words_of_columns).
#pragma once

#include <cstdint>

#include "device_util.cuh"

namespace mt {

// What a kernel needs to drop elements; by value, made on the host.
struct DropoutArgs {
  const int64_t* seed;  // one value, read by the kernel
  uint32_t sequence_lo, sequence_hi;
  uint32_t border;  // words below it drop
  float scale;      // 1 / (1 - p)
};

namespace row {

struct Dropout {
  uint32_t k0, k1, s0, s1, border;
  float scale;

  __device__ __forceinline__ void init(const DropoutArgs& a) {
    const uint64_t key = static_cast<uint64_t>(*a.seed);
    k0 = static_cast<uint32_t>(key);
    k1 = static_cast<uint32_t>(key >> 32);
    s0 = a.sequence_lo;
    s1 = a.sequence_hi;
    border = a.border;
    scale = a.scale;
  }

  // The four words of columns 4 * block .. 4 * block + 3 of a row.
  __device__ __forceinline__ void words(uint32_t row, uint32_t block, uint32_t (&w)[4]) const {
    uint32_t c0 = block, c1 = row, c2 = s0, c3 = s1, a = k0, b = k1;
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
      const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
      c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ a;
      c1 = static_cast<uint32_t>(p1);
      c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ b;
      c3 = static_cast<uint32_t>(p0);
      a += 0x9E3779B9u;
      b += 0xBB67AE85u;
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
  }

  __device__ __forceinline__ float apply(float v, uint32_t word) const {
    return word >= border ? v * scale : 0.0f;
  }

  // D() of columns c .. c + 7 of a row, c a multiple of 8.
  __device__ __forceinline__ void apply8(uint32_t row, int c, float (&v)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; k += 4) {
      uint32_t w[4];
      words(row, static_cast<uint32_t>(c + k) / 4, w);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k + i] = apply(v[k + i], w[i]);
    }
  }

  // The words of the N columns c0 + i * step (N and step multiples of 4) of a
  // lane whose warp's lanes hold neighbouring columns, c0 % 4 == lane % 4: lane
  // l of a quad computes the block of the quad's columns for every fourth step,
  // from step l on, and the quad transposes its 4 x 4 words.  All 32 lanes call
  // it together.
  template <int N>
  __device__ __forceinline__ void words_of_columns(uint32_t row, int c0, int step,
                                                   uint32_t (&out)[N]) const {
    static_assert(N % 4 == 0, "whole quads");
    const int at = threadIdx.x & 3;
    const bool odd = at & 1, upper = at & 2;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      uint32_t w[4];
      words(row, static_cast<uint32_t>(c0 + (i + at) * step) / 4, w);
      uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
      uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
      if (odd) w[0] = x, w[2] = y;
      else w[1] = x, w[3] = y;
      x = __shfl_xor_sync(0xffffffffu, upper ? w[0] : w[2], 2);
      y = __shfl_xor_sync(0xffffffffu, upper ? w[1] : w[3], 2);
      if (upper) w[0] = x, w[1] = y;
      else w[2] = x, w[3] = y;
#pragma unroll
      for (int s = 0; s < 4; ++s) out[i + s] = w[s];
    }
  }
};

}  // namespace row
}  // namespace mt
