// Dropout's random words: Philox4x32-10 (Salmon, Moraes, Dror and Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011), the counter-based
// generator of ten rounds of two 32 x 32 -> 64-bit products.  A word depends on
// key and counter alone, so the mask of any element is computed where it is
// needed, forwards and backwards, and is never stored.
//
// Cost: the wide products, which the multiplier takes at a quarter of an
// addition's rate, 20 for four words.  Of the first three rounds' six, two
// depend on the seed and the sequence, or on the row, alone and three on the
// block of columns alone, so a thread that keeps its columns from row to row
// (Columns) computes 15.  With the logic operations, comparisons and
// conversions eight values are some 140 instructions: less than 4 bytes an
// element take to move, so what surrounds them decides.
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
  static constexpr int LATE = 7;  // rounds after the third
  uint32_t k0, k1, s0, s1, border;
  float scale;
  uint32_t a_[LATE], b_[LATE];  // their keys

  static constexpr uint32_t M0 = 0xD2511F53u, M1 = 0xCD9E8D57u;
  static constexpr uint32_t W0 = 0x9E3779B9u, W1 = 0xBB67AE85u;

  __device__ __forceinline__ void init(const DropoutArgs& a) {
    const uint64_t key = static_cast<uint64_t>(*a.seed);
    k0 = static_cast<uint32_t>(key);
    k1 = static_cast<uint32_t>(key >> 32);
    s0 = a.sequence_lo;
    s1 = a.sequence_hi;
    border = a.border;
    scale = a.scale;
#pragma unroll
    for (uint32_t i = 0; i < LATE; ++i) {
      a_[i] = k0 + (i + 3) * W0;
      b_[i] = k1 + (i + 3) * W1;
      // Opaque, so that they stay in registers: the compiler would rather add
      // them up again for every block, 14 of 137 instructions for eight words.
      asm("" : "+r"(a_[i]), "+r"(b_[i]));
    }
  }

  static __device__ __forceinline__ uint32_t hi(uint64_t v) {
    return static_cast<uint32_t>(v >> 32);
  }
  static __device__ __forceinline__ uint32_t lo(uint64_t v) { return static_cast<uint32_t>(v); }
  static __device__ __forceinline__ uint64_t wide(uint32_t m, uint32_t v) {
    return static_cast<uint64_t>(m) * v;
  }

  // A round takes (c0, c1, c2, c3) to (hi(M1 c2) ^ c1 ^ a, lo(M1 c2), hi(M0 c0) ^
  // c3 ^ b, lo(M0 c0)), a and b the round's keys.  From (block, row, s0, s1):
  //   after one    (hi(M1 s0) ^ row ^ a0, lo(M1 s0), hi(M0 block) ^ s1 ^ b0, lo(M0 block)):
  //                the first of the row alone, the last two of the block alone;
  //   after two    (of the block, of the block, hi of the row ^ of the block, of the row),
  // and the third round's M0 product is of the block alone again.

  // What a row adds: the words of its product of the second round.
  struct Row {
    uint32_t h, l;
  };
  __device__ __forceinline__ Row row(uint32_t row) const {
    const uint64_t p = wide(M0, hi(wide(M1, s0)) ^ row ^ k0);
    return Row{hi(p), lo(p)};
  }
  // What a block of four columns adds.
  struct Columns {
    uint32_t c1, c2, h, l;
  };
  __device__ __forceinline__ Columns columns(uint32_t block) const {
    const uint64_t p0 = wide(M0, block), p1 = wide(M1, hi(p0) ^ s1 ^ k1);
    const uint64_t q = wide(M0, hi(p1) ^ lo(wide(M1, s0)) ^ (k0 + W0));
    return Columns{lo(p1) ^ (k0 + 2 * W0), lo(p0) ^ (k1 + W1), hi(q) ^ (k1 + 2 * W1), lo(q)};
  }
  // The block's four words in the row: the rest of round three, and seven more.
  __device__ __forceinline__ void words(const Row& r, const Columns& c, uint32_t (&w)[4]) const {
    const uint64_t p = wide(M1, r.h ^ c.c2);
    uint32_t c0 = hi(p) ^ c.c1, c1 = lo(p), c2 = c.h ^ r.l, c3 = c.l;
#pragma unroll
    for (int i = 0; i < LATE; ++i) {
      const uint64_t p0 = wide(M0, c0), p1 = wide(M1, c2);
      c0 = hi(p1) ^ c1 ^ a_[i];
      c1 = lo(p1);
      c2 = hi(p0) ^ c3 ^ b_[i];
      c3 = lo(p0);
    }
    w[0] = c0;
    w[1] = c1;
    w[2] = c2;
    w[3] = c3;
  }

  // Four values by their words.
  __device__ __forceinline__ void apply(float* v, const uint32_t (&w)[4]) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = w[i] >= border ? v[i] * scale : 0.0f;
  }

  // D() of a block's four columns.
  __device__ __forceinline__ void apply4(const Row& r, const Columns& c, float* v) const {
    uint32_t w[4];
    words(r, c, w);
    apply(v, w);
  }
  // D() of four values of four neighbouring lanes each, value i of the lanes
  // being block i's columns in order; lane l gives the block of value l.  The
  // quad transposes its 4 x 4 words.  All 32 lanes call it together.
  __device__ __forceinline__ void apply_quad(const Row& r, const Columns& c, float* v) const {
    const bool odd = threadIdx.x & 1, upper = threadIdx.x & 2;
    uint32_t w[4];
    words(r, c, w);
    uint32_t x = __shfl_xor_sync(0xffffffffu, odd ? w[0] : w[1], 1);
    uint32_t y = __shfl_xor_sync(0xffffffffu, odd ? w[2] : w[3], 1);
    if (odd) w[0] = x, w[2] = y;
    else w[1] = x, w[3] = y;
    x = __shfl_xor_sync(0xffffffffu, upper ? w[0] : w[2], 2);
    y = __shfl_xor_sync(0xffffffffu, upper ? w[1] : w[3], 2);
    if (upper) w[0] = x, w[1] = y;
    else w[2] = x, w[3] = y;
    apply(v, w);
  }
};

}  // namespace row
}  // namespace mt
