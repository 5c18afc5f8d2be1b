// Eight values of a row a thread, in the two forms that the row-wise kernels of
// mt_model.h share: ALIGNED, eight neighbouring columns that one or two 16-byte
// accesses move (every eighth column of every row starts on 16 bytes and the
// rows are whole chunks long), and else eight columns a row's threads apart, an
// element an access with neighbouring threads side by side, for rows that start
// on any element.  (Words of 16 bytes shifted into place instead take more
// instructions than single elements: a layer norm of 16384 x 8191 bf16 with
// residual 438 us against 279.)
#pragma once

#include <cstdint>

#include "philox.cuh"
#include "row_util.cuh"

namespace mt {
namespace row {

// Eight values as single accesses leave them: a register each, so that nothing
// waits for them before they are used.
template <class T>
struct Loose8 {
  T v[8];
  __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = to_f32(v[k]);
  }
  __device__ __forceinline__ void set(const float (&f)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = from_f32<T>(f[k]);
  }
};
template <class T, bool ALIGNED>
using Eight = typename std::conditional<ALIGNED, Pack8<T>, Loose8<T>>::type;

// THREADS: how many share a row (0: known at run time).
template <bool ALIGNED, int THREADS = 0>
struct Chunk {
  int first, step_;  // columns first + k * step()

  // Chunk i of thread tid of the `threads` that share a row.
  __device__ __forceinline__ Chunk(int i, int tid, int threads = THREADS)
      : first(ALIGNED ? (i * threads + tid) * 8 : i * 8 * threads + tid),
        step_(ALIGNED ? 1 : threads) {}

  __device__ __forceinline__ int step() const {
    return ALIGNED ? 1 : THREADS > 0 ? THREADS : step_;
  }
  __device__ __forceinline__ int col(int k) const { return first + k * step(); }
  // Whether value k exists; whether any does; whether all of the warp's do, which
  // is the way for all but a row's last warps: no test for each element.
  __device__ __forceinline__ bool live(int k, int d) const {
    return ALIGNED ? first < d : col(k) < d;
  }
  __device__ __forceinline__ bool any(int d) const { return first < d; }
  __device__ __forceinline__ bool whole(int d) const {
    return ALIGNED ? first < d : (first | 31) + 7 * step() < d;
  }
  __device__ __forceinline__ int count(int d) const {
    if (whole(d)) return 8;
    int n = 0;
    if constexpr (!ALIGNED) {
#pragma unroll
      for (int k = 0; k < 8; ++k) n += live(k, d);
    }
    return n;
  }

  // The values, those at or past column d zero.
  template <class T>
  __device__ __forceinline__ Eight<T, ALIGNED> load(const Matrix<const T>& m, int64_t row,
                                                    int d) const {
    const int64_t at = row * m.ld + first;
    Eight<T, ALIGNED> o{};
    if constexpr (ALIGNED) {
      if (first < d && m.ok(at, 8)) o = *reinterpret_cast<const Pack8<T>*>(m.p + at);
    } else {
      const T* p = m.p + at;
      if (whole(d)) {
#pragma unroll
        for (int k = 0; k < 8; ++k) o.v[k] = m.ok(at + k * step(), 1) ? p[k * step()] : T(0.0f);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          o.v[k] = live(k, d) && m.ok(at + k * step(), 1) ? p[k * step()] : T(0.0f);
      }
    }
    return o;
  }

  template <class T>
  __device__ __forceinline__ void store(const Matrix<T>& m, int64_t row, int d,
                                        const float (&v)[8]) const {
    if constexpr (ALIGNED) {
      if (first < d) store_step<T, true>(m, row, first, v);
    } else {
      const int64_t at = row * m.ld + first;
      T* p = m.p + at;
      if (whole(d)) {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (m.ok(at + k * step(), 1)) p[k * step()] = from_f32<T>(v[k]);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (live(k, d) && m.ok(at + k * step(), 1)) p[k * step()] = from_f32<T>(v[k]);
      }
    }
  }

  // The blocks' part of the chunk's random words (see Dropout::Columns).  Not
  // ALIGNED: of the two blocks that this lane computes for its quad.
  struct Words {
    Dropout::Columns low, high;
  };
  __device__ __forceinline__ Words words(const Dropout& drop) const {
    const int at = ALIGNED ? 0 : (threadIdx.x & 3) * step(), next = ALIGNED ? 4 : 4 * step();
    return Words{drop.columns(static_cast<uint32_t>(first + at) / 4),
                 drop.columns(static_cast<uint32_t>(first + at + next) / 4)};
  }
  // D() of the values in row r.  Not ALIGNED: whole warps together, `first` and
  // `threads` such that four lanes have a quad of columns.
  __device__ __forceinline__ void drop(const Dropout& drop, const Dropout::Row& r, const Words& w,
                                       float (&v)[8]) const {
    if constexpr (ALIGNED) {
      drop.apply4(r, w.low, v);
      drop.apply4(r, w.high, v + 4);
    } else {
      drop.apply_quad(r, w.low, v);
      drop.apply_quad(r, w.high, v + 4);
    }
  }
};

// What a thread holds of a row: E values in chunks.
template <class T, int E, bool ALIGNED, int THREADS>
struct Chunks {
  static constexpr int COUNT = E / 8;
  Eight<T, ALIGNED> item[COUNT];

  __device__ __forceinline__ void load(const Matrix<const T>& m, int64_t row, int d,
                                       int tid) {
#pragma unroll
    for (int i = 0; i < COUNT; ++i) item[i] = Chunk<ALIGNED, THREADS>(i, tid).load(m, row, d);
  }
  __device__ __forceinline__ void fill(float value) {
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = value;
#pragma unroll
    for (int i = 0; i < COUNT; ++i) item[i].set(v);
  }
  __device__ __forceinline__ void get(int i, float (&v)[8]) const { item[i].get(v); }
};

}  // namespace row
}  // namespace mt
