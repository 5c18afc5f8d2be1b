// Device helpers of the row-wise kernels: element loads and stores of the
// storage types, reductions over the threads that share a row.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_util.cuh"

namespace mt {
namespace row {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// Two e4m3 values, `lo` in the low byte (nearest even, values past 448
// clamped to it, NaN kept).
__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Sum and maximum over a warp.
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

// A strided matrix a row-wise kernel reads or writes.  Eight consecutive
// values move as 16-byte accesses (8 bytes for e4m3): the caller has checked
// the alignment of every such column of every row.  The checked build tests
// each access.
template <class T>
struct Matrix {
  T* p;
  int64_t ld, extent;
  BoundsRecord* rec;

  __device__ __forceinline__ bool ok(int64_t at, int width) const {
    return bounds_ok(rec, SITE_ROWS, at, width, extent);
  }
  __device__ __forceinline__ float load(int64_t row, int col) const {
    const int64_t at = row * ld + col;
    return ok(at, 1) ? to_f32(p[at]) : 0.0f;
  }
  __device__ __forceinline__ void store(int64_t row, int col, float v) const {
    const int64_t at = row * ld + col;
    if (ok(at, 1)) p[at] = from_f32<T>(v);
  }
};

// Eight values of a storage type as they lie in memory.
template <class T>
struct Pack8;
template <>
struct Pack8<float> {
  float4 lo, hi;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
    v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    lo = make_float4(v[0], v[1], v[2], v[3]);
    hi = make_float4(v[4], v[5], v[6], v[7]);
  }
};
template <>
struct Pack8<__half> {
  uint4 u;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Pack8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    u = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// The 16 bytes at `p` plus `shift` bytes (shift < 16), from two aligned
// 16-byte words.
__device__ __forceinline__ uint4 shifted(const uint4& lo, const uint4& hi, int shift) {
  uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
  if (shift & 8) {
#pragma unroll
    for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
  }
  if (shift & 4) {
#pragma unroll
    for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
  }
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) o[i] = __funnelshift_r(w[i], w[i + 1], 8 * (shift & 3));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// load8_any where the aligned words reach outside the matrix (its first and
// last rows): out of line, so the common path keeps its registers.
template <class T>
__device__ __noinline__ uint4 load8_single(const T* p, int count) {
  uint32_t w[4] = {0u, 0u, 0u, 0u};
  for (int i = 0; i < count; ++i)
    w[i / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i]) << (16 * (i % 2));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Columns c .. c + 7 of a row of d 16-bit values that may start on any
// element (those at or past d zero): two aligned words, shifted, or single
// elements where the words reach outside the matrix.
template <class T>
__device__ __forceinline__ Pack8<T> load8_any(const Matrix<const T>& m, int64_t row, int c,
                                              int d) {
  static_assert(sizeof(T) == 2, "16-bit values");
  const int64_t at = row * m.ld + c;
  const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(m.p + at) & 15u);
  const int64_t first = at - shift / 2;
  Pack8<T> o;
  if (first >= 0 && first + 16 <= m.extent) {
    const uint4* p = reinterpret_cast<const uint4*>(m.p + first);
    o.u = shifted(p[0], p[1], shift);
    if (c + 8 > d) {
      uint32_t w[4] = {o.u.x, o.u.y, o.u.z, o.u.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int keep = d - c - 2 * i;  // values of this word
        if (keep < 2) w[i] = keep <= 0 ? 0u : w[i] & 0xffffu;
      }
      o.u = make_uint4(w[0], w[1], w[2], w[3]);
    }
  } else {
    const int count = min(8, d - c);
    o.u = count > 0 && m.ok(at, count) ? load8_single(m.p + at, count)
                                       : make_uint4(0u, 0u, 0u, 0u);
  }
  return o;
}

// A thread's E values of a row that `threads` threads share: eight
// consecutive ones per step (VEC) or one, threads side by side.
template <int E, bool VEC>
struct Slots {
  static constexpr int STEP = VEC ? 8 : 1;
  static constexpr int COUNT = E / STEP;
  static __device__ __forceinline__ int col(int i, int tid, int threads) {
    return (i * threads + tid) * STEP;
  }
};

// What a thread holds of a row of a matrix, unconverted.
template <class T, int E, bool VEC>
struct Held {
  using S = Slots<E, VEC>;
  using Item = typename std::conditional<VEC, Pack8<T>, T>::type;
  Item item[S::COUNT];

  __device__ __forceinline__ void load(const Matrix<const T>& m, int64_t row, int d, int tid,
                                       int threads) {
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) {
      const int c = S::col(i, tid, threads);
      const int64_t at = row * m.ld + c;
      if (c < d && m.ok(at, S::STEP)) item[i] = *reinterpret_cast<const Item*>(m.p + at);
      else item[i] = Item{};
    }
  }
  __device__ __forceinline__ void fill(float value) {
    float v[S::STEP];
#pragma unroll
    for (int k = 0; k < S::STEP; ++k) v[k] = value;
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) {
      if constexpr (VEC) item[i].set(v);
      else item[i] = from_f32<T>(value);
    }
  }
  // The values of step i, in order.
  __device__ __forceinline__ void get(int i, float (&v)[S::STEP]) const {
    if constexpr (VEC) item[i].get(v);
    else v[0] = to_f32(item[i]);
  }
};

template <class T, bool VEC>
__device__ __forceinline__ void store_step(const Matrix<T>& m, int64_t row, int c,
                                           const float (&v)[VEC ? 8 : 1]) {
  const int64_t at = row * m.ld + c;
  if (!m.ok(at, VEC ? 8 : 1)) return;
  if constexpr (VEC) {
    Pack8<T> o;
    o.set(v);
    *reinterpret_cast<Pack8<T>*>(m.p + at) = o;
  } else {
    m.p[at] = from_f32<T>(v[0]);
  }
}

// Whether every eighth column of every row is aligned for Pack8.
inline bool rows_aligned(const void* p, int64_t ld, int elem) {
  const int unit = elem == 1 ? 8 : 16;
  return reinterpret_cast<uintptr_t>(p) % unit == 0 && ld * elem % unit == 0;
}

// Calls f(threads per row, values per thread) with the smallest row layout
// that holds d values, at most MOST values a thread where threads allow;
// false when d is past the widest.
template <int MOST, class F>
bool row_layout(int d, F&& f) {
  using std::integral_constant;
  auto go = [&](auto threads, auto values) { f(threads, values); return true; };
  if (d <= 256) return go(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (d <= 64 * MOST) return go(integral_constant<int, 64>{}, integral_constant<int, MOST>{});
  if (d <= 128 * MOST) return go(integral_constant<int, 128>{}, integral_constant<int, MOST>{});
  if (d <= 256 * MOST) return go(integral_constant<int, 256>{}, integral_constant<int, MOST>{});
  if (d <= 512 * MOST) return go(integral_constant<int, 512>{}, integral_constant<int, MOST>{});
  if (d <= 1024 * MOST) return go(integral_constant<int, 1024>{}, integral_constant<int, MOST>{});
  if (d <= 16384) return go(integral_constant<int, 1024>{}, integral_constant<int, 16>{});
  return false;
}

// Rows a CTA works on at a time: one, or one per warp when a warp holds a
// row.
constexpr int rows_per_cta(int threads) { return threads == 32 ? 4 : 1; }

}  // namespace row
}  // namespace mt
