// Epilogue of the fused linear layer, shared by its kernels: scale, bias,
// activation, residual, one rounding.
#pragma once

#include <cstdint>

#include <cuda.h>

#include "device_util.cuh"
#include "layers.h"
#include "row_util.cuh"

namespace mt {
namespace linear {

// 1 / (1 + exp(-z)).  exp overflows to infinity for z below -88, which gives
// the 0 that is wanted.
__device__ __forceinline__ float logistic(float z) {
  return __fdividef(1.0f, 1.0f + __expf(-z));
}

// The normal distribution's Phi(z) = (1 + erf(z / sqrt 2)) / 2 by Hastings'
// approximation of erf (Abramowitz and Stegun, Handbook of Mathematical
// Functions, 7.1.26: five coefficients, one exponential, absolute error below
// 1.5e-7), without the branches of a correctly scaled erf: every lane of a
// warp takes the same path.
__device__ __forceinline__ float normal_cdf(float z) {
  const float x = fabsf(z) * 0.70710678118654752f;
  const float t = __fdividef(1.0f, fmaf(0.3275911f, x, 1.0f));
  float p = fmaf(1.061405429f, t, -1.453152027f);
  p = fmaf(p, t, 1.421413741f);
  p = fmaf(p, t, -0.284496736f);
  p = fmaf(p, t, 0.254829592f);
  const float tail = 0.5f * p * t * __expf(-x * x);  // Phi(-|z|)
  return z > 0.0f ? 1.0f - tail : tail;
}

// The activations, in fp32.  (1 + tanh u) / 2 is the logistic function of 2u.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z < 0.0f ? 0.0f : z;  // a NaN stays one
  } else if constexpr (ACT == ACT_GELU) {
    return z * normal_cdf(z);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    return z * logistic(1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
  } else if constexpr (ACT == ACT_SILU) {
    return z * logistic(z);
  } else {
    return z;
  }
}

// Their derivatives.  Past the clamps the logistic forms' derivatives are 0
// or 1 to fp32; the clamps keep 0 * infinity out of them (a NaN passes).
template <int ACT>
__device__ __forceinline__ float activate_grad(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  } else if constexpr (ACT == ACT_GELU) {
    // Phi(z) + z * phi(z)
    return fmaf(z * 0.39894228040143268f, __expf(-0.5f * z * z),
                normal_cdf(z));
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float x = z > 30.0f ? 30.0f : z < -30.0f ? -30.0f : z;
    const float p = logistic(1.5957691216057308f * fmaf(0.044715f * x * x, x, x));
    return fmaf(p * (1.0f - p) * x, 1.5957691216057308f * fmaf(0.134145f * x, x, 1.0f), p);
  } else if constexpr (ACT == ACT_SILU) {
    const float x = z > 100.0f ? 100.0f : z < -100.0f ? -100.0f : z;
    const float p = logistic(x);
    return p * fmaf(x, 1.0f - p, 1.0f);
  } else {
    return 1.0f;
  }
}

struct LinearEpilogue {
  void* Y;
  int64_t ldy;
  void* Z;
  int64_t ldz;
  const void* residual;
  int64_t ldr;
  const float* bias;
  const float* row_scale;
  const float* col_scale;
  int T, C;
  int out_dtype, act;
  BoundsRecord* bounds;
};

// Rows of one column a thread finishes at a time.
constexpr int FINISH_ROWS = 16;
using Rows = float[FINISH_ROWS];

template <int ACT>
__device__ __forceinline__ void activate_rows(Rows& v) {
#pragma unroll
  for (int i = 0; i < FINISH_ROWS; ++i) v[i] = activate<ACT>(v[i]);
}

// What finishing FINISH_ROWS rows of a column reads besides the sums: the
// residual's bits, and lane i's share of the rows' scales.
struct Ahead {
  uint32_t residual[FINISH_ROWS];
  float row_scale;

  __device__ __forceinline__ void load(const LinearEpilogue& e, int c, int t, int t_end) {
    const int rows = c < e.C ? t_end - t : 0;
    if (e.residual) {
      const int64_t extent = view_extent(e.T, e.C, e.ldr);
      int64_t at = static_cast<int64_t>(t) * e.ldr + c;
      if (e.out_dtype == DT_F32) {
#pragma unroll
        for (int i = 0; i < FINISH_ROWS; ++i, at += e.ldr)
          residual[i] = i < rows && bounds_ok(e.bounds, SITE_C_STORE, at, 1, extent)
                            ? static_cast<const uint32_t*>(e.residual)[at]
                            : 0u;
      } else {
#pragma unroll
        for (int i = 0; i < FINISH_ROWS; ++i, at += e.ldr)
          residual[i] = i < rows && bounds_ok(e.bounds, SITE_C_STORE, at, 1, extent)
                            ? static_cast<const uint16_t*>(e.residual)[at]
                            : 0u;
      }
    }
    if (e.row_scale) {
      const int lane = threadIdx.x % 32;
      row_scale = lane < FINISH_ROWS && t + lane < t_end &&
                          bounds_ok(e.bounds, SITE_BIAS, t + lane, 1, e.T)
                      ? e.row_scale[t + lane]
                      : 0.0f;
    }
  }
};

// Column c, rows t .. of a T x C matrix with row pitch ld: v rounded and
// stored to `rows` of them.
template <class T>
__device__ __forceinline__ void store_rows(const LinearEpilogue& e, void* m, int64_t ld, int c,
                                           int t, int rows, const Rows& v) {
  T* base = static_cast<T*>(m);
  T* p = base + static_cast<int64_t>(t) * ld + c;
#pragma unroll
  for (int i = 0; i < FINISH_ROWS; ++i, p += ld)
    if (i < rows && bounds_ok(e.bounds, SITE_C_STORE, p - base, 1, view_extent(e.T, e.C, ld)))
      *p = row::from_f32<T>(v[i]);
}
__device__ __forceinline__ void store_rows(const LinearEpilogue& e, void* m, int64_t ld, int c,
                                           int t, int rows, const Rows& v) {
  if (e.out_dtype == DT_F16) store_rows<__half>(e, m, ld, c, t, rows, v);
  else if (e.out_dtype == DT_BF16) store_rows<__nv_bfloat16>(e, m, ld, c, t, rows, v);
  else store_rows<float>(e, m, ld, c, t, rows, v);
}

// Finishes column c of Y, rows t_begin .. t_end - 1 (t_end <= e.T; columns at
// or past e.C are dropped), the whole warp together: sums(t, v) gives the
// sums of rows t .. t + FINISH_ROWS - 1.  What the next rows need is read
// while these are computed.  The residual may be Y itself: each element is
// read and then written by this thread.
template <class Sums>
__device__ __forceinline__ void finish(const LinearEpilogue& e, int c, int t_begin, int t_end,
                                       Sums&& sums) {
  const bool live = c < e.C;
  const float b =
      e.bias && live && bounds_ok(e.bounds, SITE_BIAS, c, 1, e.C) ? e.bias[c] : 0.0f;
  const float s =
      e.col_scale && live && bounds_ok(e.bounds, SITE_BIAS, c, 1, e.C) ? e.col_scale[c] : 0.0f;
  Ahead next;
  next.load(e, c, t_begin, t_end);
#pragma unroll 1
  for (int t = t_begin; t < t_end; t += FINISH_ROWS) {
    const Ahead now = next;
    if (t + FINISH_ROWS < t_end) next.load(e, c, t + FINISH_ROWS, t_end);
    Rows v;
    sums(t, v);
    const int rows = live ? t_end - t : 0;
    if (e.row_scale) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i)
        v[i] = fmaf(v[i], __shfl_sync(0xffffffffu, now.row_scale, i) * s, b);
    } else {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) v[i] += b;
    }
    if (e.Z) store_rows(e, e.Z, e.ldz, c, t, rows, v);
    switch (e.act) {
      case ACT_RELU: activate_rows<ACT_RELU>(v); break;
      case ACT_GELU: activate_rows<ACT_GELU>(v); break;
      case ACT_GELU_TANH: activate_rows<ACT_GELU_TANH>(v); break;
      case ACT_SILU: activate_rows<ACT_SILU>(v); break;
      default: break;
    }
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) {
        const uint32_t r = now.residual[i];
        v[i] += e.out_dtype == DT_BF16  ? __uint_as_float(r << 16)
                : e.out_dtype == DT_F16 ? __half2float(__ushort_as_half(
                                              static_cast<unsigned short>(r)))
                                        : __uint_as_float(r);
      }
    }
    store_rows(e, e.Y, e.ldy, c, t, rows, v);
  }
}

// A built kernel (kernel null: no such form), its dynamic shared memory and
// pipeline stages.
struct LinearKernel {
  const void* kernel = nullptr;
  int smem = 0, stages = 0;
};

constexpr int LINEAR_BC = 128;  // columns of Y per tile of the split kernels

// One product of a split-kernel launch: its CTAs are first_cta and on.
struct SplitProblem {
  CUtensorMap map_w, map_x;
  LinearEpilogue ep;
  uint32_t idesc;
  int ktiles, tiles_t, first_cta;
  int w_mn, x_mn;
};
struct SplitProblems {
  SplitProblem p[2];
};

}  // namespace linear

linear::LinearKernel linear_split_kernel_for(int dtype, int bt);
cudaError_t linear_split_read_and_clear_status(unsigned int* status);
linear::LinearKernel linear_pair_kernel_for(int dtype, bool w_mn, bool x_mn);
cudaError_t launch_linear_pair(const linear::LinearKernel& k, const CUtensorMap& map_w,
                               const CUtensorMap& map_x, uint32_t idesc,
                               const linear::LinearEpilogue& ep, int kt, int clusters,
                               int fault_inject, cudaStream_t stream);
cudaError_t linear_pair_read_and_clear_status(unsigned int* status);

}  // namespace mt
