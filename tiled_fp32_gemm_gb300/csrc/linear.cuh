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

// The activations, in fp32.  (1 + tanh u) / 2 is the logistic function of 2u.
template <int ACT>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z < 0.0f ? 0.0f : z;  // a NaN stays one
  } else if constexpr (ACT == ACT_GELU) {
    return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
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
                0.5f * (1.0f + erff(z * 0.70710678118654752f)));
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

// Column c, rows t0 .. of a T x C matrix with row pitch ld: `rows` of them
// (at most FINISH_ROWS) added to v, or v rounded and stored to them.
template <class T>
__device__ __forceinline__ void add_rows(const LinearEpilogue& e, const void* m, int64_t ld,
                                         int c, int t0, int rows, Rows& v) {
  const T* base = static_cast<const T*>(m);
  const T* p = base + static_cast<int64_t>(t0) * ld + c;
#pragma unroll
  for (int i = 0; i < FINISH_ROWS; ++i, p += ld)
    if (i < rows && bounds_ok(e.bounds, SITE_C_STORE, p - base, 1, view_extent(e.T, e.C, ld)))
      v[i] += row::to_f32(*p);
}
template <class T>
__device__ __forceinline__ void store_rows(const LinearEpilogue& e, void* m, int64_t ld, int c,
                                           int t0, int rows, const Rows& v) {
  T* base = static_cast<T*>(m);
  T* p = base + static_cast<int64_t>(t0) * ld + c;
#pragma unroll
  for (int i = 0; i < FINISH_ROWS; ++i, p += ld)
    if (i < rows && bounds_ok(e.bounds, SITE_C_STORE, p - base, 1, view_extent(e.T, e.C, ld)))
      *p = row::from_f32<T>(v[i]);
}
__device__ __forceinline__ void store_rows(const LinearEpilogue& e, void* m, int64_t ld, int c,
                                           int t0, int rows, const Rows& v) {
  if (e.out_dtype == DT_F16) store_rows<__half>(e, m, ld, c, t0, rows, v);
  else if (e.out_dtype == DT_BF16) store_rows<__nv_bfloat16>(e, m, ld, c, t0, rows, v);
  else store_rows<float>(e, m, ld, c, t0, rows, v);
}

// Finishes the sums v of column c of Y, rows t0 .. (those at or past t_end <=
// e.T, and columns at or past e.C, are dropped).  The residual may be Y
// itself: each element is read and then written by this thread.
__device__ __forceinline__ void finish(const LinearEpilogue& e, int c, int t0, int t_end,
                                       Rows& v) {
  const int rows = t_end - t0;
  if (c >= e.C || rows <= 0) return;
  const float b = e.bias && bounds_ok(e.bounds, SITE_BIAS, c, 1, e.C) ? e.bias[c] : 0.0f;
  if (e.row_scale) {
    const float s = e.col_scale[c];
#pragma unroll
    for (int i = 0; i < FINISH_ROWS; ++i)
      v[i] = fmaf(v[i], (i < rows ? e.row_scale[t0 + i] : 0.0f) * s, b);
  } else if (e.bias) {
#pragma unroll
    for (int i = 0; i < FINISH_ROWS; ++i) v[i] += b;
  }
  if (e.Z) store_rows(e, e.Z, e.ldz, c, t0, rows, v);
  switch (e.act) {
    case ACT_RELU: activate_rows<ACT_RELU>(v); break;
    case ACT_GELU: activate_rows<ACT_GELU>(v); break;
    case ACT_GELU_TANH: activate_rows<ACT_GELU_TANH>(v); break;
    case ACT_SILU: activate_rows<ACT_SILU>(v); break;
    default: break;
  }
  if (e.residual) {
    if (e.out_dtype == DT_F16) add_rows<__half>(e, e.residual, e.ldr, c, t0, rows, v);
    else if (e.out_dtype == DT_BF16)
      add_rows<__nv_bfloat16>(e, e.residual, e.ldr, c, t0, rows, v);
    else add_rows<float>(e, e.residual, e.ldr, c, t0, rows, v);
  }
  store_rows(e, e.Y, e.ldy, c, t0, rows, v);
}

// A built kernel (kernel null: no such form), its dynamic shared memory and
// pipeline stages.
struct LinearKernel {
  const void* kernel = nullptr;
  int smem = 0, stages = 0;
};

constexpr int LINEAR_BC = 128;  // columns of Y per tile of the split kernels

}  // namespace linear

linear::LinearKernel linear_split_kernel_for(int dtype, int bt, bool w_mn, bool x_mn);
cudaError_t linear_split_read_and_clear_status(unsigned int* status);
linear::LinearKernel linear_pair_kernel_for(int dtype, bool w_mn, bool x_mn);
cudaError_t launch_linear_pair(const linear::LinearKernel& k, const CUtensorMap& map_w,
                               const CUtensorMap& map_x, uint32_t idesc,
                               const linear::LinearEpilogue& ep, int kt, int clusters,
                               int fault_inject, cudaStream_t stream);
cudaError_t linear_pair_read_and_clear_status(unsigned int* status);

}  // namespace mt
