// Epilogue of the fused linear layer, shared by its kernels: scale, bias,
// activation, residual, one rounding.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "device_util.cuh"
#include "layers.h"
#include "row_util.cuh"

namespace mt {
namespace linear {

// exp(x) and 1 / x on the special-function unit, one instruction past the
// scaling by log2(e) (the .ftz forms: what would be subnormal is 0).
__device__ __forceinline__ float exp_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The functions below have two forms.  F32 false, for 16-bit results and the
// derivatives: the special-function unit's exponential, whose argument's
// rounding costs up to 2^-15 of a result far out in a tail, an eighth of half
// a step of fp16.  F32 true, for fp32 results: CUDA's expf and arguments that
// keep their digits: 4096^3 with fp32 results, gelu and residual takes 103 us
// so, 98 with the F32 false form, 115 with normcdff.

// 1 / (1 + exp(-z)).
template <bool F32>
__device__ __forceinline__ float logistic(float z) {
  if constexpr (F32) {
    const float e = expf(-fabsf(z));  // never overflows
    return (z < 0.0f ? e : 1.0f) * rcp_approx(1.0f + e);
  } else {
    // exp overflows to infinity for z below -88, which gives the 0 that is
    // wanted.
    return rcp_approx(1.0f + exp_approx(-z));
  }
}

// The normal distribution's Phi(z) and *bell = exp(-z^2 / 2).  With x = |z| /
// sqrt 2, Phi(-|z|) is bell * erfcx(x) / 2, erfcx(x) = exp(x^2) erfc(x).  That
// falls from 1 to 1 / (x sqrt pi) without ever being small, so a polynomial in
// t = 1 / (1 + 0.43 x) without constant term holds it to a *relative* error,
// which is what keeps the tail's digits: these eight coefficients are a
// minimax fit (Lawson's reweighted least squares) over 0 <= x <= 10, within
// 1.0e-7, 4.5e-7 as evaluated here.  No branches: every lane of a warp takes
// the same path.
template <bool F32>
__device__ __forceinline__ float normal_cdf(float z, float* bell) {
  // Past 15 the tail is 0 in fp32; the clamp keeps infinity out of z^2.
  const float y = F32 ? fminf(fabsf(z), 15.0f) : fabsf(z);
  const float x = y * 0.70710678118654752f;
  const float t = rcp_approx(fmaf(0.43f, x, 1.0f));
  float p = fmaf(0.0731455436f, t, -0.308094499f);
  p = fmaf(p, t, 0.379885357f);
  p = fmaf(p, t, -0.0823025803f);
  p = fmaf(p, t, 0.245079788f);
  p = fmaf(p, t, 0.205472764f);
  p = fmaf(p, t, 0.244293791f);
  p = fmaf(p, t, 0.242519823f);
  if constexpr (F32) {
    // exp(-(s + d) / 2) with s + d = y^2, d what s lost in rounding.
    const float s = y * y, d = fmaf(y, y, -s);
    *bell = expf(-0.5f * s);
    *bell = fmaf(-0.5f * d, *bell, *bell);
  } else {
    *bell = exp_approx(-x * x);
  }
  const float tail = 0.5f * p * t * *bell;  // Phi(-|z|)
  return z > 0.0f ? 1.0f - tail : tail;
}

// The activations, in fp32.  (1 + tanh u) / 2 is the logistic function of 2u.
template <int ACT, bool F32>
__device__ __forceinline__ float activate(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z < 0.0f ? 0.0f : z;  // a NaN stays one
  } else if constexpr (ACT == ACT_GELU) {
    float bell;
    return z * normal_cdf<F32>(z, &bell);
  } else if constexpr (ACT == ACT_GELU_TANH) {
    return z * logistic<F32>(1.5957691216057308f * fmaf(0.044715f * z * z, z, z));
  } else if constexpr (ACT == ACT_SILU) {
    return z * logistic<F32>(z);
  } else {
    return z;
  }
}

// Their derivatives.  Past the clamps they are 0 or 1 to fp32; the clamps keep
// 0 * infinity out of them (a pre-activation past its 16-bit type is stored as
// infinity; a NaN passes).
template <int ACT>
__device__ __forceinline__ float activate_grad(float z) {
  if constexpr (ACT == ACT_RELU) {
    return z > 0.0f ? 1.0f : z != z ? z : 0.0f;
  } else if constexpr (ACT == ACT_GELU) {
    float bell;
    const float x = z > 15.0f ? 15.0f : z < -15.0f ? -15.0f : z;
    const float cdf = normal_cdf<false>(x, &bell);
    return fmaf(x * 0.39894228040143268f, bell, cdf);  // Phi(z) + z * phi(z)
  } else if constexpr (ACT == ACT_GELU_TANH) {
    const float x = z > 30.0f ? 30.0f : z < -30.0f ? -30.0f : z;
    const float p = logistic<false>(1.5957691216057308f * fmaf(0.044715f * x * x, x, x));
    return fmaf(p * (1.0f - p) * x, 1.5957691216057308f * fmaf(0.134145f * x, x, 1.0f), p);
  } else if constexpr (ACT == ACT_SILU) {
    const float x = z > 100.0f ? 100.0f : z < -100.0f ? -100.0f : z;
    const float p = logistic<false>(x);
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

template <int ACT, bool F32>
__device__ __forceinline__ void activate_rows(Rows& v) {
#pragma unroll
  for (int i = 0; i < FINISH_ROWS; ++i) v[i] = activate<ACT, F32>(v[i]);
}

template <bool F32>
__device__ __forceinline__ void activate_rows(int act, Rows& v) {
  switch (act) {
    case ACT_RELU: return activate_rows<ACT_RELU, F32>(v);
    case ACT_GELU: return activate_rows<ACT_GELU, F32>(v);
    case ACT_GELU_TANH: return activate_rows<ACT_GELU_TANH, F32>(v);
    case ACT_SILU: return activate_rows<ACT_SILU, F32>(v);
    default: return;
  }
}

// One column of a T x C matrix of T values with row pitch ld.
template <class T>
struct Column {
  T* p;  // row 0
  int64_t ld, extent;
  int c;
  BoundsRecord* rec;

  __device__ __forceinline__ Column(const LinearEpilogue& e, const void* m, int64_t ld_, int c_)
      : p(static_cast<T*>(const_cast<void*>(m)) + c_), ld(ld_),
        extent(view_extent(e.T, e.C, ld_)), c(c_), rec(e.bounds) {}
  __device__ __forceinline__ bool ok(int row) const {
    return bounds_ok(rec, SITE_C_STORE, row * ld + c, 1, extent);
  }
  // FINISH_ROWS rows from t on, the first `rows` of them: a whole block
  // without a test per row.
  __device__ __forceinline__ void load(int t, int rows, T (&v)[FINISH_ROWS]) const {
    const T* q = p + t * ld;
    if (rows >= FINISH_ROWS) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i, q += ld) v[i] = ok(t + i) ? *q : T(0.0f);
    } else {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i, q += ld)
        v[i] = i < rows && ok(t + i) ? *q : T(0.0f);
    }
  }
  __device__ __forceinline__ void store(int t, int rows, const Rows& v) const {
    T* q = p + t * ld;
    if (rows >= FINISH_ROWS) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i, q += ld)
        if (ok(t + i)) *q = row::from_f32<T>(v[i]);
    } else {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i, q += ld)
        if (i < rows && ok(t + i)) *q = row::from_f32<T>(v[i]);
    }
  }
};

// finish for results of type T.  What the next rows need is read while these
// are computed; the residual may be Y itself (each element is read and then
// written by this thread).
template <class T, class Sums>
__device__ __forceinline__ void finish_typed(const LinearEpilogue& e, int c, int t_begin,
                                             int t_end, Sums&& sums) {
  const bool live = c < e.C;
  const int lane = threadIdx.x % 32;
  const float b =
      e.bias && live && bounds_ok(e.bounds, SITE_BIAS, c, 1, e.C) ? e.bias[c] : 0.0f;
  const float s =
      e.col_scale && live && bounds_ok(e.bounds, SITE_BIAS, c, 1, e.C) ? e.col_scale[c] : 0.0f;
  const Column<T> y(e, e.Y, e.ldy, c), z(e, e.Z, e.ldz, c), r(e, e.residual, e.ldr, c);
  // Lane i's share of the rows' scales.
  auto scale_of = [&](int t) {
    return lane < FINISH_ROWS && t + lane < t_end &&
                   bounds_ok(e.bounds, SITE_BIAS, t + lane, 1, e.T)
               ? e.row_scale[t + lane]
               : 0.0f;
  };
  T next_res[FINISH_ROWS];
  float next_scale = 0.0f;
  if (e.residual && live) r.load(t_begin, t_end - t_begin, next_res);
  if (e.row_scale) next_scale = scale_of(t_begin);
#pragma unroll 1
  for (int t = t_begin; t < t_end; t += FINISH_ROWS) {
    const int rows = t_end - t;
    T res[FINISH_ROWS];
    const float scale = next_scale;
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) res[i] = next_res[i];
      if (live && rows > FINISH_ROWS)
        r.load(t + FINISH_ROWS, rows - FINISH_ROWS, next_res);
    }
    if (e.row_scale && rows > FINISH_ROWS) next_scale = scale_of(t + FINISH_ROWS);
    Rows v;
    // Lanes past the last column have left the last round early, and the
    // residual's loads are theirs alone: the sums are read by the whole warp.
    __syncwarp();
    sums(t, v);
    if (e.row_scale) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i)
        v[i] = fmaf(v[i], __shfl_sync(0xffffffffu, scale, i) * s, b);
    } else if (e.bias) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) v[i] += b;
    }
    if (!live) continue;
    if (e.Z) z.store(t, rows, v);
    activate_rows<std::is_same<T, float>::value>(e.act, v);
    if (e.residual) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) v[i] += row::to_f32(res[i]);
    }
    y.store(t, rows, v);
  }
}

// Finishes column c of Y, rows t_begin .. t_end - 1 (t_end <= e.T; columns at
// or past e.C are dropped), the whole warp together: sums(t, v), called by a
// converged warp, gives the sums of rows t .. t + FINISH_ROWS - 1.
template <class Sums>
__device__ __forceinline__ void finish(const LinearEpilogue& e, int c, int t_begin, int t_end,
                                       Sums&& sums) {
  if (e.out_dtype == DT_F16) finish_typed<__half>(e, c, t_begin, t_end, sums);
  else if (e.out_dtype == DT_BF16) finish_typed<__nv_bfloat16>(e, c, t_begin, t_end, sums);
  else finish_typed<float>(e, c, t_begin, t_end, sums);
}

// A built kernel (kernel null: no such form), its dynamic shared memory and
// pipeline stages.
struct LinearKernel {
  const void* kernel = nullptr;
  int smem = 0, stages = 0;
};

constexpr int LINEAR_BC = 128;  // columns of Y per tile of the split kernels

// One product of a split-kernel launch: its CTAs are first_cta and on.  Ep:
// what finish() does with its sums.
template <class Ep>
struct SplitProblemOf {
  CUtensorMap map_w, map_x;
  Ep ep;
  uint32_t idesc;
  int ktiles, tiles, tiles_t, first_cta;
  int split;  // CTAs that share a tile: the launch's cluster, or 1
  int w_mn, x_mn;
};
template <class Ep>
struct SplitProblemsOf {
  SplitProblemOf<Ep> p[2];
};
using SplitProblem = SplitProblemOf<LinearEpilogue>;
using SplitProblems = SplitProblemsOf<LinearEpilogue>;

}  // namespace linear

linear::LinearKernel linear_split_kernel_for(int dtype, int bt);
cudaError_t linear_split_read_and_clear_status(unsigned int* status);
linear::LinearKernel linear_pair_kernel_for(int dtype, bool w_mn, bool x_mn);
cudaError_t launch_linear_pair(const linear::LinearKernel& k, const CUtensorMap& map_w,
                               const CUtensorMap& map_x, uint32_t idesc,
                               const linear::LinearEpilogue& ep, int kt, int clusters,
                               int fault_inject, cudaStream_t stream);
cudaError_t linear_pair_read_and_clear_status(unsigned int* status);
// linear_rows.cu: plain products whose Y TMA writes, on pairs.
cudaError_t linear_rows_prepare();
cudaError_t launch_linear_rows(const LinearArgs& a, const CUtensorMap& map_x,
                               const CUtensorMap& map_w, const CUtensorMap& map_y,
                               uint32_t idesc, int kt, const PlanesPlan* planes, bool add,
                               int clusters, cudaStream_t stream);
cudaError_t linear_rows_read_and_clear_status(unsigned int* status);

}  // namespace mt
