// Internal interface between the host side of the feed-forward operators
// (layers_api.cu) and their kernels.  Not part of the C ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "kernels.h"

namespace mt {

// Storage types, as mt_dtype.
enum DType { DT_F16 = 1, DT_BF16 = 2, DT_F32 = 3, DT_E4M3 = 4 };

inline int dtype_bytes(int t) { return t == DT_F32 ? 4 : t == DT_E4M3 ? 1 : 2; }

// rms_norm.cu.  See mt_rms_norm_args for the operator.
struct RmsNormArgs {
  int64_t rows;
  int d;
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  void* h;
  int64_t ldh;
  void* y;
  int64_t ldy;
  float* scale;
  float* rstd;
  float eps;
  int dtype;
  int e4m3;        // y in 8 bits with scales
  int weight_f32;  // weight in fp32, else in dtype
  BoundsRecord* bounds;
};

cudaError_t launch_rms_norm(const RmsNormArgs& a, int sms, cudaStream_t stream);

}  // namespace mt
