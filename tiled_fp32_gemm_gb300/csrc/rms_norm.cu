// Root-mean-square norm with the residual's addition, 16- or 32-bit output
// or e4m3 output with one scale per row.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h * r * weight
//   e4m3:  scale = max(max|y| / 448, 2^-126),  q = e4m3(y / scale)
//
// max|y| = r * max|h * weight| (r is one positive factor of the row), so the
// sum of squares and the maximum come from one sweep and one reduction.
#include <cfloat>
#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "row_util.cuh"

namespace mt {
namespace {

using namespace row;

constexpr int kWideThreads = 512;

// A row of any width on one CTA: one sweep for the statistics, one for the
// outputs, which reads x and the residual again (from L2: a row of 2^20
// fp32 elements is 4 MB).  Each element is read and then written by the same
// thread, in the second sweep only, so h may be x or residual.
template <class T, bool E4M3>
__global__ void __launch_bounds__(kWideThreads) rms_norm_wide_kernel(const RmsNormArgs a) {
  __shared__ float part_sum[kWideThreads / 32], part_max[kWideThreads / 32];
  const int64_t row = blockIdx.x;
  const T* x = static_cast<const T*>(a.x) + row * a.ldx;
  const T* res = a.residual ? static_cast<const T*>(a.residual) + row * a.ldr : nullptr;
  auto weight = [&](int c) {
    return !a.weight ? 1.0f
           : a.weight_f32 ? static_cast<const float*>(a.weight)[c]
                          : to_f32(static_cast<const T*>(a.weight)[c]);
  };
  auto load = [&](int c) { return to_f32(x[c]) + (res ? to_f32(res[c]) : 0.0f); };
  float sum = 0.0f, top = 0.0f;
  for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
    const float h = load(c);
    sum = fmaf(h, h, sum);
    if (E4M3) top = fmaxf(top, fabsf(h * weight(c)));
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  sum = warp_sum(sum);
  if (E4M3) top = warp_max(top);
  if (lane == 0) {
    part_sum[warp] = sum;
    part_max[warp] = top;
  }
  __syncthreads();
  sum = warp_sum(lane < kWideThreads / 32 ? part_sum[lane] : 0.0f);
  if (E4M3) top = warp_max(lane < kWideThreads / 32 ? part_max[lane] : 0.0f);
  const float r = rsqrtf((a.d > 0 ? sum / static_cast<float>(a.d) : 0.0f) + a.eps);
  float inv = 0.0f;
  if (E4M3) {
    const float t = top * r / 448.0f;
    const float scale = t < FLT_MIN ? FLT_MIN : t;  // a NaN stays one
    inv = 1.0f / scale;
    if (threadIdx.x == 0) a.scale[row] = scale;
  }
  if (threadIdx.x == 0 && a.rstd) a.rstd[row] = r;
  for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
    const float h = load(c);
    const float y = h * r * weight(c);
    if (a.h) static_cast<T*>(a.h)[row * a.ldh + c] = from_f32<T>(h);
    if (E4M3)
      static_cast<uint8_t*>(a.y)[row * a.ldy + c] = static_cast<uint8_t>(e4m3x2(y * inv, 0.0f));
    else
      static_cast<T*>(a.y)[row * a.ldy + c] = from_f32<T>(y);
  }
}

template <class T, bool E4M3>
cudaError_t launch(const RmsNormArgs& a, cudaStream_t stream) {
  rms_norm_wide_kernel<T, E4M3>
      <<<static_cast<unsigned>(a.rows), kWideThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

template <class T>
cudaError_t launch_out(const RmsNormArgs& a, cudaStream_t stream) {
  return a.e4m3 ? launch<T, true>(a, stream) : launch<T, false>(a, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs& a, int sms, cudaStream_t stream) {
  (void)sms;
  switch (a.dtype) {
    case DT_F16: return launch_out<__half>(a, stream);
    case DT_BF16: return launch_out<__nv_bfloat16>(a, stream);
    default: return launch_out<float>(a, stream);
  }
}

}  // namespace mt
