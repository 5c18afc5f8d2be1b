// Gradient of the root-mean-square norm: with xhat = h * rstd, g = dy * weight,
//   dx = rstd * (g - xhat * mean(g * xhat)) + dh,   dweight = sum over rows of dy * xhat.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "row_util.cuh"

namespace mt {
namespace {

using namespace row;

constexpr int kWideThreads = 512;

template <class T>
__device__ __forceinline__ float weight_at(const RmsNormGradArgs& a, int c) {
  return !a.weight ? 1.0f
         : a.weight_f32 ? static_cast<const float*>(a.weight)[c]
                        : to_f32(static_cast<const T*>(a.weight)[c]);
}

// dx of a row of any width on one CTA: one sweep for the mean, one for dx,
// each element read and then written by the same thread (dx may be dy or dh).
template <class T>
__global__ void __launch_bounds__(kWideThreads) rms_norm_grad_wide_kernel(
    const RmsNormGradArgs a) {
  __shared__ float part[kWideThreads / 32];
  const int64_t row = blockIdx.x;
  const T* dy = static_cast<const T*>(a.dy) + row * a.lddy;
  const T* h = static_cast<const T*>(a.h) + row * a.ldh;
  const T* dh = a.dh ? static_cast<const T*>(a.dh) + row * a.lddh : nullptr;
  const float r = a.rstd[row];
  float dot = 0.0f;
  for (int c = threadIdx.x; c < a.d; c += kWideThreads)
    dot = fmaf(to_f32(dy[c]) * weight_at<T>(a, c), to_f32(h[c]) * r, dot);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  dot = warp_sum(dot);
  if (lane == 0) part[warp] = dot;
  __syncthreads();
  dot = warp_sum(lane < kWideThreads / 32 ? part[lane] : 0.0f);
  const float mean = dot / static_cast<float>(a.d);
  for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
    const float g = to_f32(dy[c]) * weight_at<T>(a, c);
    const float dx = r * (g - to_f32(h[c]) * r * mean) + (dh ? to_f32(dh[c]) : 0.0f);
    static_cast<T*>(a.dx)[row * a.lddx + c] = from_f32<T>(dx);
  }
}

// dweight, first step: column sums of dy * xhat over one block of rows.  A
// CTA takes 32 columns, its 8 warps every eighth row of the block.
constexpr int kColumnWarps = 8;

template <class T>
__global__ void __launch_bounds__(32 * kColumnWarps) rms_norm_grad_columns_kernel(
    const RmsNormGradArgs a, int64_t rows_per_block, float* partial) {
  __shared__ float sums[kColumnWarps][32];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  const int64_t first = blockIdx.y * rows_per_block;
  const int64_t last = min(a.rows, first + rows_per_block);
  float s = 0.0f;
  if (c < a.d)
    for (int64_t i = first + warp; i < last; i += kColumnWarps)
      s = fmaf(to_f32(static_cast<const T*>(a.dy)[i * a.lddy + c]),
               to_f32(static_cast<const T*>(a.h)[i * a.ldh + c]) * a.rstd[i], s);
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kColumnWarps; ++w) s += sums[w][lane];
    partial[static_cast<int64_t>(blockIdx.y) * a.d + c] = s;
  }
}

// Adds the partial rows: a CTA takes 32 columns, its 32 warps every 32nd row.
__global__ void __launch_bounds__(1024) add_rows_kernel(const float* rows, int count, int cols,
                                                        float* out) {
  __shared__ float sums[32][33];
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int i = warp; i < count; i += 32) s += rows[static_cast<int64_t>(i) * cols + c];
  sums[warp][lane] = s;
  __syncthreads();
  // Warp w adds the 32 sums of column w.
  s = warp_sum(sums[lane][warp]);
  const int cw = blockIdx.x * 32 + warp;
  if (lane == 0 && cw < cols) out[cw] = s;
}

// Blocks of rows of the column sums: enough CTAs for four waves of eight on
// each SM, at least 32 rows each.
int column_blocks(int64_t rows, int cols, int sms) {
  const int64_t strips = (cols + 31) / 32;
  const int64_t want = std::max<int64_t>(1, 32 * static_cast<int64_t>(sms) / strips);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (rows + 31) / 32)));
}

template <class T>
cudaError_t launch(const RmsNormGradArgs& a, float* partial, int sms, cudaStream_t stream) {
  // The column sums come first: dx may overwrite dy.
  if (a.dweight) {
    const int blocks = column_blocks(a.rows, a.d, sms);
    const int64_t per = (a.rows + blocks - 1) / blocks;
    rms_norm_grad_columns_kernel<T>
        <<<dim3((a.d + 31) / 32, blocks), 32 * kColumnWarps, 0, stream>>>(a, per, partial);
    const cudaError_t e = launch_add_rows(partial, blocks, a.d, a.dweight, stream);
    if (e != cudaSuccess) return e;
  }
  if (a.rows > 0)
    rms_norm_grad_wide_kernel<T>
        <<<static_cast<unsigned>(a.rows), kWideThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_add_rows(const float* rows, int count, int cols, float* out,
                            cudaStream_t stream) {
  add_rows_kernel<<<(cols + 31) / 32, 1024, 0, stream>>>(rows, count, cols, out);
  return cudaGetLastError();
}

int64_t rms_norm_grad_workspace(const RmsNormGradArgs& a, int sms) {
  if (!a.dweight) return 0;
  return static_cast<int64_t>(column_blocks(a.rows, a.d, sms)) * a.d * 4;
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, void* workspace, int sms,
                                 cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  switch (a.dtype) {
    case DT_F16: return launch<__half>(a, partial, sms, stream);
    case DT_BF16: return launch<__nv_bfloat16>(a, partial, sms, stream);
    default: return launch<float>(a, partial, sms, stream);
  }
}

}  // namespace mt
