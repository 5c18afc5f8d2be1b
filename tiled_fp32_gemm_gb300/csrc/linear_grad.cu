// The elementwise part of the linear layer's gradient: dz = dY * act'(Z) and
// its column sums (the bias gradient) in one pass over dY and Z.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "linear.cuh"
#include "row_util.cuh"

namespace mt {
namespace {

using namespace linear;
using namespace row;

constexpr int kWarps = 8;

// A CTA takes 32 columns of a block of rows, its warps every eighth row.
template <class T, int ACT>
__global__ void __launch_bounds__(32 * kWarps) linear_dz_kernel(const LinearDzArgs a,
                                                                int64_t rows_per_block,
                                                                float* partial) {
  __shared__ float sums[kWarps][32];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  const int64_t first = blockIdx.y * rows_per_block;
  const int64_t last = min(a.M, first + rows_per_block);
  float s = 0.0f;
  if (c < a.N)
    for (int64_t i = first + warp; i < last; i += kWarps) {
      float dz = to_f32(static_cast<const T*>(a.dY)[i * a.lddy + c]);
      if (ACT != ACT_NONE)  // never fused into the sum: the same bits with and without dZ
        dz = __fmul_rn(
            dz, activate_grad<ACT>(to_f32(static_cast<const T*>(a.Z)[i * a.ldz + c])));
      if (a.dZ) static_cast<T*>(a.dZ)[i * a.lddz + c] = from_f32<T>(dz);
      s += dz;
    }
  if (!a.dbias) return;
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.N) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) s += sums[w][lane];
    partial[static_cast<int64_t>(blockIdx.y) * a.N + c] = s;
  }
}

int row_blocks(const LinearDzArgs& a, int sms) {
  const int64_t strips = (a.N + 31) / 32;
  const int64_t want = std::max<int64_t>(1, 32 * static_cast<int64_t>(sms) / strips);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (a.M + 31) / 32)));
}

template <class T, int ACT>
cudaError_t launch(const LinearDzArgs& a, float* partial, int sms, cudaStream_t stream) {
  const int blocks = row_blocks(a, sms);
  const int64_t per = (a.M + blocks - 1) / blocks;
  const cudaError_t e = launch_dependent(linear_dz_kernel<T, ACT>,
                                         dim3((a.N + 31) / 32, blocks), 32 * kWarps, stream, a,
                                         per, partial);
  if (e != cudaSuccess || !a.dbias) return e;
  return launch_add_rows(partial, blocks, a.N, a.dbias, a.bounds, stream);
}

template <class T>
cudaError_t launch_act(const LinearDzArgs& a, float* partial, int sms, cudaStream_t stream) {
  switch (a.act) {
    case ACT_RELU: return launch<T, ACT_RELU>(a, partial, sms, stream);
    case ACT_GELU: return launch<T, ACT_GELU>(a, partial, sms, stream);
    case ACT_GELU_TANH: return launch<T, ACT_GELU_TANH>(a, partial, sms, stream);
    case ACT_SILU: return launch<T, ACT_SILU>(a, partial, sms, stream);
    default: return launch<T, ACT_NONE>(a, partial, sms, stream);
  }
}

}  // namespace

int64_t linear_dz_workspace(const LinearDzArgs& a, int sms) {
  return a.dbias ? static_cast<int64_t>(row_blocks(a, sms)) * a.N * 4 : 0;
}

cudaError_t launch_linear_dz(const LinearDzArgs& a, void* partial, int sms,
                             cudaStream_t stream) {
  float* p = static_cast<float*>(partial);
  return a.dtype == DT_F16 ? launch_act<__half>(a, p, sms, stream)
                           : launch_act<__nv_bfloat16>(a, p, sms, stream);
}

}  // namespace mt
