// The elementwise part of the linear layer's gradient: dz = dY * act'(Z) and
// its column sums (the bias gradient) in one pass over dY and Z.  Bound by
// memory: dY and Z are read once and dz is written once.
//
// A cluster of CLUSTER CTAs takes a strip of columns of a group of rows, each
// CTA its share of the rows; the CTAs' column sums are added through
// distributed shared memory in rank order, so one group of rows (small
// batches) needs no second kernel.  More groups leave one row of sums each,
// which launch_add_rows adds in order.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "linear.cuh"
#include "row_util.cuh"
#include "tcgen05.cuh"

namespace mt {
namespace {

using namespace linear;
using namespace row;

constexpr int CLUSTER = 8;
constexpr int WARPS = 8;
constexpr int BATCH = 4;  // rows a warp has in flight

// Columns a lane takes of a row: eight side by side moved as 16 bytes, or
// four single ones, 32 apart.
template <bool VEC>
struct Lane {
  static constexpr int STEP = VEC ? 8 : 1;
  static constexpr int COUNT = VEC ? 1 : 4;
  static constexpr int STRIP = 32 * STEP * COUNT;
  static __device__ __forceinline__ int col(int i, int lane) { return (i * 32 + lane) * STEP; }
};

template <class T>
struct Operands {
  Matrix<const T> dY, Z;
  Matrix<T> dZ;
  Matrix<float> sums;  // a row per group
};

template <class T, int ACT, bool VEC>
__global__ void __launch_bounds__(32 * WARPS)
    linear_dz_kernel(const LinearDzArgs a, const Operands<T> o, int ctas,
                     int64_t rows_per_cta) {
  using L = Lane<VEC>;
  using Item = typename Held<T, L::STEP, VEC>::Item;
  __shared__ float warp_sums[WARPS][L::STRIP], cta_sums[L::STRIP];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int cta = static_cast<int>(blockIdx.x) % ctas;  // of the strip's
  const int c0 = static_cast<int>(blockIdx.x) / ctas * L::STRIP;
  const int64_t first = cta * rows_per_cta;
  const int64_t last = min(a.M, first + rows_per_cta);
  float s[L::COUNT][L::STEP];
#pragma unroll
  for (int i = 0; i < L::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < L::STEP; ++k) s[i][k] = 0.0f;
  for (int64_t row0 = first + warp; row0 < last; row0 += BATCH * WARPS) {
    Item dy[BATCH][L::COUNT], z[BATCH][L::COUNT];
#pragma unroll
    for (int r = 0; r < BATCH; ++r)
#pragma unroll
      for (int i = 0; i < L::COUNT; ++i) {
        const int64_t row = row0 + r * WARPS;
        const int c = c0 + L::col(i, lane);
        const bool live = row < last && c < a.N;
        const int64_t at = row * o.dY.ld + c, zt = row * o.Z.ld + c;
        dy[r][i] = live && o.dY.ok(at, L::STEP) ? *reinterpret_cast<const Item*>(o.dY.p + at)
                                                : Item{};
        if (ACT != ACT_NONE)
          z[r][i] = live && o.Z.ok(zt, L::STEP) ? *reinterpret_cast<const Item*>(o.Z.p + zt)
                                                : Item{};
      }
#pragma unroll
    for (int r = 0; r < BATCH; ++r)
#pragma unroll
      for (int i = 0; i < L::COUNT; ++i) {
        const int64_t row = row0 + r * WARPS;
        const int c = c0 + L::col(i, lane);
        if (row >= last || c >= a.N) continue;
        float v[L::STEP], zv[L::STEP];
        if constexpr (VEC) {
          dy[r][i].get(v);
          if (ACT != ACT_NONE) z[r][i].get(zv);
        } else {
          v[0] = to_f32(dy[r][i]);
          if (ACT != ACT_NONE) zv[0] = to_f32(z[r][i]);
        }
#pragma unroll
        for (int k = 0; k < L::STEP; ++k) {
          // Never fused into the sum: the same bits with and without dZ.
          if (ACT != ACT_NONE) v[k] = __fmul_rn(v[k], activate_grad<ACT>(zv[k]));
          s[i][k] += v[k];
        }
        if (a.dZ) store_step<T, VEC>(o.dZ, row, c, v);
      }
  }
  if (!a.dbias) return;  // the whole cluster
#pragma unroll
  for (int i = 0; i < L::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < L::STEP; ++k) warp_sums[warp][L::col(i, lane) + k] = s[i][k];
  __syncthreads();
  if (threadIdx.x < L::STRIP) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) t += warp_sums[w][threadIdx.x];
    cta_sums[threadIdx.x] = t;
  }
  tc::cluster_sync();
  constexpr int SHARE = L::STRIP / CLUSTER;
  if (threadIdx.x < SHARE) {
    const int j = static_cast<int>(tc::cluster_ctarank()) * SHARE + threadIdx.x, c = c0 + j;
    float t = 0.0f;
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r)
      t += tc::ld_cluster_f32(tc::map_to_cta(smem_u32(cta_sums + j), r));
    if (c < a.N) o.sums.store(cta / CLUSTER, c, t);
  }
  tc::cluster_sync();  // no CTA leaves while its sums are being read
}

template <class T>
bool vectored(const LinearDzArgs& a) {
  return a.N % 8 == 0 && rows_aligned(a.dY, a.lddy, 2) &&
         rows_aligned(a.Z, a.act == ACT_NONE ? 0 : a.ldz, 2) && rows_aligned(a.dZ, a.lddz, 2);
}

// Groups of rows: four CTAs on every SM, but no CTA with fewer than 64 rows
// once there is one group.
int row_groups(const LinearDzArgs& a, int strip, int sms) {
  const int64_t strips = (a.N - 1) / strip + 1;
  const int64_t want = 4 * static_cast<int64_t>(sms) / (strips * CLUSTER);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, a.M / (64 * CLUSTER))));
}

template <class T, int ACT, bool VEC>
cudaError_t launch(const LinearDzArgs& a, float* partial, int sms, cudaStream_t stream) {
  constexpr int STRIP = Lane<VEC>::STRIP;
  const int groups = row_groups(a, STRIP, sms);
  int ctas = groups * CLUSTER;
  int64_t per = (a.M + ctas - 1) / ctas;
  float* sums = groups > 1 ? partial : a.dbias;
  LinearDzArgs args = a;
  Operands<T> o{
      {static_cast<const T*>(a.dY), a.lddy, view_extent(a.M, a.N, a.lddy), a.bounds},
      {static_cast<const T*>(a.Z), a.ldz, view_extent(a.M, a.N, a.ldz), a.bounds},
      {static_cast<T*>(a.dZ), a.lddz, view_extent(a.M, a.N, a.lddz), a.bounds},
      {sums, a.N, static_cast<int64_t>(groups) * a.N, a.bounds}};
  void* list[] = {&args, &o, &ctas, &per};
  const cudaError_t e = launch_dependent(
      reinterpret_cast<const void*>(linear_dz_kernel<T, ACT, VEC>),
      dim3(static_cast<unsigned>(ctas) * static_cast<unsigned>((a.N - 1) / STRIP + 1)),
      32 * WARPS, 0, CLUSTER, stream, list);
  if (e != cudaSuccess || !a.dbias || groups == 1) return e;
  return launch_add_rows(partial, groups, a.N, a.dbias, a.bounds, stream);
}

template <class T, int ACT>
cudaError_t launch_vec(const LinearDzArgs& a, float* partial, int sms, cudaStream_t stream) {
  return vectored<T>(a) ? launch<T, ACT, true>(a, partial, sms, stream)
                        : launch<T, ACT, false>(a, partial, sms, stream);
}

template <class T>
cudaError_t launch_act(const LinearDzArgs& a, float* partial, int sms, cudaStream_t stream) {
  switch (a.act) {
    case ACT_RELU: return launch_vec<T, ACT_RELU>(a, partial, sms, stream);
    case ACT_GELU: return launch_vec<T, ACT_GELU>(a, partial, sms, stream);
    case ACT_GELU_TANH: return launch_vec<T, ACT_GELU_TANH>(a, partial, sms, stream);
    case ACT_SILU: return launch_vec<T, ACT_SILU>(a, partial, sms, stream);
    default: return launch_vec<T, ACT_NONE>(a, partial, sms, stream);
  }
}

}  // namespace

int64_t linear_dz_workspace(const LinearDzArgs& a, int sms) {
  // The wider strip has the more groups.
  const int groups = row_groups(a, Lane<true>::STRIP, sms);
  return a.dbias && groups > 1 ? static_cast<int64_t>(groups) * a.N * 4 : 0;
}

cudaError_t launch_linear_dz(const LinearDzArgs& a, void* partial, int sms,
                             cudaStream_t stream) {
  float* p = static_cast<float*>(partial);
  return a.dtype == DT_F16 ? launch_act<__half>(a, p, sms, stream)
                           : launch_act<__nv_bfloat16>(a, p, sms, stream);
}

}  // namespace mt
