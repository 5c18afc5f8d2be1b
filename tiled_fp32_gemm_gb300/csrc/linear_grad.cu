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

constexpr int STRIP = 32 * 8;  // columns of a strip: a lane takes eight side by side

template <class T>
struct Operands {
  Matrix<const T> dY, Z;
  Matrix<T> dZ;
  Matrix<float> sums;  // a row per group
};

// ALIGNED: every eighth column of every row starts on 16 bytes and N % 8 ==
// 0; else rows start on any element (load8_any).  Rows of dZ are always
// aligned and padded to whole chunks.
template <class T, int ACT, bool ALIGNED>
__global__ void __launch_bounds__(32 * WARPS, 3)
    linear_dz_kernel(const LinearDzArgs a, const Operands<T> o, int ctas,
                     int64_t rows_per_cta) {
  constexpr int BATCH = ALIGNED ? 4 : 2;  // rows a warp has in flight
  __shared__ float warp_sums[WARPS][STRIP], cta_sums[STRIP];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int cta = static_cast<int>(blockIdx.x) % ctas;  // of the strip's
  const int c0 = static_cast<int>(blockIdx.x) / ctas * STRIP, c = c0 + lane * 8;
  const int64_t first = cta * rows_per_cta;
  const int64_t last = min(a.M, first + rows_per_cta);
  auto load = [&](const Matrix<const T>& m, int64_t row) {
    if constexpr (ALIGNED) {
      const int64_t at = row * m.ld + c;
      return m.ok(at, 8) ? *reinterpret_cast<const Pack8<T>*>(m.p + at) : Pack8<T>{};
    } else {
      return load8_any(m, row, c, a.N);
    }
  };
  float s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = 0.0f;
  if (c < a.N) {
    for (int64_t row0 = first + warp; row0 < last; row0 += BATCH * WARPS) {
      Pack8<T> dy[BATCH], z[BATCH];
#pragma unroll
      for (int r = 0; r < BATCH; ++r) {
        const int64_t row = row0 + r * WARPS;
        if (row >= last) break;
        dy[r] = load(o.dY, row);
        if (ACT != ACT_NONE) z[r] = load(o.Z, row);
      }
#pragma unroll
      for (int r = 0; r < BATCH; ++r) {
        const int64_t row = row0 + r * WARPS;
        if (row >= last) break;
        float v[8], zv[8];
        dy[r].get(v);
        if (ACT != ACT_NONE) z[r].get(zv);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          // Never fused into the sum: the same bits with and without dZ.
          if (ACT != ACT_NONE) v[k] = __fmul_rn(v[k], activate_grad<ACT>(zv[k]));
          s[k] += v[k];
        }
        if (a.dZ) store_step<T, true>(o.dZ, row, c, v);
      }
    }
  }
  if (!a.dbias) return;  // the whole cluster
#pragma unroll
  for (int k = 0; k < 8; ++k) warp_sums[warp][lane * 8 + k] = s[k];
  __syncthreads();
  static_assert(32 * WARPS == STRIP, "a thread per column");
  float t = 0.0f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) t += warp_sums[w][threadIdx.x];
  cta_sums[threadIdx.x] = t;
  tc::cluster_sync();
  constexpr int SHARE = STRIP / CLUSTER;
  if (threadIdx.x < SHARE) {
    const int j = static_cast<int>(tc::cluster_ctarank()) * SHARE + threadIdx.x;
    t = 0.0f;
#pragma unroll
    for (int r = 0; r < CLUSTER; ++r)
      t += tc::ld_cluster_f32(tc::map_to_cta(smem_u32(cta_sums + j), r));
    if (c0 + j < a.N) o.sums.store(cta / CLUSTER, c0 + j, t);
  }
  tc::cluster_sync();  // no CTA leaves while its sums are being read
}

bool aligned(const LinearDzArgs& a) {
  return a.N % 8 == 0 && rows_aligned(a.dY, a.lddy, 2) &&
         (a.act == ACT_NONE || rows_aligned(a.Z, a.ldz, 2));
}

// Groups of rows: four CTAs on every SM, but no CTA with fewer than 16 rows
// once there is one group.
int row_groups(const LinearDzArgs& a, int sms) {
  const int64_t strips = (a.N - 1) / STRIP + 1;
  const int64_t want = 4 * static_cast<int64_t>(sms) / (strips * CLUSTER);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, a.M / (16 * CLUSTER))));
}

template <class T, int ACT>
cudaError_t launch(const LinearDzArgs& a, float* partial, int sms, cudaStream_t stream) {
  const int groups = row_groups(a, sms);
  int ctas = groups * CLUSTER;
  int64_t per = (a.M + ctas - 1) / ctas;
  float* sums = groups > 1 ? partial : a.dbias;
  LinearDzArgs args = a;
  Operands<T> o{
      {static_cast<const T*>(a.dY), a.lddy, view_extent(a.M, a.N, a.lddy), a.bounds},
      {static_cast<const T*>(a.Z), a.ldz, view_extent(a.M, a.N, a.ldz), a.bounds},
      {static_cast<T*>(a.dZ), a.lddz, a.M * a.lddz, a.bounds},
      {sums, a.N, static_cast<int64_t>(groups) * a.N, a.bounds}};
  void* list[] = {&args, &o, &ctas, &per};
  const cudaError_t e = launch_dependent(
      aligned(a) ? reinterpret_cast<const void*>(linear_dz_kernel<T, ACT, true>)
                 : reinterpret_cast<const void*>(linear_dz_kernel<T, ACT, false>),
      dim3(static_cast<unsigned>(ctas) * static_cast<unsigned>((a.N - 1) / STRIP + 1)),
      32 * WARPS, 0, CLUSTER, stream, list);
  if (e != cudaSuccess || !a.dbias || groups == 1) return e;
  return launch_add_rows(partial, groups, a.N, a.dbias, a.bounds, stream);
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
  const int groups = row_groups(a, sms);
  return a.dbias && groups > 1 ? static_cast<int64_t>(groups) * a.N * 4 : 0;
}

cudaError_t launch_linear_dz(const LinearDzArgs& a, void* partial, int sms,
                             cudaStream_t stream) {
  float* p = static_cast<float*>(partial);
  return a.dtype == DT_F16 ? launch_act<__half>(a, p, sms, stream)
                           : launch_act<__nv_bfloat16>(a, p, sms, stream);
}

}  // namespace mt
