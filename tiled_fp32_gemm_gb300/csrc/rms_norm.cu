// Root-mean-square norm with the residual's addition, 16- or 32-bit output
// or e4m3 output with one scale per row.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h * r * weight
//   e4m3:  scale = max(max|y| / 448, 2^-126),  q = e4m3(y / scale)
//
// max|y| = r * max|h * weight| (r is one positive factor of the row), so the
// sum of squares and the maximum come from one sweep and one reduction.  The
// operator is bound by memory: every element of x, residual, h and y moves
// once, in rms_norm_kernel.  Measured on GB300, with residual, share of the
// copy bandwidth: 8192 x 8192 bf16 84 us, 0.94; fp32 177 us, 0.89; rows that do
// not start on 16 bytes (8000 x 8191 fp16), two bytes an access, 127 us, 0.61;
// to e4m3, 32768 x 8192 bf16 298 us, 0.93.
#include <cfloat>
#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "row_util.cuh"

namespace mt {
namespace {

using namespace row;

template <class T>
struct Operands {
  Matrix<const T> x, residual;
  Matrix<T> h, y;
  Matrix<uint8_t> q;
  Matrix<float> rstd, scale;
};

// r and, for 8-bit output, 1 / scale of a row; one thread writes them.
template <class T, bool E4M3>
__device__ __forceinline__ float row_factors(const RmsNormArgs& a, const Operands<T>& o,
                                             int64_t row, float sum, float top, bool writer,
                                             float* inv) {
  const float m = (a.d > 0 ? sum / static_cast<float>(a.d) : 0.0f) + a.eps;
  const float r = m == 0.0f ? 0.0f : rsqrtf(m);  // zeros stay zeros without an eps
  if (writer && a.rstd) o.rstd.store(row, 0, r);
  if (E4M3) {
    const float t = top * r / 448.0f;
    const float scale = t < FLT_MIN ? FLT_MIN : t;  // a NaN stays one
    *inv = 1.0f / scale;
    if (writer) o.scale.store(row, 0, scale);
  }
  return r;
}

// Sum and maximum over the THREADS threads of a row, in every one of them.
template <int THREADS, bool E4M3>
__device__ __forceinline__ void reduce_row(float& sum, float& top) {
  sum = warp_sum(sum);
  if (E4M3) top = warp_max(top);
  if constexpr (THREADS > 32) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float sums[WARPS], tops[WARPS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) {
      sums[warp] = sum;
      if (E4M3) tops[warp] = top;
    }
    __syncthreads();
    sum = warp_sum(lane < WARPS ? sums[lane] : 0.0f);
    if (E4M3) top = warp_max(lane < WARPS ? tops[lane] : 0.0f);
  }
}

// A row held in the registers of THREADS threads, E values each: read once,
// reduced once, written.  Each thread reads its values before it writes
// them, so h may be x or residual and y may be x.
template <class T, class W, bool E4M3, int THREADS, int E, bool VEC>
__global__ void __launch_bounds__(THREADS* rows_per_cta(THREADS))
    rms_norm_kernel(const RmsNormArgs a, const Operands<T> o, const Matrix<const W> weight) {
  using S = Slots<E, VEC>;
  grid_launch_dependents();
  grid_wait();
  const int tid = threadIdx.x % THREADS;
  const int64_t row =
      static_cast<int64_t>(blockIdx.x) * rows_per_cta(THREADS) + threadIdx.x / THREADS;
  if (row >= a.rows) return;  // a whole warp
  Held<T, E, VEC> x, res;
  Held<W, E, VEC> w;
  x.load(o.x, row, a.d, tid, THREADS);
  if (a.residual) res.load(o.residual, row, a.d, tid, THREADS);
  if (a.weight) w.load(weight, 0, a.d, tid, THREADS);
  float h[S::COUNT][S::STEP];
  float sum = 0.0f, top = 0.0f;
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i) {
    x.get(i, h[i]);
    if (a.residual) {
      float v[S::STEP];
      res.get(i, v);
#pragma unroll
      for (int k = 0; k < S::STEP; ++k) h[i][k] += v[k];
    }
#pragma unroll
    for (int k = 0; k < S::STEP; ++k) sum = fmaf(h[i][k], h[i][k], sum);
    if (E4M3) {
      float v[S::STEP];
      if (a.weight) w.get(i, v);
#pragma unroll
      for (int k = 0; k < S::STEP; ++k)
        top = fmaxf(top, fabsf(a.weight ? h[i][k] * v[k] : h[i][k]));
    }
  }
  reduce_row<THREADS, E4M3>(sum, top);
  float inv = 0.0f;
  const float r = row_factors<T, E4M3>(a, o, row, sum, top, tid == 0, &inv);
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i) {
    const int c = S::col(i, tid, THREADS);
    if (c >= a.d) break;
    if (a.h) store_step<T, VEC>(o.h, row, c, h[i]);
    float y[S::STEP];
    if (a.weight) w.get(i, y);
#pragma unroll
    for (int k = 0; k < S::STEP; ++k)
      y[k] = (a.weight ? h[i][k] * r * y[k] : h[i][k] * r) * (E4M3 ? inv : 1.0f);
    if constexpr (E4M3) {
      const int64_t at = row * o.q.ld + c;
      if (!o.q.ok(at, S::STEP)) continue;
      if constexpr (VEC) {
        const uint32_t lo = e4m3x2(y[0], y[1]) | static_cast<uint32_t>(e4m3x2(y[2], y[3])) << 16;
        const uint32_t hi = e4m3x2(y[4], y[5]) | static_cast<uint32_t>(e4m3x2(y[6], y[7])) << 16;
        *reinterpret_cast<uint2*>(o.q.p + at) = make_uint2(lo, hi);
      } else {
        o.q.p[at] = static_cast<uint8_t>(e4m3x2(y[0], 0.0f));
      }
    } else {
      store_step<T, VEC>(o.y, row, c, y);
    }
  }
}

// A row too wide for registers, on one CTA: one sweep for the statistics,
// one for the outputs, which reads x and the residual again (from L2: a row
// of 2^20 fp32 elements is 4 MB; 2048 x 40000 bf16 with residual 246 us, 0.39 of
// the copy bandwidth).  Each element is read and then written by
// the same thread, in the second sweep only, so h may be x or residual.
constexpr int kWideThreads = 512;

template <class T, class W, bool E4M3>
__global__ void __launch_bounds__(kWideThreads)
    rms_norm_wide_kernel(const RmsNormArgs a, const Operands<T> o,
                         const Matrix<const W> weight) {
  grid_launch_dependents();
  grid_wait();
  const int64_t row = blockIdx.x;
  auto load = [&](int c) {
    return o.x.load(row, c) + (a.residual ? o.residual.load(row, c) : 0.0f);
  };
  auto weight_at = [&](int c) { return a.weight ? weight.load(0, c) : 1.0f; };
  float sum = 0.0f, top = 0.0f;
  for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
    const float h = load(c);
    sum = fmaf(h, h, sum);
    if (E4M3) top = fmaxf(top, fabsf(h * weight_at(c)));
  }
  reduce_row<kWideThreads, E4M3>(sum, top);
  float inv = 0.0f;
  const float r = row_factors<T, E4M3>(a, o, row, sum, top, threadIdx.x == 0, &inv);
  for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
    const float h = load(c);
    const float y = h * r * weight_at(c);
    if (a.h) o.h.store(row, c, h);
    if constexpr (E4M3) {
      const int64_t at = row * o.q.ld + c;
      if (o.q.ok(at, 1)) o.q.p[at] = static_cast<uint8_t>(e4m3x2(y * inv, 0.0f));
    } else {
      o.y.store(row, c, y);
    }
  }
}

template <class T, class W, bool E4M3>
cudaError_t launch(const RmsNormArgs& a, cudaStream_t stream) {
  const int64_t n = a.rows;
  const Operands<T> o{
      {static_cast<const T*>(a.x), a.ldx, view_extent(n, a.d, a.ldx), a.bounds},
      {static_cast<const T*>(a.residual), a.ldr, view_extent(n, a.d, a.ldr), a.bounds},
      {static_cast<T*>(a.h), a.ldh, view_extent(n, a.d, a.ldh), a.bounds},
      {static_cast<T*>(a.y), a.ldy, view_extent(n, a.d, a.ldy), a.bounds},
      {static_cast<uint8_t*>(a.y), a.ldy, view_extent(n, a.d, a.ldy), a.bounds},
      {a.rstd, 1, n, a.bounds},
      {a.scale, 1, n, a.bounds}};
  const Matrix<const W> weight{static_cast<const W*>(a.weight), 0, a.d, a.bounds};
  const int e = sizeof(T);
  const bool vec = a.d % 8 == 0 && rows_aligned(a.x, a.ldx, e) &&
                   rows_aligned(a.residual, a.residual ? a.ldr : 0, e) &&
                   rows_aligned(a.h, a.h ? a.ldh : 0, e) &&
                   rows_aligned(a.y, a.ldy, E4M3 ? 1 : e) &&
                   rows_aligned(a.weight, 0, sizeof(W));
  cudaError_t err = cudaSuccess;
  const bool held = row_layout<16>(a.d, [&](auto threads, auto values) {
    constexpr int THREADS = decltype(threads)::value, E = decltype(values)::value;
    constexpr int ROWS = rows_per_cta(THREADS);
    err = launch_dependent(vec ? rms_norm_kernel<T, W, E4M3, THREADS, E, true>
                               : rms_norm_kernel<T, W, E4M3, THREADS, E, false>,
                           static_cast<unsigned>((n + ROWS - 1) / ROWS), THREADS * ROWS, stream,
                           a, o, weight);
  });
  if (!held)
    err = launch_dependent(rms_norm_wide_kernel<T, W, E4M3>, static_cast<unsigned>(n),
                           kWideThreads, stream, a, o, weight);
  return err;
}

template <class T>
cudaError_t launch_out(const RmsNormArgs& a, cudaStream_t stream) {
  if (a.weight_f32)
    return a.e4m3 ? launch<T, float, true>(a, stream) : launch<T, float, false>(a, stream);
  return a.e4m3 ? launch<T, T, true>(a, stream) : launch<T, T, false>(a, stream);
}

}  // namespace

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case DT_F16: return launch_out<__half>(a, stream);
    case DT_BF16: return launch_out<__nv_bfloat16>(a, stream);
    default: return launch_out<float>(a, stream);
  }
}

}  // namespace mt
