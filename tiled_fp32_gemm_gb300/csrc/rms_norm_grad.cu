// Gradient of the root-mean-square norm: with xhat = h * rstd, g = dy * weight,
//   dx = rstd * (g - xhat * mean(g * xhat)) + dh,   dweight = sum over rows of dy * xhat.
// Bound by memory: dy, h, dh and dx move once, in rms_norm_grad_kernel, which
// keeps its columns' share of dweight in registers from row to row; the CTAs'
// shares are added in a fixed order by a second kernel.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "row_util.cuh"

namespace mt {
namespace {

using namespace row;

template <class T>
struct Operands {
  Matrix<const T> dy, h, dh;
  Matrix<T> dx;
  Matrix<const float> rstd;
  Matrix<float> partial;  // one row of d sums per group of rows
};

// Threads of an SM the register kernel is built for: 16-bit rows moved by
// 16-byte accesses hold 4 registers per matrix and 8 values.
template <class T, bool VEC>
constexpr int sm_threads() {
  return sizeof(T) == 2 && VEC ? 1024 : 512;
}
constexpr int ctas_per_sm(int threads, int sm) { return sm > threads ? sm / threads : 1; }

// A row held in the registers of THREADS threads, E values each; rows
// strided over the grid.  The next row's values are loaded before this row's
// reduction, so a barrier leaves loads in flight.  Each thread reads its
// values of a row before it writes them, so dx may be dy or dh.
template <class T, class W, int THREADS, int E, bool VEC>
__global__ void __launch_bounds__(THREADS* rows_per_cta(THREADS),
                                  ctas_per_sm(THREADS* rows_per_cta(THREADS),
                                              sm_threads<T, VEC>()))
    rms_norm_grad_kernel(const RmsNormGradArgs a, const Operands<T> o,
                         const Matrix<const W> weight) {
  using S = Slots<E, VEC>;
  constexpr int ROWS = rows_per_cta(THREADS), WARPS = THREADS / 32;
  __shared__ float sums[2][WARPS];  // by turns, so one barrier a row is enough
  const int tid = threadIdx.x % THREADS, lane = threadIdx.x % 32, warp = tid / 32;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / THREADS;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * ROWS;
  struct Row {
    Held<T, E, VEC> dy, h, dh;
    float r;
    __device__ __forceinline__ void load(const RmsNormGradArgs& a, const Operands<T>& o,
                                         int64_t row, int tid) {
      if (row >= a.rows) return;
      dy.load(o.dy, row, a.d, tid, THREADS);
      h.load(o.h, row, a.d, tid, THREADS);
      if (a.dh) dh.load(o.dh, row, a.d, tid, THREADS);
      r = o.rstd.load(row, 0);
    }
  };
  grid_launch_dependents();
  grid_wait();
  Held<W, E, VEC> w;
  if (a.weight) w.load(weight, 0, a.d, tid, THREADS);
  float dw[S::COUNT][S::STEP];
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < S::STEP; ++k) dw[i][k] = 0.0f;
  Row next;
  next.load(a, o, group, tid);
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += groups, turn ^= 1) {
    Row now = next;
    next.load(a, o, row + groups, tid);
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) {
      float vy[S::STEP], vh[S::STEP], vw[S::STEP];
      now.dy.get(i, vy);
      now.h.get(i, vh);
      if (a.weight) w.get(i, vw);
#pragma unroll
      for (int k = 0; k < S::STEP; ++k) {
        const float xhat = vh[k] * now.r;
        dw[i][k] = fmaf(vy[k], xhat, dw[i][k]);
        dot = fmaf(a.weight ? vy[k] * vw[k] : vy[k], xhat, dot);
      }
    }
    now.dy.keep();
    now.h.keep();
    w.keep();
    dot = warp_sum(dot);
    if constexpr (THREADS > 32) {
      if (lane == 0) sums[turn][warp] = dot;
      __syncthreads();
      dot = warp_sum(lane < WARPS ? sums[turn][lane] : 0.0f);
    }
    const float mean = dot / static_cast<float>(a.d);
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) {
      const int c = S::col(i, tid, THREADS);
      if (c >= a.d) break;
      float vy[S::STEP], vh[S::STEP], vw[S::STEP], vd[S::STEP];
      now.dy.get(i, vy);
      now.h.get(i, vh);
      if (a.weight) w.get(i, vw);
      if (a.dh) now.dh.get(i, vd);
#pragma unroll
      for (int k = 0; k < S::STEP; ++k) {
        const float g = a.weight ? vy[k] * vw[k] : vy[k];
        const float dx = now.r * (g - vh[k] * now.r * mean);
        vy[k] = a.dh ? dx + vd[k] : dx;
      }
      store_step<T, VEC>(o.dx, row, c, vy);
    }
  }
  if (!a.dweight) return;
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i) {
    const int c = S::col(i, tid, THREADS);
    if (c < a.d) store_step<float, VEC>(o.partial, group, c, dw[i]);
  }
}

// dx of a row too wide for registers, on one CTA: one sweep for the mean, one
// for dx, each element read and then written by the same thread.
constexpr int kWideThreads = 512;

template <class T, class W>
__global__ void __launch_bounds__(kWideThreads)
    rms_norm_grad_wide_kernel(const RmsNormGradArgs a, const Operands<T> o,
                              const Matrix<const W> weight) {
  __shared__ float part[kWideThreads / 32];
  grid_launch_dependents();
  grid_wait();
  const int64_t row = blockIdx.x;
  auto weight_at = [&](int c) { return a.weight ? weight.load(0, c) : 1.0f; };
  const float r = o.rstd.load(row, 0);
  float dot = 0.0f;
  for (int c = threadIdx.x; c < a.d; c += kWideThreads)
    dot = fmaf(o.dy.load(row, c) * weight_at(c), o.h.load(row, c) * r, dot);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  dot = warp_sum(dot);
  if (lane == 0) part[warp] = dot;
  __syncthreads();
  dot = warp_sum(lane < kWideThreads / 32 ? part[lane] : 0.0f);
  const float mean = dot / static_cast<float>(a.d);
  for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
    const float g = o.dy.load(row, c) * weight_at(c);
    const float dx = r * (g - o.h.load(row, c) * r * mean) + (a.dh ? o.dh.load(row, c) : 0.0f);
    o.dx.store(row, c, dx);
  }
}

// dweight of wide rows: column sums of dy * xhat over one block of rows.  A
// CTA takes 32 columns, its 8 warps every eighth row of the block.
constexpr int kColumnWarps = 8;

template <class T>
__global__ void __launch_bounds__(32 * kColumnWarps)
    rms_norm_grad_columns_kernel(const RmsNormGradArgs a, const Operands<T> o,
                                 int64_t rows_per_block) {
  __shared__ float sums[kColumnWarps][32];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  const int64_t first = blockIdx.y * rows_per_block;
  const int64_t last = min(a.rows, first + rows_per_block);
  float s = 0.0f;
  if (c < a.d)
    for (int64_t i = first + warp; i < last; i += kColumnWarps)
      s = fmaf(o.dy.load(i, c), o.h.load(i, c) * o.rstd.load(i, 0), s);
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
    s = 0.0f;
#pragma unroll
    for (int w = 0; w < kColumnWarps; ++w) s += sums[w][lane];
    o.partial.store(blockIdx.y, c, s);
  }
}

// Adds the partial rows: a CTA takes 32 columns, its 32 warps every 32nd row.
__global__ void __launch_bounds__(1024) add_rows_kernel(const Matrix<const float> rows,
                                                        int count, int cols,
                                                        const Matrix<float> out) {
  __shared__ float sums[32][33];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int i = warp; i < count; i += 32) s += rows.load(i, c);
  sums[warp][lane] = s;
  __syncthreads();
  // Warp w adds the 32 sums of column w.
  s = warp_sum(sums[lane][warp]);
  const int cw = blockIdx.x * 32 + warp;
  if (lane == 0 && cw < cols) out.store(0, cw, s);
}

// Whether every matrix of a call is read and written by 16-byte accesses.
template <class T, class W>
bool vectored(const RmsNormGradArgs& a) {
  const int e = sizeof(T);
  return a.d % 8 == 0 && rows_aligned(a.dy, a.lddy, e) && rows_aligned(a.h, a.ldh, e) &&
         rows_aligned(a.dh, a.dh ? a.lddh : 0, e) && rows_aligned(a.dx, a.lddx, e) &&
         rows_aligned(a.weight, 0, sizeof(W));
}

// CTAs of the register kernel: those resident at once, and no more groups of
// rows than rows.
int held_ctas(const RmsNormGradArgs& a, int threads, int sm, int sms) {
  const int rows = rows_per_cta(threads);
  const int64_t want = (a.rows + rows - 1) / rows;
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>(want, int64_t(sms) * ctas_per_sm(threads * rows, sm))));
}

// Blocks of rows of the wide column sums: enough CTAs for four waves of eight
// on each SM, at least 32 rows each.
int column_blocks(int64_t rows, int cols, int sms) {
  const int64_t strips = (cols + 31) / 32;
  const int64_t want = std::max<int64_t>(1, 32 * static_cast<int64_t>(sms) / strips);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (rows + 31) / 32)));
}

// Most partial rows of dweight a call writes.
int64_t partial_rows(const RmsNormGradArgs& a, int sms) {
  int64_t n = 0;
  const bool held = row_layout<8>(a.d, [&](auto threads, auto) {
    constexpr int THREADS = decltype(threads)::value;
    n = static_cast<int64_t>(held_ctas(a, THREADS, 1024, sms)) * rows_per_cta(THREADS);
  });
  return held ? n : column_blocks(a.rows, a.d, sms);
}

template <class T, class W>
cudaError_t launch(const RmsNormGradArgs& a, float* partial, int sms, cudaStream_t stream) {
  const int64_t n = a.rows;
  int parts = static_cast<int>(partial_rows(a, sms));
  const Operands<T> o{
      {static_cast<const T*>(a.dy), a.lddy, view_extent(n, a.d, a.lddy), a.bounds},
      {static_cast<const T*>(a.h), a.ldh, view_extent(n, a.d, a.ldh), a.bounds},
      {static_cast<const T*>(a.dh), a.lddh, view_extent(n, a.d, a.lddh), a.bounds},
      {static_cast<T*>(a.dx), a.lddx, view_extent(n, a.d, a.lddx), a.bounds},
      {a.rstd, 1, n, a.bounds},
      {partial, a.d, static_cast<int64_t>(parts) * a.d, a.bounds}};
  const Matrix<const W> weight{static_cast<const W*>(a.weight), 0, a.d, a.bounds};
  const bool vec = vectored<T, W>(a);
  const int sm = vec ? sm_threads<T, true>() : sm_threads<T, false>();
  cudaError_t err = cudaSuccess;
  const bool held = row_layout<8>(a.d, [&](auto threads, auto values) {
    constexpr int THREADS = decltype(threads)::value, E = decltype(values)::value;
    const int ctas = held_ctas(a, THREADS, sm, sms), block = THREADS * rows_per_cta(THREADS);
    parts = ctas * rows_per_cta(THREADS);
    err = launch_dependent(vec ? rms_norm_grad_kernel<T, W, THREADS, E, true>
                               : rms_norm_grad_kernel<T, W, THREADS, E, false>,
                           ctas, block, stream, a, o, weight);
  });
  if (!held) {
    // The column sums come first: dx may overwrite dy.
    if (a.dweight)
      err = launch_dependent(rms_norm_grad_columns_kernel<T>, dim3((a.d + 31) / 32, parts),
                             32 * kColumnWarps, stream, a, o, (n + parts - 1) / parts);
    if (err == cudaSuccess && n > 0)
      err = launch_dependent(rms_norm_grad_wide_kernel<T, W>, static_cast<unsigned>(n),
                             kWideThreads, stream, a, o, weight);
  }
  if (err != cudaSuccess || !a.dweight) return err;
  return launch_add_rows(partial, parts, a.d, a.dweight, a.bounds, stream);
}

template <class T>
cudaError_t launch_weight(const RmsNormGradArgs& a, float* partial, int sms,
                          cudaStream_t stream) {
  return a.weight_f32 ? launch<T, float>(a, partial, sms, stream)
                      : launch<T, T>(a, partial, sms, stream);
}

}  // namespace

cudaError_t launch_add_rows(const float* rows, int count, int cols, float* out,
                            BoundsRecord* bounds, cudaStream_t stream) {
  return launch_dependent(
      add_rows_kernel, dim3((cols + 31) / 32), 1024, stream,
      Matrix<const float>{rows, cols, static_cast<int64_t>(count) * cols, bounds}, count, cols,
      Matrix<float>{out, cols, cols, bounds});
}

int64_t rms_norm_grad_workspace(const RmsNormGradArgs& a, int sms) {
  return a.dweight ? partial_rows(a, sms) * a.d * 4 : 0;
}

cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, void* workspace, int sms,
                                 cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  switch (a.dtype) {
    case DT_F16: return launch_weight<__half>(a, partial, sms, stream);
    case DT_BF16: return launch_weight<__nv_bfloat16>(a, partial, sms, stream);
    default: return launch_weight<float>(a, partial, sms, stream);
  }
}

}  // namespace mt
