// Layer norm with dropout and the residual's addition.
//
//   h = D(x) + residual,  m = mean h,  r = 1 / sqrt(mean (h - m)^2 + eps),
//   y = (h - m) * r * weight + bias
//
// The operator is bound by memory: every element of x, residual, h and y moves
// once, and h stays in registers between the statistics and y.  The variance
// is the mean square of differences, in one sweep and one barrier: a warp sums
// its values, takes their differences from its own mean, and the warps' pairs
// (sum, squares about their mean) are joined by
//   squares = sum_w (squares_w + n_w * (mean_w - m)^2)
// (Chan, Golub and LeVeque, "Updating formulae and a pairwise algorithm for
// computing sample variances", 1979).  Arithmetic in pairs of values (one
// instruction each): with dropout 222 -> 198 us.  Measured on GB300, with
// residual, share of the copy rate: 16384 x 8192 bf16 172 us, 0.92; with dropout 198
// us, 0.80, where random words and memory take turns; fp32, unaligned, 8192 x 4095
// 82 us, 0.96; 16-bit unaligned 16384 x 4095 116 us, 0.68.
#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "model.h"
#include "pair_math.cuh"
#include "philox.cuh"
#include "row_chunk.cuh"

namespace mt {
namespace {

using namespace row;

template <class T>
struct Operands {
  Matrix<const T> x, residual;
  Matrix<T> h, y;
  Matrix<float> mean, rstd;
};

struct Stats {
  float mean, rstd;
};

__device__ __forceinline__ Stats stats_of(float mean, float squares, int d, float eps) {
  const float v = (d > 0 ? squares / static_cast<float>(d) : 0.0f) + eps;
  return Stats{mean, v == 0.0f ? 0.0f : rsqrtf(v)};  // a constant row stays one without an eps
}

// A warp's part of a row: how many values, their mean, their squares about it.
struct Part {
  float n, mean, squares;
};

// The row's mean and squares from the parts of the warps that share it, in
// every thread.  One barrier.
template <int THREADS>
__device__ __forceinline__ Part join(const Part& mine, int d) {
  if constexpr (THREADS == 32) {
    return mine;
  } else {
    constexpr int WARPS = THREADS / 32;
    __shared__ Part parts[WARPS];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (lane == 0) parts[warp] = mine;
    __syncthreads();
    const Part p = lane < WARPS ? parts[lane] : Part{0.0f, 0.0f, 0.0f};
    const float mean = d > 0 ? warp_sum(p.n * p.mean) / static_cast<float>(d) : 0.0f;
    const float off = p.mean - mean;
    return Part{static_cast<float>(d), mean,
                warp_sum(p.n > 0.0f ? fmaf(p.n * off, off, p.squares) : 0.0f)};
  }
}

// A row held in the registers of THREADS threads, E values each in chunks of
// eight: read once, reduced once, written.  Each thread reads its values before
// it writes them, so h may be x or residual and y may be x.  Single elements: 64
// registers a thread, for 1024 threads on an SM; what one row's barrier leaves idle
// the others fill (with 68, 512 threads of a row have the SM to themselves, and
// 16384 x 8191 takes 416 us instead of 277).  Aligned rows take less by themselves;
// held to that number they are scheduled for it (16384 x 8192 with dropout 220 us
// instead of 198).
template <class T, class W, bool DROP, int THREADS, int E, bool ALIGNED>
__global__ void __launch_bounds__(THREADS* rows_per_cta(THREADS),
                                  ALIGNED ? 0 : 1024 / (THREADS * rows_per_cta(THREADS)))
    layer_norm_kernel(const LayerNormArgs a, const Operands<T> o, const Matrix<const W> weight,
                      const Matrix<const W> bias) {
  using C = Chunks<T, E, ALIGNED, THREADS>;
  using At = Chunk<ALIGNED, THREADS>;
  grid_launch_dependents();
  grid_wait();
  const int tid = threadIdx.x % THREADS;
  const int64_t row =
      static_cast<int64_t>(blockIdx.x) * rows_per_cta(THREADS) + threadIdx.x / THREADS;
  if (row >= a.rows) return;  // a whole warp
  C x, res;
  x.load(o.x, row, a.d, tid);
  if (a.residual) res.load(o.residual, row, a.d, tid);
  float h[C::COUNT][8];
#pragma unroll
  for (int i = 0; i < C::COUNT; ++i) x.get(i, h[i]);
  if constexpr (DROP) {
    Dropout drop;
    drop.init(a.dropout);
    const Dropout::Row of_row = drop.row(static_cast<uint32_t>(row));
#pragma unroll
    for (int i = 0; i < C::COUNT; ++i) {
      const At at(i, tid);
      at.drop(drop, of_row, at.words(drop), h[i]);
    }
  }
  // Columns at or past d are zeros, which the sum does not feel.
  float2 sum2 = both(0.0f);
  int count = 0;
#pragma unroll
  for (int i = 0; i < C::COUNT; ++i) {
    if (a.residual) {
      float v[8];
      res.get(i, v);
#pragma unroll
      for (int k = 0; k < 8; k += 2) put2(h[i] + k, add2(get2(h[i] + k), get2(v + k)));
    }
#pragma unroll
    for (int k = 0; k < 8; k += 2) sum2 = add2(sum2, get2(h[i] + k));
    count += At(i, tid).count(a.d);
  }
  Part part;
  part.n = static_cast<float>(__reduce_add_sync(0xffffffffu, count));
  part.mean = part.n > 0.0f ? warp_sum(sum2.x + sum2.y) / part.n : 0.0f;
  float2 squares = both(0.0f);
#pragma unroll
  for (int i = 0; i < C::COUNT; ++i) {
    const At at(i, tid);
    const bool whole = at.whole(a.d);
    if (ALIGNED && !whole) break;
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float2 c = add2(get2(h[i] + k), both(-part.mean));
      if (!ALIGNED && !whole) {
        if (!at.live(k, a.d)) c.x = 0.0f;
        if (!at.live(k + 1, a.d)) c.y = 0.0f;
      }
      squares = fma2(c, c, squares);
    }
  }
  __syncwarp();
  part.squares = warp_sum(squares.x + squares.y);
  // Read while the row's statistics meet.
  Chunks<W, E, ALIGNED, THREADS> w, b;
  if (a.weight) w.load(weight, 0, a.d, tid);
  if (a.bias) b.load(bias, 0, a.d, tid);
  part = join<THREADS>(part, a.d);
  const Stats s = stats_of(part.mean, part.squares, a.d, a.eps);
  if (tid == 0) {
    if (a.mean) o.mean.store(row, 0, s.mean);
    if (a.rstd) o.rstd.store(row, 0, s.rstd);
  }
#pragma unroll
  for (int i = 0; i < C::COUNT; ++i) {
    const At at(i, tid);
    if (!at.any(a.d)) break;
    if (a.h) at.store(o.h, row, a.d, h[i]);
    float vw[8], vb[8];
    if (a.weight) w.get(i, vw);
    if (a.bias) b.get(i, vb);
#pragma unroll
    for (int k = 0; k < 8; k += 2) {
      float2 v = mul2(add2(get2(h[i] + k), both(-s.mean)), both(s.rstd));
      const float2 scale = a.weight ? get2(vw + k) : both(1.0f);
      if (a.bias) v = fma2(v, scale, get2(vb + k));
      else if (a.weight) v = mul2(v, scale);
      put2(h[i] + k, v);
    }
    at.store(o.y, row, a.d, h[i]);
  }
}

// A row too wide for registers, on one CTA: one sweep for the mean, one for
// the squares about it, one for the outputs, which read x and the residual
// again (from L2).  Each element is read and then written by the same thread,
// in the last sweep only, so h may be x or residual and y may be x.
constexpr int kWideThreads = 512;

__device__ __forceinline__ float wide_sum(float v, float (&part)[kWideThreads / 32]) {
  v = warp_sum(v);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  return warp_sum(threadIdx.x % 32 < kWideThreads / 32 ? part[threadIdx.x % 32] : 0.0f);
}

template <class T, class W, bool DROP, bool ALIGNED>
__global__ void __launch_bounds__(kWideThreads)
    layer_norm_wide_kernel(const LayerNormArgs a, const Operands<T> o,
                           const Matrix<const W> weight, const Matrix<const W> bias) {
  using At = Chunk<ALIGNED, kWideThreads>;
  __shared__ float sums[kWideThreads / 32], squares[kWideThreads / 32];
  grid_launch_dependents();
  grid_wait();
  const int64_t row = blockIdx.x;
  Dropout drop{};
  Dropout::Row of_row{};
  if (DROP) {
    drop.init(a.dropout);
    of_row = drop.row(static_cast<uint32_t>(row));
  }
  // Calls f(chunk, h) for this thread's chunks, all warps as many times.
  auto sweep = [&](auto&& f) {
    for (int i = 0; i * 8 * kWideThreads < a.d; ++i) {
      const At at(i, threadIdx.x);
      const auto x = at.load(o.x, row, a.d);
      Eight<T, ALIGNED> r{};
      if (a.residual) r = at.load(o.residual, row, a.d);
      float h[8], v[8];
      x.get(h);
      r.get(v);
      __syncwarp();
      if (DROP) at.drop(drop, of_row, at.words(drop), h);
#pragma unroll
      for (int k = 0; k < 8; ++k) h[k] += v[k];
      f(at, h);
    }
  };
  float t = 0.0f;
  sweep([&](const At&, const float(&h)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) t += h[k];
  });
  const float mean = wide_sum(t, sums) / static_cast<float>(a.d);
  t = 0.0f;
  sweep([&](const At& at, const float(&h)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float v = at.live(k, a.d) ? h[k] - mean : 0.0f;
      t = fmaf(v, v, t);
    }
  });
  const Stats s = stats_of(mean, wide_sum(t, squares), a.d, a.eps);
  if (threadIdx.x == 0) {
    if (a.mean) o.mean.store(row, 0, s.mean);
    if (a.rstd) o.rstd.store(row, 0, s.rstd);
  }
  sweep([&](const At& at, float(&h)[8]) {
    if (a.h) at.store(o.h, row, a.d, h);
    Eight<W, ALIGNED> w{}, b{};
    if (a.weight) w = at.load(weight, 0, a.d);
    if (a.bias) b = at.load(bias, 0, a.d);
    float vw[8], vb[8];
    w.get(vw);
    b.get(vb);
#pragma unroll
    for (int k = 0; k < 8; ++k)
      h[k] = fmaf((h[k] - s.mean) * s.rstd, a.weight ? vw[k] : 1.0f, vb[k]);
    at.store(o.y, row, a.d, h);
  });
}

// Calls f(threads per row, values per thread) with a row's layout; false past
// 16384.  A warp by itself up to 512: no barrier, and no idle half of a second
// warp's values (65536 x 417 bf16 with dropout 77 us, 152 with 64 threads of 16).
template <class F>
bool norm_layout(int d, F&& f) {
  if (d > 256 && d <= 512) {
    f(std::integral_constant<int, 32>{}, std::integral_constant<int, 16>{});
    return true;
  }
  return row_layout<16>(d, f);
}

template <class T, class W, bool DROP>
cudaError_t launch(const LayerNormArgs& a, cudaStream_t stream) {
  const int64_t n = a.rows;
  const Operands<T> o{
      {static_cast<const T*>(a.x), a.ldx, view_extent(n, a.d, a.ldx), a.bounds},
      {static_cast<const T*>(a.residual), a.ldr, view_extent(n, a.d, a.ldr), a.bounds},
      {static_cast<T*>(a.h), a.ldh, view_extent(n, a.d, a.ldh), a.bounds},
      {static_cast<T*>(a.y), a.ldy, view_extent(n, a.d, a.ldy), a.bounds},
      {a.mean, 1, n, a.bounds},
      {a.rstd, 1, n, a.bounds}};
  const Matrix<const W> weight{static_cast<const W*>(a.weight), 0, a.d, a.bounds};
  const Matrix<const W> bias{static_cast<const W*>(a.bias), 0, a.d, a.bounds};
  const int e = sizeof(T);
  const bool aligned = a.d % 8 == 0 && rows_aligned(a.x, a.ldx, e) &&
                   rows_aligned(a.residual, a.residual ? a.ldr : 0, e) &&
                   rows_aligned(a.h, a.h ? a.ldh : 0, e) && rows_aligned(a.y, a.ldy, e) &&
                   rows_aligned(a.weight, 0, sizeof(W)) && rows_aligned(a.bias, 0, sizeof(W));
  cudaError_t err = cudaSuccess;
  const bool held = norm_layout(a.d, [&](auto threads, auto values) {
    constexpr int THREADS = decltype(threads)::value, E = decltype(values)::value;
    constexpr int ROWS = rows_per_cta(THREADS);
    err = launch_dependent(aligned ? layer_norm_kernel<T, W, DROP, THREADS, E, true>
                                   : layer_norm_kernel<T, W, DROP, THREADS, E, false>,
                           static_cast<unsigned>((n + ROWS - 1) / ROWS), THREADS * ROWS, stream,
                           a, o, weight, bias);
  });
  if (!held)
    err = launch_dependent(aligned ? layer_norm_wide_kernel<T, W, DROP, true>
                                   : layer_norm_wide_kernel<T, W, DROP, false>,
                           static_cast<unsigned>(n), kWideThreads, stream, a, o, weight, bias);
  return err;
}

template <class T>
cudaError_t launch_drop(const LayerNormArgs& a, cudaStream_t stream) {
  if (a.weight_f32)
    return a.drop ? launch<T, float, true>(a, stream) : launch<T, float, false>(a, stream);
  return a.drop ? launch<T, T, true>(a, stream) : launch<T, T, false>(a, stream);
}

}  // namespace

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t stream) {
  switch (a.dtype) {
    case DT_F16: return launch_drop<__half>(a, stream);
    case DT_BF16: return launch_drop<__nv_bfloat16>(a, stream);
    default: return launch_drop<float>(a, stream);
  }
}

}  // namespace mt
