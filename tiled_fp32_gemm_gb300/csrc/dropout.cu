// Dropout with the residual's addition: y = D(x) + residual.
//
// Bound by memory as long as the random words keep up: 4 or 6 bytes an element
// in 16 bits against a quarter of a Philox block (some 15 instruction slots).
// A CTA takes whole rows side by side, or strips of one; a thread holds several
// rows' loads in flight.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "model.h"
#include "philox.cuh"
#include "row_util.cuh"

namespace mt {
namespace {

using namespace row;

constexpr int kThreads = 256;

template <class T>
struct Operands {
  Matrix<const T> x, residual;
  Matrix<T> y;
};

// Aligned rows, eight columns an access.  `across` threads (a power of two)
// lie side by side on a row, which `strips` CTAs cut where it is wider.
template <class T, bool RES>
__global__ void __launch_bounds__(kThreads)
    dropout_kernel(const DropoutCall a, const Operands<T> o, int across, int strips) {
  constexpr int BATCH = sizeof(T) == 4 ? 2 : 4;  // rows a thread has in flight
  grid_launch_dependents();
  grid_wait();
  const int tid = threadIdx.x % across, down = kThreads / across;
  const int strip = static_cast<int>(blockIdx.x) % strips;
  const int group = static_cast<int>(blockIdx.x) / strips;
  const int groups = static_cast<int>(gridDim.x) / strips;
  const int64_t c64 = (static_cast<int64_t>(strip) * across + tid) * 8;
  if (c64 >= a.d) return;
  const int c = static_cast<int>(c64);
  Dropout drop;
  drop.init(a.dropout);
  const int64_t step = static_cast<int64_t>(groups) * down;
  auto load = [&](const Matrix<const T>& m, int64_t row) {
    const int64_t at = row * m.ld + c;
    return m.ok(at, 8) ? *reinterpret_cast<const Pack8<T>*>(m.p + at) : Pack8<T>{};
  };
  for (int64_t row0 = static_cast<int64_t>(group) * down + threadIdx.x / across;
       row0 < a.rows; row0 += BATCH * step) {
    Pack8<T> x[BATCH], r[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int64_t row = row0 + i * step;
      if (row >= a.rows) break;
      x[i] = load(o.x, row);
      if (RES) r[i] = load(o.residual, row);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int64_t row = row0 + i * step;
      if (row >= a.rows) break;
      float v[8];
      x[i].get(v);
      drop.apply8(static_cast<uint32_t>(row), c, v);
      if (RES) {
        float u[8];
        r[i].get(u);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += u[k];
      }
      store_step<T, true>(o.y, row, c, v);
    }
  }
}

// Rows that start on any element: a warp takes 32 neighbouring columns at a
// time, N such strips a warp's width of the CTA apart.
template <class T, bool RES>
__global__ void __launch_bounds__(kThreads)
    dropout_single_kernel(const DropoutCall a, const Operands<T> o, int across, int strips) {
  constexpr int N = 8;
  grid_launch_dependents();
  grid_wait();
  const int tid = threadIdx.x % across, down = kThreads / across;  // across >= 32
  const int strip = static_cast<int>(blockIdx.x) % strips;
  const int group = static_cast<int>(blockIdx.x) / strips;
  const int groups = static_cast<int>(gridDim.x) / strips;
  const int64_t first = static_cast<int64_t>(strip) * across * N;
  if (first + tid - static_cast<int>(threadIdx.x % 32) >= a.d) return;  // a whole warp
  const int c0 = static_cast<int>(first) + tid;
  Dropout drop;
  drop.init(a.dropout);
  for (int64_t row = static_cast<int64_t>(group) * down + threadIdx.x / across;
       row < a.rows; row += static_cast<int64_t>(groups) * down) {
    T x[N], r[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * across;
      const int64_t ax = row * o.x.ld + c, ar = row * o.residual.ld + c;
      x[i] = c < a.d && o.x.ok(ax, 1) ? o.x.p[ax] : T(0.0f);
      if (RES) r[i] = c < a.d && o.residual.ok(ar, 1) ? o.residual.p[ar] : T(0.0f);
    }
    uint32_t words[N];
    __syncwarp();
    drop.words_of_columns(static_cast<uint32_t>(row), c0, across, words);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * across;
      const float v = drop.apply(to_f32(x[i]), words[i]);
      if (c < a.d) o.y.store(row, c, RES ? v + to_f32(r[i]) : v);
    }
  }
}

template <class T, bool RES>
cudaError_t launch(const DropoutCall& a, int sms, cudaStream_t stream) {
  const int64_t n = a.rows;
  const Operands<T> o{
      {static_cast<const T*>(a.x), a.ldx, view_extent(n, a.d, a.ldx), a.bounds},
      {static_cast<const T*>(a.residual), a.ldr, view_extent(n, a.d, a.ldr), a.bounds},
      {static_cast<T*>(a.y), a.ldy, view_extent(n, a.d, a.ldy), a.bounds}};
  const int e = sizeof(T);
  const bool vec = a.d % 8 == 0 && rows_aligned(a.x, a.ldx, e) &&
                   rows_aligned(a.residual, RES ? a.ldr : 0, e) && rows_aligned(a.y, a.ldy, e);
  const int per = 8;  // columns a thread takes of a row, in either form
  int across = vec ? 1 : 32;
  while (across < kThreads && static_cast<int64_t>(across) * per < a.d) across *= 2;
  const int64_t strips = (a.d + static_cast<int64_t>(across) * per - 1) / (across * per);
  const int down = kThreads / across;
  // Enough CTAs for eight waves of eight on every SM, no more than there are
  // rows for.
  const int64_t groups = std::min((n + down - 1) / down,
                                  std::max<int64_t>(1, 64 * static_cast<int64_t>(sms) / strips));
  const unsigned grid = static_cast<unsigned>(groups * strips);
  const int cut = static_cast<int>(strips);
  return vec ? launch_dependent(dropout_kernel<T, RES>, grid, kThreads, stream, a, o, across, cut)
             : launch_dependent(dropout_single_kernel<T, RES>, grid, kThreads, stream, a, o,
                                across, cut);
}

template <class T>
cudaError_t launch_residual(const DropoutCall& a, int sms, cudaStream_t stream) {
  return a.residual ? launch<T, true>(a, sms, stream) : launch<T, false>(a, sms, stream);
}

}  // namespace

cudaError_t launch_dropout(const DropoutCall& a, int sms, cudaStream_t stream) {
  switch (a.dtype) {
    case DT_F16: return launch_residual<__half>(a, sms, stream);
    case DT_BF16: return launch_residual<__nv_bfloat16>(a, sms, stream);
    default: return launch_residual<float>(a, sms, stream);
  }
}

}  // namespace mt
