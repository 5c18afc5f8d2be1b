// Dropout with the residual's addition: y = D(x) + residual.
//
// Bound by memory with a residual (16384 x 8192 bf16 124 us, 0.96 of the copy
// rate), by the random words without (104 us, 0.76: the wide products fill the
// multiplier four fifths of the time); fp32 is 0.98 of it.  Rows that do not start
// on 16 bytes are bound by their single-element accesses (16384 x 8191 bf16 208
// us).  Two rows a thread in flight and four CTAs an SM, whose threads set up
// their columns once: four rows and three CTAs 127 us, two and five 130; eight
// times as many CTAs, that set up as much oftener, 148.
#include <algorithm>
#include <cstdint>

#include <cuda_runtime.h>

#include "model.h"
#include "philox.cuh"
#include "row_chunk.cuh"

namespace mt {
namespace {

using namespace row;

constexpr int kThreads = 256;
constexpr int kCtasPerSm = 4;

template <class T>
struct Operands {
  Matrix<const T> x, residual;
  Matrix<T> y;
};

// `across` threads (a power of two) share a row, a chunk of eight columns
// each, or, where it is wider, one of the row's `strips`.  A thread keeps its
// columns from row to row, and their part of the random words with them.
// ACROSS: across, 0 where it is known at run time only.
template <class T, bool RES, bool ALIGNED, int ACROSS>
__global__ void __launch_bounds__(kThreads, kCtasPerSm)
    dropout_kernel(const DropoutCall a, const Operands<T> o, int across, int strips) {
  using At = Chunk<ALIGNED, ACROSS>;
  constexpr int BATCH = sizeof(T) == 4 ? 1 : 2;  // rows a thread has in flight
  grid_launch_dependents();
  grid_wait();
  const int strip = static_cast<int>(blockIdx.x) % strips;
  const int group = static_cast<int>(blockIdx.x) / strips;
  const int groups = static_cast<int>(gridDim.x) / strips;
  if (ACROSS > 0) across = ACROSS;
  const int down = kThreads / across;
  const At at(strip, threadIdx.x % across, across);
  Dropout drop;
  drop.init(a.dropout);
  const typename At::Words words = at.words(drop);
  const int64_t step = static_cast<int64_t>(groups) * down;
  const int lead = threadIdx.x / across;
  // All threads of the CTA go round together: lanes exchange random words.
  for (int64_t row0 = static_cast<int64_t>(group) * down; row0 < a.rows; row0 += BATCH * step) {
    Eight<T, ALIGNED> x[BATCH], r[BATCH];
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int64_t row = row0 + lead + i * step;
      if (row >= a.rows) break;
      x[i] = at.load(o.x, row, a.d);
      if (RES) r[i] = at.load(o.residual, row, a.d);
    }
#pragma unroll
    for (int i = 0; i < BATCH; ++i) {
      const int64_t row = row0 + lead + i * step;
      float v[8];
      x[i].get(v);
      __syncwarp();
      at.drop(drop, drop.row(static_cast<uint32_t>(row)), words, v);
      if (row >= a.rows) continue;
      if (RES) {
        float u[8];
        r[i].get(u);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += u[k];
      }
      at.store(o.y, row, a.d, v);
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
  const bool aligned = a.d % 8 == 0 && rows_aligned(a.x, a.ldx, e) &&
                       rows_aligned(a.residual, RES ? a.ldr : 0, e) &&
                       rows_aligned(a.y, a.ldy, e);
  int across = aligned ? 1 : 4;  // four lanes share a quad's random words
  while (across < kThreads && static_cast<int64_t>(across) * 8 < a.d) across *= 2;
  const int64_t strips = (a.d + static_cast<int64_t>(across) * 8 - 1) / (across * 8);
  const int down = kThreads / across;
  // Two rounds of resident CTAs on every SM: each sets up its columns' part of
  // the random words once.  No more than there are rows for.
  const int64_t groups =
      std::min((n + down - 1) / down,
               std::max<int64_t>(1, 2 * kCtasPerSm * static_cast<int64_t>(sms) / strips));
  const unsigned grid = static_cast<unsigned>(groups * strips);
  const int cut = static_cast<int>(strips);
  const bool wide = across == kThreads;
  auto* const kernel = aligned ? dropout_kernel<T, RES, true, 0>
                       : wide  ? dropout_kernel<T, RES, false, kThreads>
                               : dropout_kernel<T, RES, false, 0>;
  return launch_dependent(kernel, grid, kThreads, stream, a, o, across, cut);
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
