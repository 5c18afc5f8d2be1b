// Gradient of the root-mean-square norm: with xhat = h * rstd, g = dy * weight,
//   dx = rstd * (g - xhat * mean(g * xhat)) + dh,   dweight = sum over rows of dy * xhat.
// Bound by memory: dy, h, dh and dx move once; a thread keeps its columns'
// share of dweight in registers from row to row, and the CTAs' shares are
// added in a fixed order by a second kernel.  Rows that start on 16 bytes
// stream through shared memory (rms_norm_grad_staged_kernel), others through
// registers (rms_norm_grad_kernel), rows too wide for either are read twice.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "row_util.cuh"
#include "tcgen05.cuh"

namespace mt {
namespace {

using namespace row;

__device__ unsigned int g_status;  // bit 0: a bounded wait expired

template <class T>
struct Operands {
  Matrix<const T> dy, h, dh;
  Matrix<T> dx;
  Matrix<const float> rstd;
  Matrix<float> partial;  // one row of d sums per group of rows
};

// How the staged kernel shares its threads out: `threads` take a row (at most
// e values each), `groups` rows make up a stage.
struct Staging {
  int threads, groups, e, most, stages;
  int dh;  // 0: none, 1: in the ring, 2: read where it is needed
  int stage_bytes, smem_bytes;
};
constexpr int kStagedBytes = 200 * 1024;
constexpr int kBarrierBytes = 256;

// Rows of up to 16384 values, in one of three forms: 16 values a thread and
// 608 threads (96 registers each, which leave nothing to spill); the same
// with 800 threads (72 registers, up to 36 bytes of spill stores a thread for
// 16-bit rows, 64 for fp32) where they hold two rows and 608 would hold one,
// or where 608 would not hold a row; 32 values and 512 threads past that (96
// registers: with the copy warp they are 17 warps; up to 128 bytes of spill
// stores, 208 for fp32).  false when two stages do not fit.  Measured on GB300
// (bf16 with dh, share of the measured copy bandwidth): 2048 values 0.98, 4096
// 0.94, 8192 0.93, 7168 (one group of 448 threads) 0.85, 5120 in the 608 form
// 0.57 and in the 800 form 0.76, 12288 0.58, 16384 0.51; fp32, 8192 values
// 0.80.
bool staging_of(int d, int elem, bool dh, Staging* s) {
  if (d > 16384) return false;
  s->e = d <= 16 * 800 ? 16 : 32;
  s->threads = (d + 32 * s->e - 1) / (32 * s->e) * 32;
  // dh stays out of the ring where three stages of a row would not fit.
  const int row_bytes = d * elem;
  s->dh = !dh ? 0 : 9 * row_bytes <= kStagedBytes ? 1 : 2;
  const int mats = s->dh == 1 ? 3 : 2, rows = kStagedBytes / (3 * mats * row_bytes);
  const bool two = 2 * s->threads > 608 && 2 * s->threads <= 800 && rows >= 2;
  s->most = s->e == 32 ? 512 : two || s->threads > 608 ? 800 : 608;
  s->groups = s->most / s->threads;
  if (s->threads > 32) s->groups = std::min(s->groups, 15);  // named barriers
  s->groups = std::max(1, std::min(s->groups, rows));
  s->stage_bytes = s->groups * mats * row_bytes;
  s->stages = std::min(8, kStagedBytes / s->stage_bytes);
  // The column sums of the groups meet in the ring.
  s->smem_bytes = std::max(s->stages * s->stage_bytes, d * 4) + kBarrierBytes + 128;
  return s->stages >= 2;
}

// Rows stream through a ring of shared-memory stages: the last warp copies
// the next rows of dy, h and dh (bulk copies) while the others work, so the
// loads in flight do not depend on registers or on the barrier inside a row.
// A group of `threads` threads takes a row of the stage: its mean, then dx,
// both from shared memory, the one beside the other of the row before, so one
// barrier a row is all that is waited for.  dx may be dy or dh: a row's copies
// have landed before it is written.  Waits are bounded; after one that ran out
// (recorded in the status word) the results are unspecified.  Measured on
// GB300, 16384 x 8192 bf16 with dh: 170 us, 6.3 TB/s (209 us with the rows in
// registers and loads one row ahead).
template <class T, class W, int E, int MOST, int DH>
__global__ void __launch_bounds__(MOST + 32, 1)
    rms_norm_grad_staged_kernel(const RmsNormGradArgs a, const Operands<T> o,
                                const Matrix<const W> weight, const Staging g) {
  using S = Slots<E, true>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);  // full[stages], empty[stages]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 16);
  uint8_t* ring = smem + kBarrierBytes;
  __shared__ float sums[2][MOST / 32];  // by turns: one barrier a row is enough
  const tc::WaitCtx wc{abort_flag, &g_status};
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int workers = g.threads * g.groups, worker_warps = workers / 32;
  const int row_bytes = a.d * static_cast<int>(sizeof(T)), mats = DH == 1 ? 3 : 2;
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + 8 + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      tc::mbar_init(full(s), 1);               // the copy warp's arrival + bytes
      tc::mbar_init(empty(s), worker_warps);  // every worker warp
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  grid_launch_dependents();
  grid_wait();

  const int64_t step = static_cast<int64_t>(gridDim.x) * g.groups;
  const int64_t row_0 = static_cast<int64_t>(blockIdx.x) * g.groups;
  float dw[S::COUNT][8];
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = 0.0f;
  const int group = static_cast<int>(threadIdx.x) / g.threads;
  const int tid = static_cast<int>(threadIdx.x) % g.threads;
  int issued = 0;
  if (warp == worker_warps) {
    for (int64_t row0 = row_0; row0 < a.rows && !a.fault_inject; row0 += step, ++issued) {
      const int s = issued % g.stages, round = issued / g.stages;
      if (issued >= g.stages &&
          !__all_sync(0xffffffffu, tc::wait_phase(empty(s), (round + 1) & 1u, wc)))
        break;
      const int rows = static_cast<int>(min(static_cast<int64_t>(g.groups), a.rows - row0));
      if (lane == 0) tc::mbar_arrive_expect_tx(full(s), rows * mats * row_bytes);
      __syncwarp();
      // A matrix without gaps between its rows arrives in one copy.
      for (int m = 0; m < mats; ++m) {
        const Matrix<const T>& from = m == 0 ? o.dy : m == 1 ? o.h : o.dh;
        const bool packed = from.ld == a.d;
        for (int i = lane; i < (packed ? 1 : rows); i += 32)
          tc::bulk_copy_g2s(
              smem_u32(ring + s * g.stage_bytes + (m * g.groups + i) * row_bytes),
              from.p + (row0 + i) * from.ld, packed ? rows * row_bytes : row_bytes, full(s));
      }
    }
  } else {
    Held<W, E, true> w;
    if (a.weight) w.load(weight, 0, a.d, tid, g.threads);
    else w.fill(1.0f);
    const int warps = g.threads / 32, first_warp = group * warps;
    auto rstd_of = [&](int64_t row) { return row < a.rows ? o.rstd.load(row, 0) : 0.0f; };
    auto values = [&](int n, int m) {  // matrix m of the group's row of stage n
      return reinterpret_cast<const T*>(ring + n % g.stages * g.stage_bytes) +
             (m * g.groups + group) * a.d;
    };
    // First sweep of the group's n-th row: its dweight and, for every warp of
    // the group, the sum of dy * weight * xhat.
    auto first_sweep = [&](int n, bool live, float r) {
      tc::wait_phase(full(n % g.stages), (n / g.stages) & 1u, wc);
      const T *dy = values(n, 0), *h = values(n, 1);
      float dot = 0.0f;
#pragma unroll
      for (int i = 0; i < S::COUNT; ++i) {
        const int c = S::col(i, tid, g.threads);
        if (!live || c >= a.d) break;
        float vy[8], vh[8], vw[8];
        reinterpret_cast<const Pack8<T>*>(dy + c)->get(vy);
        reinterpret_cast<const Pack8<T>*>(h + c)->get(vh);
        w.get(i, vw);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float xhat = vh[k] * r;
          dw[i][k] = fmaf(vy[k], xhat, dw[i][k]);
          dot = fmaf(vy[k] * vw[k], xhat, dot);
        }
      }
      dot = warp_sum(dot);
      if (lane == 0) sums[n & 1][warp] = dot;
    };
    auto meet = [&] {
      __syncwarp();  // lane 0 alone wrote or arrived last; bar.sync wants the warp converged
      if (warps > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(g.threads) : "memory");
    };
    float r = rstd_of(row_0 + group), r_next = rstd_of(row_0 + step + group);
    if (row_0 < a.rows) first_sweep(0, row_0 + group < a.rows, r);
    meet();
    int n = 0;
    for (int64_t row0 = row_0; row0 < a.rows; row0 += step, ++n) {
      const int64_t row = row0 + group;
      const bool live = row < a.rows;  // the whole group
      // dx = r * (g - back * h) + dh, back = r * mean(g * xhat): with r factored
      // in once more (r * g - r * back * h), r * back would pass fp32's range
      // for rows of values near 1e-19 or 1e19, whose gradient does not.
      const float dot = warp_sum(lane < warps ? sums[n & 1][first_warp + lane] : 0.0f);
      const float back = r * (dot / static_cast<float>(a.d));
      // The next row's first sweep runs beside this row's second.
      const float r_after = rstd_of(row + 2 * step);
      if (row0 + step < a.rows) first_sweep(n + 1, row + step < a.rows, r_next);
      const T *dy = values(n, 0), *h = values(n, 1), *dh = values(n, 2);
#pragma unroll
      for (int i = 0; i < S::COUNT; ++i) {
        const int c = S::col(i, tid, g.threads);
        if (!live || c >= a.d) break;
        float vy[8], vh[8], vw[8], dx[8];
        reinterpret_cast<const Pack8<T>*>(dy + c)->get(vy);
        reinterpret_cast<const Pack8<T>*>(h + c)->get(vh);
        w.get(i, vw);
        if (DH == 1) reinterpret_cast<const Pack8<T>*>(dh + c)->get(dx);
        if (DH == 2)
          reinterpret_cast<const Pack8<T>*>(o.dh.p + row * o.dh.ld + c)->get(dx);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float grad = vy[k] * vw[k];
          dx[k] = fmaf(r, fmaf(-back, vh[k], grad), DH ? dx[k] : 0.0f);
        }
        store_step<T, true>(o.dx, row, c, dx);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(empty(n % g.stages));
      r = r_next;
      r_next = r_after;
      meet();
    }
  }
  __syncthreads();
  if (warp == worker_warps) {
    // After a wait that ran out: let the copies issued land before the CTA
    // exits.
    if (*abort_flag)
      for (int i = issued > g.stages ? issued - g.stages : 0; i < issued; ++i)
        tc::wait_phase(full(i % g.stages), (i / g.stages) & 1u, wc, false);
  }
  if (!a.dweight) return;
  // The groups' column sums, in group order; the ring is idle.
  float* columns = reinterpret_cast<float*>(ring);
  for (int turn = 0; turn < g.groups; ++turn) {
    if (warp < worker_warps && group == turn) {
#pragma unroll
      for (int i = 0; i < S::COUNT; ++i) {
        const int c = S::col(i, tid, g.threads);
        if (c >= a.d) break;
        if (turn > 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) dw[i][k] += columns[c + k];
        }
        if (turn == g.groups - 1) {
          store_step<float, true>(o.partial, blockIdx.x, c, dw[i]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) columns[c + k] = dw[i][k];
        }
      }
    }
    if (g.groups > 1) __syncthreads();
  }
}

// Threads of an SM the register kernel is built for.
constexpr int kSmThreads = 512;
constexpr int ctas_per_sm(int threads) { return kSmThreads > threads ? kSmThreads / threads : 1; }

// A row held in the registers of THREADS threads, E values each; rows
// strided over the grid.  Up to 512 threads the next row's values are loaded
// before this row's reduction, so a barrier leaves loads in flight; 1024 have
// no registers for that (with them, 8000 x 8191 fp16 with dh took 309 us,
// without 135 to 139: 0.56 of the copy rate, two bytes an access).
// Each thread reads its values of a row before it writes them, so dx may be
// dy or dh.
template <class T, class W, int THREADS, int E, bool DH>
__global__ void __launch_bounds__(THREADS* rows_per_cta(THREADS),
                                  ctas_per_sm(THREADS* rows_per_cta(THREADS)))
    rms_norm_grad_kernel(const RmsNormGradArgs a, const Operands<T> o,
                         const Matrix<const W> weight) {
  using S = Slots<E, false>;
  constexpr int ROWS = rows_per_cta(THREADS), WARPS = THREADS / 32;
  constexpr bool AHEAD = THREADS <= 512;
  __shared__ float sums[2][WARPS];  // by turns, so one barrier a row is enough
  const int tid = threadIdx.x % THREADS, lane = threadIdx.x % 32, warp = tid / 32;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / THREADS;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * ROWS;
  struct Row {
    Held<T, E, false> dy, h, dh;
    float r;
    __device__ __forceinline__ void load(const RmsNormGradArgs& a, const Operands<T>& o,
                                         int64_t row, int tid) {
      if (row >= a.rows) return;
      dy.load(o.dy, row, a.d, tid, THREADS);
      h.load(o.h, row, a.d, tid, THREADS);
      if (DH) dh.load(o.dh, row, a.d, tid, THREADS);
      r = o.rstd.load(row, 0);
    }
  };
  grid_launch_dependents();
  grid_wait();
  Held<W, E, false> w;
  if (a.weight) w.load(weight, 0, a.d, tid, THREADS);
  else w.fill(1.0f);
  float dw[S::COUNT][S::STEP];
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < S::STEP; ++k) dw[i][k] = 0.0f;
  Row next;
  if (AHEAD) next.load(a, o, group, tid);
  int turn = 0;
  for (int64_t row = group; row < a.rows; row += groups, turn ^= 1) {
    Row now;
    if constexpr (AHEAD) {
      now = next;
      next.load(a, o, row + groups, tid);
    } else {
      now.load(a, o, row, tid);
    }
    const float r = now.r;
    float dot = 0.0f;
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) {
      float vy[S::STEP], vh[S::STEP], vw[S::STEP];
      now.dy.get(i, vy);
      now.h.get(i, vh);
      w.get(i, vw);
#pragma unroll
      for (int k = 0; k < S::STEP; ++k) {
        const float xhat = vh[k] * r;
        dw[i][k] = fmaf(vy[k], xhat, dw[i][k]);
        dot = fmaf(vy[k] * vw[k], xhat, dot);
      }
    }
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
      w.get(i, vw);
      if (DH) now.dh.get(i, vd);
#pragma unroll
      for (int k = 0; k < S::STEP; ++k) {
        const float g = vy[k] * vw[k];
        vy[k] = fmaf(r, fmaf(-mean, vh[k] * r, g), DH ? vd[k] : 0.0f);
      }
      store_step<T, false>(o.dx, row, c, vy);
    }
  }
  if (!a.dweight) return;
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i) {
    const int c = S::col(i, tid, THREADS);
    if (c < a.d) store_step<float, false>(o.partial, group, c, dw[i]);
  }
}

// dx of a row too wide for registers, on one CTA: one sweep for the mean, one
// for dx, each element read and then written by the same thread.  2048 x 40000
// bf16 with dh and dweight: 506 us, 0.19 of the copy rate.
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
    const float dx =
        fmaf(r, fmaf(-mean, o.h.load(row, c) * r, g), a.dh ? o.dh.load(row, c) : 0.0f);
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
bool vectored(const RmsNormGradArgs& a) {
  const int e = dtype_bytes(a.dtype);
  return a.d % 8 == 0 && rows_aligned(a.dy, a.lddy, e) && rows_aligned(a.h, a.ldh, e) &&
         rows_aligned(a.dh, a.dh ? a.lddh : 0, e) && rows_aligned(a.dx, a.lddx, e) &&
         rows_aligned(a.weight, 0, a.weight_f32 ? 4 : e);
}

// CTAs of a kernel that takes `rows` rows a CTA at a time, `per_sm` of them
// resident on an SM: no more than there are rows for.
int ctas_of(int64_t n, int rows, int per_sm, int sms) {
  return static_cast<int>(std::max<int64_t>(
      1, std::min<int64_t>((n + rows - 1) / rows, int64_t(sms) * per_sm)));
}

// Blocks of rows of the wide column sums: enough CTAs for four waves of eight
// on each SM, at least 32 rows each.
int column_blocks(int64_t rows, int cols, int sms) {
  const int64_t strips = (cols + 31) / 32;
  const int64_t want = std::max<int64_t>(1, 32 * static_cast<int64_t>(sms) / strips);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (rows + 31) / 32)));
}

// Which kernel a call takes, and the partial rows of dweight it writes.
enum Path { STAGED, HELD, WIDE };

Path path_of(const RmsNormGradArgs& a, int sms, Staging* g, int* parts) {
  const int e = dtype_bytes(a.dtype);
  if (vectored(a) && staging_of(a.d, e, a.dh != nullptr, g)) {
    *parts = ctas_of(a.rows, g->groups, 1, sms);
    return STAGED;
  }
  const bool held = row_layout<8>(a.d, [&](auto threads, auto) {
    constexpr int ROWS = rows_per_cta(decltype(threads)::value);
    *parts = ctas_of(a.rows, ROWS, ctas_per_sm(decltype(threads)::value * ROWS), sms) * ROWS;
  });
  if (held) return HELD;
  *parts = column_blocks(a.rows, a.d, sms);
  return WIDE;
}

template <class T, class W>
cudaError_t launch(const RmsNormGradArgs& a, float* partial, int sms, cudaStream_t stream) {
  const int64_t n = a.rows;
  Staging g{};
  int parts = 0;
  const Path path = path_of(a, sms, &g, &parts);
  const Operands<T> o{
      {static_cast<const T*>(a.dy), a.lddy, view_extent(n, a.d, a.lddy), a.bounds},
      {static_cast<const T*>(a.h), a.ldh, view_extent(n, a.d, a.ldh), a.bounds},
      {static_cast<const T*>(a.dh), a.lddh, view_extent(n, a.d, a.lddh), a.bounds},
      {static_cast<T*>(a.dx), a.lddx, view_extent(n, a.d, a.lddx), a.bounds},
      {a.rstd, 1, n, a.bounds},
      {partial, a.d, static_cast<int64_t>(parts) * a.d, a.bounds}};
  const Matrix<const W> weight{static_cast<const W*>(a.weight), 0, a.d, a.bounds};
  cudaError_t err = cudaSuccess;
  if (path == STAGED) {
    // By form and dh; 32 values a thread never have dh in the ring.
    const int form = (g.e == 32 ? 6 : g.most == 800 ? 3 : 0) + g.dh;
#define MT_FORM(E, MOST, DH) \
  reinterpret_cast<const void*>(rms_norm_grad_staged_kernel<T, W, E, MOST, DH>)
    const void* const kernels[9] = {MT_FORM(16, 608, 0), MT_FORM(16, 608, 1), MT_FORM(16, 608, 2),
                                    MT_FORM(16, 800, 0), MT_FORM(16, 800, 1), MT_FORM(16, 800, 2),
                                    MT_FORM(32, 512, 0), nullptr,             MT_FORM(32, 512, 2)};
#undef MT_FORM
    const void* kernel = kernels[form];
    static std::atomic<uint64_t> ready[9];  // by kernel: devices whose limit is set
    int dev = 0;
    err = cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    std::atomic<uint64_t>& done = ready[form];
    if (err == cudaSuccess && !(done.load(std::memory_order_acquire) & bit)) {
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kStagedBytes + kBarrierBytes + 128);
      if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    }
    RmsNormGradArgs args = a;
    Operands<T> ops = o;
    Matrix<const W> w = weight;
    void* list[] = {&args, &ops, &w, &g};
    if (err == cudaSuccess)
      err = launch_dependent(kernel, static_cast<unsigned>(parts), g.threads * g.groups + 32,
                             g.smem_bytes, 1, stream, list);
  } else if (path == HELD) {
    row_layout<8>(a.d, [&](auto threads, auto values) {
      constexpr int THREADS = decltype(threads)::value, E = decltype(values)::value;
      constexpr int ROWS = rows_per_cta(THREADS);
      err = launch_dependent(a.dh ? rms_norm_grad_kernel<T, W, THREADS, E, true>
                                  : rms_norm_grad_kernel<T, W, THREADS, E, false>,
                             parts / ROWS, THREADS * ROWS, stream, a, o, weight);
    });
  } else {
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
  Staging g{};
  int parts = 0;
  path_of(a, sms, &g, &parts);
  return a.dweight ? static_cast<int64_t>(parts) * a.d * 4 : 0;
}

cudaError_t rms_norm_grad_read_and_clear_status(unsigned int* status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
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
