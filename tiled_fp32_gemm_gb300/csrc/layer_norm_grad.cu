// Gradient of the layer norm with dropout and the residual's addition: with
// xhat = (h - mean) * rstd, g = dy * weight,
//   dres = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dh,   dx = D(dres),
//   dweight = sum over rows of dy * xhat,   dbias = sum over rows of dy.
// Bound by memory: dy, h, dh, dx and (with dropout) dres move once; a thread
// keeps its columns' shares of dweight and dbias in registers from row to row,
// and the CTAs' shares are added in a fixed order by a second kernel.  Rows
// that start on 16 bytes stream through shared memory
// (layer_norm_grad_staged_kernel), others through registers
// (layer_norm_grad_kernel); rows too wide for either are read twice.
#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "model.h"
#include "philox.cuh"
#include "row_util.cuh"
#include "tcgen05.cuh"

namespace mt {
namespace {

using namespace row;

__device__ unsigned int g_status;  // bit 0: a bounded wait expired

template <class T>
struct Operands {
  Matrix<const T> dy, h, dh;
  Matrix<T> dx, dres;
  Matrix<const float> mean, rstd;
  // For every group of rows a row of d sums of dy * xhat, then one of dy: the
  // groups' dweight rows first.
  Matrix<float> partial_w, partial_b;
};

// What a row needs besides its values.
struct RowStats {
  float mean, rstd;
};

// One element's gradient before dh.
__device__ __forceinline__ float grad_of(float g, float xhat, float mean_g, float mean_gx,
                                         float rstd) {
  return rstd * fmaf(-xhat, mean_gx, g - mean_g);
}

// How the staged kernel shares its threads out: `threads` take a row (at most
// e values each), `groups` rows make up a stage.
struct Staging {
  int threads, groups, e, most, stages;
  int dh;  // 0: none, 1: in the ring, 2: read where it is needed
  int stage_bytes, smem_bytes;
};
constexpr int kStagedBytes = 200 * 1024;
constexpr int kBarrierBytes = 256;

// Rows of up to 16384 values: 16 values a thread and 512 threads, or 32 values
// past 8192.  false when two stages do not fit.
bool staging_of(int d, int elem, bool dh, Staging* s) {
  if (d > 16384) return false;
  s->most = 512;
  s->e = d <= 16 * 512 ? 16 : 32;
  s->threads = (d + 32 * s->e - 1) / (32 * s->e) * 32;
  const int row_bytes = d * elem;
  // dh stays out of the ring where three stages of a row would not fit, and
  // where a thread has 32 values.
  s->dh = !dh ? 0 : s->e == 16 && 9 * row_bytes <= kStagedBytes ? 1 : 2;
  const int mats = s->dh == 1 ? 3 : 2, rows = kStagedBytes / (3 * mats * row_bytes);
  s->groups = s->most / s->threads;
  if (s->threads > 32) s->groups = std::min(s->groups, 15);  // named barriers
  s->groups = std::max(1, std::min(s->groups, rows));
  s->stage_bytes = s->groups * mats * row_bytes;
  s->stages = std::min(8, kStagedBytes / s->stage_bytes);
  // The column sums of the groups meet in the ring.
  s->smem_bytes = std::max(s->stages * s->stage_bytes, 2 * d * 4) + kBarrierBytes + 128;
  return s->stages >= 2;
}

// Rows stream through a ring of shared-memory stages: the last warp copies the
// next rows of dy, h and dh (bulk copies) while the others work.  A group of
// `threads` threads takes a row of the stage: the sums that its means need,
// then its gradient, both from shared memory, the one beside the other of the
// row before, so one barrier a row is all that is waited for.  dx and dres may
// be dy or dh: a row's copies have landed before it is written.  Waits are
// bounded; after one that ran out (recorded in the status word) the results
// are unspecified.
template <class T, class W, int E, int MOST, int DH, bool DROP>
__global__ void __launch_bounds__(MOST + 32, 1)
    layer_norm_grad_staged_kernel(const LayerNormGradArgs a, const Operands<T> o,
                                  const Matrix<const W> weight, const Staging g) {
  using S = Slots<E, true>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~static_cast<uintptr_t>(127));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);  // full[stages], empty[stages]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 16);
  uint8_t* ring = smem + kBarrierBytes;
  __shared__ float2 sums[2][MOST / 32];  // by turns: one barrier a row is enough
  const tc::WaitCtx wc{abort_flag, &g_status};
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int workers = g.threads * g.groups, worker_warps = workers / 32;
  const int row_bytes = a.d * static_cast<int>(sizeof(T)), mats = DH == 1 ? 3 : 2;
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + 8 + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      tc::mbar_init(full(s), 1);              // the copy warp's arrival + bytes
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
  float dw[S::COUNT][8], db[S::COUNT][8];
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = db[i][k] = 0.0f;
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
    Dropout drop{};
    if (DROP) drop.init(a.dropout);
    Held<W, E, true> w;
    if (a.weight) w.load(weight, 0, a.d, tid, g.threads);
    else w.fill(1.0f);
    const int warps = g.threads / 32, first_warp = group * warps;
    const float per_d = 1.0f / static_cast<float>(a.d);
    auto stats_of = [&](int64_t row) {
      return row < a.rows ? RowStats{o.mean.load(row, 0), o.rstd.load(row, 0)}
                          : RowStats{0.0f, 0.0f};
    };
    auto values = [&](int n, int m) {  // matrix m of the group's row of stage n
      return reinterpret_cast<const T*>(ring + n % g.stages * g.stage_bytes) +
             (m * g.groups + group) * a.d;
    };
    // First sweep of the group's n-th row: its dweight and dbias and, for every
    // warp of the group, the sums of g and of g * xhat.
    auto first_sweep = [&](int n, bool live, const RowStats& r) {
      tc::wait_phase(full(n % g.stages), (n / g.stages) & 1u, wc);
      const T *dy = values(n, 0), *h = values(n, 1);
      float sum = 0.0f, dot = 0.0f;
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
          const float xhat = (vh[k] - r.mean) * r.rstd;
          dw[i][k] = fmaf(vy[k], xhat, dw[i][k]);
          db[i][k] += vy[k];
          const float grad = vy[k] * vw[k];
          sum += grad;
          dot = fmaf(grad, xhat, dot);
        }
      }
      sum = warp_sum(sum);
      dot = warp_sum(dot);
      if (lane == 0) sums[n & 1][warp] = make_float2(sum, dot);
    };
    auto meet = [&] {
      __syncwarp();  // lane 0 alone wrote or arrived last; bar.sync wants the warp converged
      if (warps > 1)
        asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(g.threads) : "memory");
    };
    RowStats r = stats_of(row_0 + group), r_next = stats_of(row_0 + step + group);
    if (row_0 < a.rows) first_sweep(0, row_0 + group < a.rows, r);
    meet();
    int n = 0;
    for (int64_t row0 = row_0; row0 < a.rows; row0 += step, ++n) {
      const int64_t row = row0 + group;
      const bool live = row < a.rows;  // the whole group
      const float2 s = lane < warps ? sums[n & 1][first_warp + lane] : make_float2(0.0f, 0.0f);
      const float mean_g = warp_sum(s.x) * per_d, mean_gx = warp_sum(s.y) * per_d;
      // The next row's first sweep runs beside this row's second.
      const RowStats r_after = stats_of(row + 2 * step);
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
          const float xhat = (vh[k] - r.mean) * r.rstd;
          const float v = grad_of(vy[k] * vw[k], xhat, mean_g, mean_gx, r.rstd);
          dx[k] = DH ? v + dx[k] : v;
        }
        if (DROP) {
          if (a.dres) store_step<T, true>(o.dres, row, c, dx);
          drop.apply8(static_cast<uint32_t>(row), c, dx);
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
  if (!a.dweight && !a.dbias) return;
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
          for (int k = 0; k < 8; ++k) {
            dw[i][k] += columns[c + k];
            db[i][k] += columns[a.d + c + k];
          }
        }
        if (turn == g.groups - 1) {
          if (a.dweight) store_step<float, true>(o.partial_w, blockIdx.x, c, dw[i]);
          if (a.dbias) store_step<float, true>(o.partial_b, blockIdx.x, c, db[i]);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            columns[c + k] = dw[i][k];
            columns[a.d + c + k] = db[i][k];
          }
        }
      }
    }
    if (g.groups > 1) __syncthreads();
  }
}

// Threads of an SM the register kernel is built for.
constexpr int kSmThreads = 512;
constexpr int ctas_per_sm(int threads) { return kSmThreads > threads ? kSmThreads / threads : 1; }

// A row held in the registers of THREADS threads, E values each; rows strided
// over the grid.  Up to 512 threads the next row's values are loaded before
// this row's reduction, so a barrier leaves loads in flight; 1024 have no
// registers for that.  Each thread reads its values of a row before it writes
// them, so dx and dres may be dy or dh.
template <class T, class W, int THREADS, int E, bool DH, bool DROP>
__global__ void __launch_bounds__(THREADS* rows_per_cta(THREADS),
                                  ctas_per_sm(THREADS* rows_per_cta(THREADS)))
    layer_norm_grad_kernel(const LayerNormGradArgs a, const Operands<T> o,
                           const Matrix<const W> weight) {
  using S = Slots<E, false>;
  constexpr int ROWS = rows_per_cta(THREADS), WARPS = THREADS / 32;
  constexpr bool AHEAD = THREADS <= 512;
  __shared__ float2 sums[2][WARPS];  // by turns, so one barrier a row is enough
  const int tid = threadIdx.x % THREADS, lane = threadIdx.x % 32, warp = tid / 32;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / THREADS;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * ROWS;
  struct Row {
    Held<T, E, false> dy, h, dh;
    RowStats r;
    __device__ __forceinline__ void load(const LayerNormGradArgs& a, const Operands<T>& o,
                                         int64_t row, int tid) {
      if (row >= a.rows) return;
      dy.load(o.dy, row, a.d, tid, THREADS);
      h.load(o.h, row, a.d, tid, THREADS);
      if (DH) dh.load(o.dh, row, a.d, tid, THREADS);
      r = RowStats{o.mean.load(row, 0), o.rstd.load(row, 0)};
    }
  };
  grid_launch_dependents();
  grid_wait();
  Dropout drop{};
  if (DROP) drop.init(a.dropout);
  Held<W, E, false> w;
  if (a.weight) w.load(weight, 0, a.d, tid, THREADS);
  else w.fill(1.0f);
  const float per_d = 1.0f / static_cast<float>(a.d);
  float dw[E], db[E];
#pragma unroll
  for (int i = 0; i < E; ++i) dw[i] = db[i] = 0.0f;
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
    float sum = 0.0f, dot = 0.0f;
    // Columns at or past d hold zeros of dy, but their h is not the mean.
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const float vy = to_f32(now.dy.item[i]), grad = vy * to_f32(w.item[i]);
      const float xhat = (to_f32(now.h.item[i]) - now.r.mean) * now.r.rstd;
      if (S::col(i, tid, THREADS) >= a.d) break;
      dw[i] = fmaf(vy, xhat, dw[i]);
      db[i] += vy;
      sum += grad;
      dot = fmaf(grad, xhat, dot);
    }
    __syncwarp();
    sum = warp_sum(sum);
    dot = warp_sum(dot);
    if constexpr (THREADS > 32) {
      if (lane == 0) sums[turn][warp] = make_float2(sum, dot);
      __syncthreads();
      const float2 s = lane < WARPS ? sums[turn][lane] : make_float2(0.0f, 0.0f);
      sum = warp_sum(s.x);
      dot = warp_sum(s.y);
    }
    const float mean_g = sum * per_d, mean_gx = dot * per_d;
    uint32_t words[E];
    if (DROP) drop.words_of_columns(static_cast<uint32_t>(row), tid, THREADS, words);
#pragma unroll
    for (int i = 0; i < E; ++i) {
      const int c = S::col(i, tid, THREADS);
      if (c >= a.d) break;
      const float xhat = (to_f32(now.h.item[i]) - now.r.mean) * now.r.rstd;
      const float grad = to_f32(now.dy.item[i]) * to_f32(w.item[i]);
      float v = grad_of(grad, xhat, mean_g, mean_gx, now.r.rstd);
      if (DH) v += to_f32(now.dh.item[i]);
      if (DROP) {
        if (a.dres) o.dres.store(row, c, v);
        v = drop.apply(v, words[i]);
      }
      o.dx.store(row, c, v);
    }
    __syncwarp();
  }
#pragma unroll
  for (int i = 0; i < E; ++i) {
    const int c = S::col(i, tid, THREADS);
    if (c >= a.d) break;
    if (a.dweight) o.partial_w.store(group, c, dw[i]);
    if (a.dbias) o.partial_b.store(group, c, db[i]);
  }
}

// dx and dres of a row too wide for registers, on one CTA: one sweep for the
// means, one for the gradient, each element read and then written by the same
// thread.
constexpr int kWideThreads = 512;

template <class T, class W, bool DROP>
__global__ void __launch_bounds__(kWideThreads)
    layer_norm_grad_wide_kernel(const LayerNormGradArgs a, const Operands<T> o,
                                const Matrix<const W> weight) {
  constexpr int N = 4;  // columns of a thread that share random words
  __shared__ float2 part[kWideThreads / 32];
  grid_launch_dependents();
  grid_wait();
  const int64_t row = blockIdx.x;
  Dropout drop{};
  if (DROP) drop.init(a.dropout);
  auto weight_at = [&](int c) { return a.weight ? weight.load(0, c) : 1.0f; };
  const float mean = o.mean.load(row, 0), r = o.rstd.load(row, 0);
  float sum = 0.0f, dot = 0.0f;
  for (int c = threadIdx.x; c < a.d; c += kWideThreads) {
    const float grad = o.dy.load(row, c) * weight_at(c);
    sum += grad;
    dot = fmaf(grad, (o.h.load(row, c) - mean) * r, dot);
  }
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  __syncwarp();
  sum = warp_sum(sum);
  dot = warp_sum(dot);
  if (lane == 0) part[warp] = make_float2(sum, dot);
  __syncthreads();
  const float2 s = lane < kWideThreads / 32 ? part[lane] : make_float2(0.0f, 0.0f);
  const float per_d = 1.0f / static_cast<float>(a.d);
  const float mean_g = warp_sum(s.x) * per_d, mean_gx = warp_sum(s.y) * per_d;
  for (int c0 = threadIdx.x; c0 - lane < a.d; c0 += N * kWideThreads) {
    uint32_t words[N];
    if (DROP) drop.words_of_columns(static_cast<uint32_t>(row), c0, kWideThreads, words);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = c0 + i * kWideThreads;
      if (c >= a.d) break;
      const float xhat = (o.h.load(row, c) - mean) * r;
      float v = grad_of(o.dy.load(row, c) * weight_at(c), xhat, mean_g, mean_gx, r);
      if (a.dh) v += o.dh.load(row, c);
      if (DROP) {
        if (a.dres) o.dres.store(row, c, v);
        v = drop.apply(v, words[i]);
      }
      o.dx.store(row, c, v);
    }
    __syncwarp();
  }
}

// dweight and dbias of wide rows: column sums of dy * xhat and of dy over one
// block of rows.  A CTA takes 32 columns, its 8 warps every eighth row of the
// block.
constexpr int kColumnWarps = 8;

template <class T>
__global__ void __launch_bounds__(32 * kColumnWarps)
    layer_norm_grad_columns_kernel(const LayerNormGradArgs a, const Operands<T> o,
                                   int64_t rows_per_block) {
  __shared__ float2 sums[kColumnWarps][32];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  const int64_t first = blockIdx.y * rows_per_block;
  const int64_t last = min(a.rows, first + rows_per_block);
  float2 s = make_float2(0.0f, 0.0f);
  if (c < a.d)
    for (int64_t i = first + warp; i < last; i += kColumnWarps) {
      const float dy = o.dy.load(i, c);
      s.x = fmaf(dy, (o.h.load(i, c) - o.mean.load(i, 0)) * o.rstd.load(i, 0), s.x);
      s.y += dy;
    }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < a.d) {
    s = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < kColumnWarps; ++w) {
      s.x += sums[w][lane].x;
      s.y += sums[w][lane].y;
    }
    if (a.dweight) o.partial_w.store(blockIdx.y, c, s.x);
    if (a.dbias) o.partial_b.store(blockIdx.y, c, s.y);
  }
}

// Whether every matrix of a call is read and written by 16-byte accesses.
bool vectored(const LayerNormGradArgs& a) {
  const int e = dtype_bytes(a.dtype);
  return a.d % 8 == 0 && rows_aligned(a.dy, a.lddy, e) && rows_aligned(a.h, a.ldh, e) &&
         rows_aligned(a.dh, a.dh ? a.lddh : 0, e) && rows_aligned(a.dx, a.lddx, e) &&
         rows_aligned(a.dres, a.dres ? a.lddres : 0, e) &&
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

Path path_of(const LayerNormGradArgs& a, int sms, Staging* g, int* parts) {
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

template <class T, class W, int DH, bool DROP>
const void* staged_kernel(int e) {
  // 32 values a thread never have dh in the ring.
  if constexpr (DH != 1)
    if (e == 32)
      return reinterpret_cast<const void*>(
          layer_norm_grad_staged_kernel<T, W, 32, 512, DH, DROP>);
  return reinterpret_cast<const void*>(layer_norm_grad_staged_kernel<T, W, 16, 512, DH, DROP>);
}

template <class T, class W, bool DROP>
cudaError_t launch(const LayerNormGradArgs& a, float* partial, int sms, cudaStream_t stream) {
  const int64_t n = a.rows;
  Staging g{};
  int parts = 0;
  const Path path = path_of(a, sms, &g, &parts);
  const int64_t sums = static_cast<int64_t>(parts) * a.d;
  float* const partial_b = a.dweight ? partial + sums : partial;
  const Operands<T> o{
      {static_cast<const T*>(a.dy), a.lddy, view_extent(n, a.d, a.lddy), a.bounds},
      {static_cast<const T*>(a.h), a.ldh, view_extent(n, a.d, a.ldh), a.bounds},
      {static_cast<const T*>(a.dh), a.lddh, view_extent(n, a.d, a.lddh), a.bounds},
      {static_cast<T*>(a.dx), a.lddx, view_extent(n, a.d, a.lddx), a.bounds},
      {static_cast<T*>(a.dres), a.lddres, view_extent(n, a.d, a.lddres), a.bounds},
      {a.mean, 1, n, a.bounds},
      {a.rstd, 1, n, a.bounds},
      {partial, a.d, sums, a.bounds},
      {partial_b, a.d, sums, a.bounds}};
  const Matrix<const W> weight{static_cast<const W*>(a.weight), 0, a.d, a.bounds};
  cudaError_t err = cudaSuccess;
  if (path == STAGED) {
    const void* kernel = g.dh == 0   ? staged_kernel<T, W, 0, DROP>(g.e)
                         : g.dh == 1 ? staged_kernel<T, W, 1, DROP>(g.e)
                                     : staged_kernel<T, W, 2, DROP>(g.e);
    static std::atomic<uint64_t> ready[6];  // by kernel: devices whose limit is set
    int dev = 0;
    err = cudaGetDevice(&dev);
    const uint64_t bit = uint64_t(1) << (dev & 63);
    std::atomic<uint64_t>& done = ready[g.dh + (g.e == 32 ? 3 : 0)];
    if (err == cudaSuccess && !(done.load(std::memory_order_acquire) & bit)) {
      err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kStagedBytes + kBarrierBytes + 128);
      if (err == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    }
    LayerNormGradArgs args = a;
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
      err = launch_dependent(a.dh ? layer_norm_grad_kernel<T, W, THREADS, E, true, DROP>
                                  : layer_norm_grad_kernel<T, W, THREADS, E, false, DROP>,
                             parts / ROWS, THREADS * ROWS, stream, a, o, weight);
    });
  } else {
    // The column sums come first: dx may overwrite dy.
    if (a.dweight || a.dbias)
      err = launch_dependent(layer_norm_grad_columns_kernel<T>, dim3((a.d + 31) / 32, parts),
                             32 * kColumnWarps, stream, a, o, (n + parts - 1) / parts);
    if (err == cudaSuccess && n > 0)
      err = launch_dependent(layer_norm_grad_wide_kernel<T, W, DROP>, static_cast<unsigned>(n),
                             kWideThreads, stream, a, o, weight);
  }
  if (err == cudaSuccess && a.dweight)
    err = launch_add_rows(partial, parts, a.d, a.dweight, a.bounds, stream);
  if (err == cudaSuccess && a.dbias)
    err = launch_add_rows(partial_b, parts, a.d, a.dbias, a.bounds, stream);
  return err;
}

template <class T>
cudaError_t launch_weight(const LayerNormGradArgs& a, float* partial, int sms,
                          cudaStream_t stream) {
  if (a.weight_f32)
    return a.drop ? launch<T, float, true>(a, partial, sms, stream)
                  : launch<T, float, false>(a, partial, sms, stream);
  return a.drop ? launch<T, T, true>(a, partial, sms, stream)
                : launch<T, T, false>(a, partial, sms, stream);
}

}  // namespace

int64_t layer_norm_grad_workspace(const LayerNormGradArgs& a, int sms) {
  Staging g{};
  int parts = 0;
  path_of(a, sms, &g, &parts);
  return static_cast<int64_t>(parts) * a.d * 4 * ((a.dweight != nullptr) + (a.dbias != nullptr));
}

cudaError_t layer_norm_grad_read_and_clear_status(unsigned int* status) {
  cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(unsigned int));
  if (e != cudaSuccess) return e;
  const unsigned int zero = 0;
  return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));
}

cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& a, void* workspace, int sms,
                                   cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  switch (a.dtype) {
    case DT_F16: return launch_weight<__half>(a, partial, sms, stream);
    case DT_BF16: return launch_weight<__nv_bfloat16>(a, partial, sms, stream);
    default: return launch_weight<float>(a, partial, sms, stream);
  }
}

}  // namespace mt
