// Gradient of the layer norm with dropout and the residual's addition: with
// xhat = (h - mean) * rstd, g = dy * weight,
//   dres = rstd * (g - mean(g) - xhat * mean(g * xhat)) + dh,   dx = D(dres),
//   dweight = sum over rows of dy * xhat,   dbias = sum over rows of dy.
// Bound by memory: dy, h, dh, dx and (with dropout) dres move once; a thread
// keeps its columns' shares of dweight and dbias in registers from row to row,
// and the CTAs' shares are added in a fixed order by a second kernel.  Rows
// that start on 16 bytes stream through shared memory
// (layer_norm_grad_staged_kernel), others through registers
// (layer_norm_grad_kernel).  Of rows too wide for either dy and h pass three times, once
// for the column sums where they are wanted (layer_norm_grad_columns_kernel) and twice
// for dx (layer_norm_grad_wide_kernel, the second time mostly from L2).  Arithmetic in
// pairs of values, one instruction each.
//
// Measured on GB300 (bf16 with dh, the required bytes' share of the copy rate): 16384 x
// 4096 100 us, 0.79, with dropout 141 us, 0.70; 16384 x 8192 194 us, 0.81; 4096 x 16384 200 us, 0.40
// (32 values a thread spill 150 bytes); fp32 8192 x 8192 206 us, 0.77; unaligned
// 16384 x 4095 127 us, 0.62.  Too wide: 4096 x 20000 221 us, 0.44 (150 us, 0.64 without
// column sums); 4096 x 20001 322 us, 0.30; unaligned past 8192, 4096 x 12001 206 us,
// 0.28; fp32 2048 x 13000 139 us, 0.45, 2048 x 16384 155 us, 0.51.
#pragma once

#include <algorithm>
#include <atomic>
#include <cstdint>

#include <cuda_runtime.h>

#include "model.h"
#include "pair_math.cuh"
#include "philox.cuh"
#include "row_chunk.cuh"
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

// What two elements of a row share.
struct RowPair {
  float2 mean, rstd;  // the mean's negative
  __device__ __forceinline__ explicit RowPair(const RowStats& r)
      : mean(both(-r.mean)), rstd(both(r.rstd)) {}
  __device__ __forceinline__ float2 xhat(float2 h) const { return mul2(add2(h, mean), rstd); }
};

// First sweep of eight elements: their share of dweight and dbias, and of the
// row's sums of g and of g * xhat.
__device__ __forceinline__ void accumulate8(const RowPair& r, const float (&dy)[8],
                                            const float (&h)[8], const float (&w)[8],
                                            float2 (&dw)[4], float2 (&db)[4], float2& sum,
                                            float2& dot) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 y = make_float2(dy[2 * k], dy[2 * k + 1]);
    const float2 x = r.xhat(make_float2(h[2 * k], h[2 * k + 1]));
    const float2 g = mul2(y, make_float2(w[2 * k], w[2 * k + 1]));
    dw[k] = fma2(y, x, dw[k]);
    db[k] = add2(db[k], y);
    sum = add2(sum, g);
    dot = fma2(g, x, dot);
  }
}

// Second sweep: v = rstd * (g - mean(g) - xhat * mean(g * xhat)) + v.
__device__ __forceinline__ void gradient8(const RowPair& r, float mean_g, float mean_gx,
                                          const float (&dy)[8], const float (&h)[8],
                                          const float (&w)[8], float (&v)[8]) {
  const float2 off = both(-mean_g), back = both(-mean_gx);
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float2 x = r.xhat(make_float2(h[2 * k], h[2 * k + 1]));
    const float2 g = mul2(make_float2(dy[2 * k], dy[2 * k + 1]),
                          make_float2(w[2 * k], w[2 * k + 1]));
    const float2 d = fma2(r.rstd, fma2(x, back, add2(g, off)), make_float2(v[2 * k], v[2 * k + 1]));
    v[2 * k] = d.x;
    v[2 * k + 1] = d.y;
  }
}

// How the staged kernel shares its threads out: `threads` take a row (at most
// e values each), `groups` rows make up a stage.
struct Staging {
  int threads, groups, e, most, stages;
  int dh;  // 0: none, 1: in the ring, 2: read where it is needed
  int word_bytes;  // dropout: the columns' part of the random words
  int stage_bytes, smem_bytes;
};
constexpr int kStagedBytes = 224 * 1024;
constexpr int kBarrierBytes = 256;

// Rows of up to 16384 values: 512 threads of 16 values, or of 32 past 8192: 16
// warps, which leaves 128 registers a thread (a 17th warp would leave 96, and
// spills).  false when two stages do not fit.
bool staging_of(int d, int elem, bool dh, bool drop, Staging* s) {
  if (d > 16384) return false;
  s->word_bytes = drop ? 4 * d : 0;
  const int ring = (drop ? kStagedBytes : 200 * 1024) - s->word_bytes;
  s->most = 512;
  s->e = d <= 16 * 512 ? 16 : 32;
  s->threads = (d + 32 * s->e - 1) / (32 * s->e) * 32;
  const int row_bytes = d * elem;
  // dh stays out of the ring where three stages of a row would not fit, and
  // where a thread has 32 values.
  s->dh = !dh ? 0 : s->e == 16 && 9 * row_bytes <= ring ? 1 : 2;
  const int mats = s->dh == 1 ? 3 : 2, rows = ring / (3 * mats * row_bytes);
  s->groups = s->most / s->threads;
  if (s->threads > 32) s->groups = std::min(s->groups, 15);  // named barriers
  s->groups = std::max(1, std::min(s->groups, rows));
  s->stage_bytes = s->groups * mats * row_bytes;
  s->stages = std::min(8, ring / s->stage_bytes);
  // The column sums of the groups meet in the ring.
  s->smem_bytes =
      s->word_bytes + std::max(s->stages * s->stage_bytes, 2 * d * 4) + kBarrierBytes + 128;
  return s->stages >= 2;
}

// Rows stream through a ring of shared-memory stages, which the first warp
// fills (bulk copies of dy, h and dh) as the rows in them are done with: the
// stage of the row before is filled again while this row is worked on.  A group of
// `threads` threads takes a row of the stage: the sums that its means need,
// then its gradient, both from shared memory, the one beside the other of the
// row before, so one barrier a row is all that is waited for.  dx and dres may
// be dy or dh: a row's copies have landed before it is written.  Waits are
// bounded; after one that ran out (recorded in the status word) the results
// are unspecified.
template <class T, class W, int E, int MOST, int DH, bool DROP>
__global__ void __launch_bounds__(MOST, 1)
    layer_norm_grad_staged_kernel(const LayerNormGradArgs a, const Operands<T> o,
                                  const Matrix<const W> weight, const Staging g) {
  using S = Slots<E, true>;
  extern __shared__ __align__(128) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);  // full[stages], empty[stages]
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 16);
  Dropout::Columns* const words = reinterpret_cast<Dropout::Columns*>(smem + kBarrierBytes);
  uint8_t* const ring = smem + kBarrierBytes + g.word_bytes;
  __shared__ float sums[2][2][MOST / 32];  // by turns: one barrier a row is enough
  const tc::WaitCtx wc{abort_flag, &g_status};
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int worker_warps = g.threads * g.groups / 32;
  const int row_bytes = a.d * static_cast<int>(sizeof(T)), mats = DH == 1 ? 3 : 2;
  const int mat_bytes = g.groups * row_bytes;
  auto full = [&](int s) { return smem_u32(bars + s); };
  auto empty = [&](int s) { return smem_u32(bars + 8 + s); };
  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      tc::mbar_init(full(s), 1);              // the first warp's arrival + bytes
      tc::mbar_init(empty(s), worker_warps);  // every warp
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  grid_launch_dependents();
  grid_wait();
  Dropout drop{};
  if (DROP) {
    drop.init(a.dropout);
    for (int i = threadIdx.x; i < a.d / 4; i += static_cast<int>(blockDim.x))
      words[i] = drop.columns(static_cast<uint32_t>(i));
    __syncthreads();
  }

  // A stage of the ring and how often it has gone round, mod 2.
  struct Turn {
    int slot = 0;
    uint32_t phase = 0;
    __device__ __forceinline__ void next(int stages) {
      if (++slot == stages) slot = 0, phase ^= 1u;
    }
  };
  const int64_t step = static_cast<int64_t>(gridDim.x) * g.groups;
  const int64_t row_0 = static_cast<int64_t>(blockIdx.x) * g.groups;
  const int group = static_cast<int>(threadIdx.x) / g.threads;
  const int tid = static_cast<int>(threadIdx.x) % g.threads;
  int issued = 0;
  Turn fill;
  // The copies of the CTA's next rows, by its first warp.
  auto issue = [&] {
    const int64_t row0 = row_0 + issued * step;
    if (row0 >= a.rows || a.fault_inject) return;
    const int s = fill.slot;
    if (issued >= g.stages &&
        !__all_sync(0xffffffffu, tc::wait_phase(empty(s), fill.phase ^ 1u, wc)))
      return;
    const int rows = static_cast<int>(min(static_cast<int64_t>(g.groups), a.rows - row0));
    if (lane == 0) tc::mbar_arrive_expect_tx(full(s), rows * mats * row_bytes);
    __syncwarp();
    // A matrix without gaps between its rows arrives in one copy.
    for (int m = 0; m < mats; ++m) {
      const Matrix<const T>& from = m == 0 ? o.dy : m == 1 ? o.h : o.dh;
      const bool packed = from.ld == a.d;
      for (int i = lane; i < (packed ? 1 : rows); i += 32)
        tc::bulk_copy_g2s(smem_u32(ring + s * g.stage_bytes + m * mat_bytes + i * row_bytes),
                          from.p + (row0 + i) * from.ld, packed ? rows * row_bytes : row_bytes,
                          full(s));
    }
    __syncwarp();
    ++issued;
    fill.next(g.stages);
  };
  if (warp == 0)
    for (int i = 0; i < g.stages; ++i) issue();

  // The weight: as it is used where registers allow, else as it is stored.
  constexpr bool WIDE_W = E <= 16;
  float wide_w[WIDE_W ? S::COUNT : 1][8];
  Held<W, E, true> stored_w;
  if (a.weight) stored_w.load(weight, 0, a.d, tid, g.threads);
  else stored_w.fill(1.0f);
  if constexpr (WIDE_W) {
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) stored_w.get(i, wide_w[i]);
  }
  auto weight_of = [&](int i, float(&v)[8]) {
    if constexpr (WIDE_W) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = wide_w[i][k];
    } else {
      stored_w.get(i, v);
    }
  };
  float2 dw[S::COUNT][4], db[S::COUNT][4];
#pragma unroll
  for (int i = 0; i < S::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[i][k] = db[i][k] = both(0.0f);

  const int warps = g.threads / 32, first_warp = group * warps;
  const float per_d = 1.0f / static_cast<float>(a.d);
  auto stats_of = [&](int64_t row) {
    return row < a.rows ? RowStats{o.mean.load(row, 0), o.rstd.load(row, 0)}
                        : RowStats{0.0f, 0.0f};
  };
  // This thread's first value of the group's row in a stage, and chunk i of
  // matrix m from there.
  auto stage = [&](int slot) {
    return ring + slot * g.stage_bytes + group * row_bytes + tid * 8 * static_cast<int>(sizeof(T));
  };
  const int chunk_bytes = g.threads * 8 * static_cast<int>(sizeof(T));
  auto get = [&](const uint8_t* at, int m, int i, float(&v)[8]) {
    reinterpret_cast<const Pack8<T>*>(at + m * mat_bytes + i * chunk_bytes)->get(v);
  };
  // First sweep of the group's next row: its dweight and dbias and, for every
  // warp of the group, the sums of g and of g * xhat.  After the first exchange
  // even lanes add up the one, odd lanes the other.
  auto first_sweep = [&](const Turn& at, int turn, bool live, const RowStats& r) {
    tc::wait_phase(full(at.slot), at.phase, wc);
    const uint8_t* const from = stage(at.slot);
    const RowPair p(r);
    float2 sum2 = both(0.0f), dot2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) {
      if (!live || S::col(i, tid, g.threads) >= a.d) break;
      float vy[8], vh[8], vw[8];
      get(from, 0, i, vy);
      get(from, 1, i, vh);
      weight_of(i, vw);
      accumulate8(p, vy, vh, vw, dw[i], db[i], sum2, dot2);
    }
    __syncwarp();
    const float sum = sum2.x + sum2.y, dot = dot2.x + dot2.y;
    const bool odd = lane & 1;
    float t = (odd ? dot : sum) + __shfl_xor_sync(0xffffffffu, odd ? sum : dot, 1);
#pragma unroll
    for (int off = 2; off < 32; off *= 2) t += __shfl_xor_sync(0xffffffffu, t, off);
    if (lane < 2) sums[turn][lane][warp] = t;
  };
  auto meet = [&] {
    __syncwarp();  // some lanes wrote or arrived last; bar.sync wants the warp converged
    if (warps > 1)
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(g.threads) : "memory");
  };
  RowStats r = stats_of(row_0 + group), r_next = stats_of(row_0 + step + group);
  Turn now, next;
  if (row_0 < a.rows) first_sweep(now, 0, row_0 + group < a.rows, r);
  meet();
  int turn = 0;
  for (int64_t row0 = row_0; row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + group;
    const bool live = row < a.rows;  // the whole group
    // The warps' sums: lanes 0 .. 15 add up the one, 16 .. 31 the other.
    static_assert(MOST / 32 <= 16, "half a warp for each sum");
    const int w = lane & 15;
    float t = w < warps ? sums[turn][lane / 16][first_warp + w] : 0.0f;
#pragma unroll
    for (int off = 1; off < 16; off *= 2) t += __shfl_xor_sync(0xffffffffu, t, off);
    const float mean_g = __shfl_sync(0xffffffffu, t, 0) * per_d;
    const float mean_gx = __shfl_sync(0xffffffffu, t, 16) * per_d;
    if (warp == 0 && row0 > row_0) issue();
    // The next row's first sweep runs beside this row's second.
    const RowStats r_after = stats_of(row + 2 * step);
    next.next(g.stages);
    if (row0 + step < a.rows) first_sweep(next, turn ^ 1, row + step < a.rows, r_next);
    const uint8_t* const from = stage(now.slot);
    const RowPair p(r);
    const Dropout::Row of_row = DROP ? drop.row(static_cast<uint32_t>(row)) : Dropout::Row{};
#pragma unroll
    for (int i = 0; i < S::COUNT; ++i) {
      const int c = S::col(i, tid, g.threads);
      if (!live || c >= a.d) break;
      float vy[8], vh[8], vw[8], dx[8];
      get(from, 0, i, vy);
      get(from, 1, i, vh);
      weight_of(i, vw);
      if (DH == 0) {
#pragma unroll
        for (int k = 0; k < 8; ++k) dx[k] = 0.0f;
      }
      if (DH == 1) get(from, 2, i, dx);
      if (DH == 2) reinterpret_cast<const Pack8<T>*>(o.dh.p + row * o.dh.ld + c)->get(dx);
      gradient8(p, mean_g, mean_gx, vy, vh, vw, dx);
      if (DROP) {
        if (a.dres) store_step<T, true>(o.dres, row, c, dx);
        drop.apply4(of_row, words[c / 4], dx);
        drop.apply4(of_row, words[c / 4 + 1], dx + 4);
      }
      store_step<T, true>(o.dx, row, c, dx);
    }
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(empty(now.slot));
    now.next(g.stages);
    r = r_next;
    r_next = r_after;
    meet();
  }
  __syncthreads();
  if (warp == 0 && *abort_flag) {
    // After a wait that ran out: let the copies issued land before the CTA
    // exits.
    for (int i = issued > g.stages ? issued - g.stages : 0; i < issued; ++i)
      tc::wait_phase(full(i % g.stages), (i / g.stages) & 1u, wc, false);
  }
  if (!a.dweight && !a.dbias) return;
  // The groups' column sums, in group order; the ring is idle.
  float* columns = reinterpret_cast<float*>(ring);
  for (int turn = 0; turn < g.groups; ++turn) {
    if (group == turn) {
#pragma unroll
      for (int i = 0; i < S::COUNT; ++i) {
        const int c = S::col(i, tid, g.threads);
        if (c >= a.d) break;
        float vw[8], vb[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          vw[k] = k % 2 ? dw[i][k / 2].y : dw[i][k / 2].x;
          vb[k] = k % 2 ? db[i][k / 2].y : db[i][k / 2].x;
          if (turn > 0) {
            vw[k] += columns[c + k];
            vb[k] += columns[a.d + c + k];
          }
        }
        if (turn == g.groups - 1) {
          if (a.dweight) store_step<float, true>(o.partial_w, blockIdx.x, c, vw);
          if (a.dbias) store_step<float, true>(o.partial_b, blockIdx.x, c, vb);
        } else {
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            columns[c + k] = vw[k];
            columns[a.d + c + k] = vb[k];
          }
        }
      }
    }
    if (g.groups > 1) __syncthreads();
  }
}

// Threads of an SM the register kernel is built for, and CTAs of that many.
constexpr int kSmThreads = 512;
constexpr int ctas_per_sm(int threads) { return kSmThreads / threads; }

// Calls f(threads per row, values per thread) with the register kernel's
// layout for rows of d values; false past 8192.
template <class F>
bool held_layout(int d, F&& f) {
  using std::integral_constant;
  auto go = [&](auto threads, auto values) { f(threads, values); return true; };
  if (d <= 256) return go(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  if (d <= 512) return go(integral_constant<int, 64>{}, integral_constant<int, 8>{});
  if (d <= 1024) return go(integral_constant<int, 128>{}, integral_constant<int, 8>{});
  if (d <= 2048) return go(integral_constant<int, 256>{}, integral_constant<int, 8>{});
  if (d <= 4096) return go(integral_constant<int, 512>{}, integral_constant<int, 8>{});
  if (d <= 8192) return go(integral_constant<int, 512>{}, integral_constant<int, 16>{});
  return false;
}

// A row held in the registers of THREADS threads, E values each, an element an
// access; rows strided over the grid.  With eight values a thread the next
// row's are loaded before this row's reduction, so a barrier leaves loads in
// flight; 16 leave no registers for that.  Each thread reads its values of a row
// before it writes them, so dx and dres may be dy or dh.
template <class T, class W, int THREADS, int E, bool DH, bool DROP>
__global__ void __launch_bounds__(THREADS* rows_per_cta(THREADS),
                                  ctas_per_sm(THREADS* rows_per_cta(THREADS)))
    layer_norm_grad_kernel(const LayerNormGradArgs a, const Operands<T> o,
                           const Matrix<const W> weight) {
  using C = Chunks<T, E, false, THREADS>;
  using At = Chunk<false, THREADS>;
  constexpr int ROWS = rows_per_cta(THREADS), WARPS = THREADS / 32;
  constexpr bool AHEAD = E == 8;
  __shared__ float2 sums[2][WARPS];  // by turns, so one barrier a row is enough
  const int tid = threadIdx.x % THREADS, lane = threadIdx.x % 32, warp = tid / 32;
  const int64_t group = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / THREADS;
  const int64_t groups = static_cast<int64_t>(gridDim.x) * ROWS;
  struct Row {
    C dy, h, dh;
    RowStats r;
    __device__ __forceinline__ void load(const LayerNormGradArgs& a, const Operands<T>& o,
                                         int64_t row, int tid) {
      if (row >= a.rows) return;
      dy.load(o.dy, row, a.d, tid);
      h.load(o.h, row, a.d, tid);
      if (DH) dh.load(o.dh, row, a.d, tid);
      r = RowStats{o.mean.load(row, 0), o.rstd.load(row, 0)};
    }
  };
  grid_launch_dependents();
  grid_wait();
  Dropout drop{};
  if (DROP) drop.init(a.dropout);
  Chunks<W, E, false, THREADS> w;
  if (a.weight) w.load(weight, 0, a.d, tid);
  else w.fill(1.0f);
  const float per_d = 1.0f / static_cast<float>(a.d);
  float2 dw[C::COUNT][4], db[C::COUNT][4];
#pragma unroll
  for (int i = 0; i < C::COUNT; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) dw[i][k] = db[i][k] = both(0.0f);
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
    const RowPair p(now.r);
    // Columns at or past d hold zeros of dy, so they add nothing to any sum.
    float2 sum2 = both(0.0f), dot2 = both(0.0f);
#pragma unroll
    for (int i = 0; i < C::COUNT; ++i) {
      float vy[8], vh[8], vw[8];
      now.dy.get(i, vy);
      now.h.get(i, vh);
      w.get(i, vw);
      accumulate8(p, vy, vh, vw, dw[i], db[i], sum2, dot2);
    }
    float sum = warp_sum(sum2.x + sum2.y), dot = warp_sum(dot2.x + dot2.y);
    if constexpr (THREADS > 32) {
      if (lane == 0) sums[turn][warp] = make_float2(sum, dot);
      __syncthreads();
      const float2 s = lane < WARPS ? sums[turn][lane] : make_float2(0.0f, 0.0f);
      sum = warp_sum(s.x);
      dot = warp_sum(s.y);
    }
    const float mean_g = sum * per_d, mean_gx = dot * per_d;
    const Dropout::Row of_row = DROP ? drop.row(static_cast<uint32_t>(row)) : Dropout::Row{};
#pragma unroll
    for (int i = 0; i < C::COUNT; ++i) {
      const At at(i, tid);
      float vy[8], vh[8], vw[8], v[8];
      now.dy.get(i, vy);
      now.h.get(i, vh);
      w.get(i, vw);
      if (DH) {
        now.dh.get(i, v);
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = 0.0f;
      }
      gradient8(p, mean_g, mean_gx, vy, vh, vw, v);
      if (DROP) {
        if (a.dres) at.store(o.dres, row, a.d, v);
        __syncwarp();
        at.drop(drop, of_row, at.words(drop), v);
      }
      at.store(o.dx, row, a.d, v);
    }
  }
#pragma unroll
  for (int i = 0; i < C::COUNT; ++i) {
    const At at(i, tid);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (!at.live(k, a.d)) break;
      if (a.dweight)
        o.partial_w.store(group, at.col(k), k % 2 ? dw[i][k / 2].y : dw[i][k / 2].x);
      if (a.dbias) o.partial_b.store(group, at.col(k), k % 2 ? db[i][k / 2].y : db[i][k / 2].x);
    }
  }
}

// dx and dres of a row too wide for registers, on one CTA: one sweep for the
// means, one for the gradient, each element read and then written by the same
// thread.
constexpr int kWideThreads = 512;

template <class T, class W, bool DROP, bool ALIGNED>
__global__ void __launch_bounds__(kWideThreads)
    layer_norm_grad_wide_kernel(const LayerNormGradArgs a, const Operands<T> o,
                                const Matrix<const W> weight) {
  using At = Chunk<ALIGNED, kWideThreads>;
  __shared__ float2 part[kWideThreads / 32];
  grid_launch_dependents();
  grid_wait();
  const int64_t row = blockIdx.x;
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  Dropout drop{};
  Dropout::Row of_row{};
  if (DROP) {
    drop.init(a.dropout);
    of_row = drop.row(static_cast<uint32_t>(row));
  }
  const RowPair p(RowStats{o.mean.load(row, 0), o.rstd.load(row, 0)});
  // Calls f(chunk, dy, h, weight) for this thread's chunks, all warps as many times.
  auto sweep = [&](auto&& f) {
    for (int i = 0; i * 8 * kWideThreads < a.d; ++i) {
      const At at(i, threadIdx.x);
      const auto y = at.load(o.dy, row, a.d), h = at.load(o.h, row, a.d);
      float vy[8], vh[8], vw[8];
      if (a.weight) at.load(weight, 0, a.d).get(vw);
      y.get(vy);
      h.get(vh);
      if (!a.weight) {
#pragma unroll
        for (int k = 0; k < 8; ++k) vw[k] = 1.0f;
      }
      f(at, vy, vh, vw);
    }
  };
  float2 sum2 = both(0.0f), dot2 = both(0.0f);
  sweep([&](const At&, const float(&y)[8], const float(&h)[8], const float(&w)[8]) {
    float2 dw[4] = {}, db[4] = {};  // not wanted here
    accumulate8(p, y, h, w, dw, db, sum2, dot2);
  });
  __syncwarp();
  const float2 mine = make_float2(warp_sum(sum2.x + sum2.y), warp_sum(dot2.x + dot2.y));
  if (lane == 0) part[warp] = mine;
  __syncthreads();
  const float2 s = lane < kWideThreads / 32 ? part[lane] : make_float2(0.0f, 0.0f);
  const float per_d = 1.0f / static_cast<float>(a.d);
  const float mean_g = warp_sum(s.x) * per_d, mean_gx = warp_sum(s.y) * per_d;
  sweep([&](const At& at, const float(&y)[8], const float(&h)[8], const float(&w)[8]) {
    Eight<T, ALIGNED> add{};
    if (a.dh) add = at.load(o.dh, row, a.d);
    float v[8];
    add.get(v);
    gradient8(p, mean_g, mean_gx, y, h, w, v);
    if (DROP) {
      if (a.dres) at.store(o.dres, row, a.d, v);
      __syncwarp();
      at.drop(drop, of_row, at.words(drop), v);
    }
    at.store(o.dx, row, a.d, v);
  });
}

// dweight and dbias of wide rows: column sums of dy * xhat and of dy over one
// block of rows.  A CTA takes a strip of 256 columns, eight a lane, its 8 warps
// every eighth row of the block.
constexpr int kColumnWarps = 8, kStrip = 256;

template <class T, bool ALIGNED>
__global__ void __launch_bounds__(32 * kColumnWarps)
    layer_norm_grad_columns_kernel(const LayerNormGradArgs a, const Operands<T> o,
                                   int64_t rows_per_block) {
  __shared__ float2 sums[kColumnWarps][kStrip];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const Chunk<ALIGNED, 32> at(blockIdx.x, lane);
  const int64_t first = blockIdx.y * rows_per_block;
  const int64_t last = min(a.rows, first + rows_per_block);
  const float ones[8] = {1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f, 1.0f};
  float2 dw[4], db[4], sum2 = both(0.0f), dot2 = both(0.0f);
#pragma unroll
  for (int k = 0; k < 4; ++k) dw[k] = db[k] = both(0.0f);
#pragma unroll 2
  for (int64_t i = first + warp; i < last; i += kColumnWarps) {
    float y[8], h[8];
    at.load(o.dy, i, a.d).get(y);
    at.load(o.h, i, a.d).get(h);
    const RowPair p(RowStats{o.mean.load(i, 0), o.rstd.load(i, 0)});
    accumulate8(p, y, h, ones, dw, db, sum2, dot2);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k)
    sums[warp][k * 32 + lane] = k % 2 ? make_float2(dw[k / 2].y, db[k / 2].y)
                                      : make_float2(dw[k / 2].x, db[k / 2].x);
  __syncthreads();
  static_assert(32 * kColumnWarps == kStrip, "a thread per column: value `warp` of its lane");
  if (!at.live(warp, a.d)) return;
  float2 s = both(0.0f);
#pragma unroll
  for (int w = 0; w < kColumnWarps; ++w) s = add2(s, sums[w][threadIdx.x]);
  if (a.dweight) o.partial_w.store(blockIdx.y, at.col(warp), s.x);
  if (a.dbias) o.partial_b.store(blockIdx.y, at.col(warp), s.y);
}

// Adds the partial rows of both gradients in order: a CTA takes 32 columns of
// one (blockIdx.y), its 32 warps every 32nd row.
struct Sums {
  Matrix<const float> rows;
  Matrix<float> out;
};
__global__ void __launch_bounds__(1024)
    layer_norm_grad_sums_kernel(const Sums first, const Sums second, int count, int cols) {
  __shared__ float sums[32][33];
  grid_launch_dependents();
  grid_wait();
  const Sums& s = blockIdx.y ? second : first;
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int c = blockIdx.x * 32 + lane;
  float t = 0.0f;
  if (c < cols)
    for (int i = warp; i < count; i += 32) t += s.rows.load(i, c);
  sums[warp][lane] = t;
  __syncthreads();
  // Warp w adds the 32 sums of column w.
  t = warp_sum(sums[lane][warp]);
  const int cw = blockIdx.x * 32 + warp;
  if (lane == 0 && cw < cols) s.out.store(0, cw, t);
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

// Blocks of rows of the wide column sums: enough CTAs for two waves of eight
// on each SM, at least 32 rows each.
int column_blocks(int64_t rows, int cols, int sms) {
  const int64_t strips = (cols + kStrip - 1) / kStrip;
  const int64_t want = std::max<int64_t>(1, 16 * static_cast<int64_t>(sms) / strips);
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(want, (rows + 31) / 32)));
}

// Which kernel a call takes, and the partial rows of dweight it writes.
enum Path { STAGED, HELD, WIDE };

Path path_of(const LayerNormGradArgs& a, int sms, Staging* g, int* parts) {
  const int e = dtype_bytes(a.dtype);
  if (vectored(a) && staging_of(a.d, e, a.dh != nullptr, a.drop != 0, g)) {
    *parts = ctas_of(a.rows, g->groups, 1, sms);
    return STAGED;
  }
  const bool held = held_layout(a.d, [&](auto threads, auto) {
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
      err = launch_dependent(kernel, static_cast<unsigned>(parts), g.threads * g.groups,
                             g.smem_bytes, 1, stream, list);
  } else if (path == HELD) {
    held_layout(a.d, [&](auto threads, auto values) {
      constexpr int THREADS = decltype(threads)::value, E = decltype(values)::value;
      constexpr int ROWS = rows_per_cta(THREADS);
      err = launch_dependent(a.dh ? layer_norm_grad_kernel<T, W, THREADS, E, true, DROP>
                                  : layer_norm_grad_kernel<T, W, THREADS, E, false, DROP>,
                             parts / ROWS, THREADS * ROWS, stream, a, o, weight);
    });
  } else {
    // The column sums come first: dx may overwrite dy.
    const bool aligned = vectored(a);
    if (a.dweight || a.dbias)
      err = launch_dependent(aligned ? layer_norm_grad_columns_kernel<T, true>
                                     : layer_norm_grad_columns_kernel<T, false>,
                             dim3((a.d + kStrip - 1) / kStrip, parts), 32 * kColumnWarps, stream,
                             a, o, (n + parts - 1) / parts);
    if (err == cudaSuccess && n > 0)
      err = launch_dependent(aligned ? layer_norm_grad_wide_kernel<T, W, DROP, true>
                                     : layer_norm_grad_wide_kernel<T, W, DROP, false>,
                             static_cast<unsigned>(n), kWideThreads, stream, a, o, weight);
  }
  if (err != cudaSuccess || (!a.dweight && !a.dbias)) return err;
  const Sums w{{partial, a.d, sums, a.bounds}, {a.dweight, a.d, a.d, a.bounds}};
  const Sums b{{partial_b, a.d, sums, a.bounds}, {a.dbias, a.d, a.d, a.bounds}};
  return launch_dependent(layer_norm_grad_sums_kernel,
                          dim3((a.d + 31) / 32, a.dweight && a.dbias ? 2 : 1), 1024, stream,
                          a.dweight ? w : b, b, parts, a.d);
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

// One storage type's part (layer_norm_grad_<type>.cu): the call, and its status
// word read and cleared.
#define MT_LAYER_NORM_GRAD_TYPE(NAME, T)                                                     \
  cudaError_t launch_layer_norm_grad_##NAME(const LayerNormGradArgs& a, float* partial,      \
                                            int sms, cudaStream_t stream) {                  \
    return launch_weight<T>(a, partial, sms, stream);                                        \
  }                                                                                          \
  cudaError_t layer_norm_grad_##NAME##_read_and_clear_status(unsigned int* status) {         \
    cudaError_t e = cudaMemcpyFromSymbol(status, g_status, sizeof(unsigned int));            \
    if (e != cudaSuccess) return e;                                                          \
    const unsigned int zero = 0;                                                             \
    return cudaMemcpyToSymbol(g_status, &zero, sizeof(unsigned int));                        \
  }

}  // namespace mt
