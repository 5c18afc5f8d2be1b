// What the vocabulary loss does with its logits: the forward pass's softmax
// statistics (HeadStats) and the gradient's D (HeadGrad), as epilogues of the
// fused products' kernels.  Logits exist in tensor memory and registers alone.
//
// Large batches (CTA pairs) put the tokens on tensor memory's lanes: a thread
// then holds one token and walks over 128 columns of the vocabulary, so the
// statistics need no exchange between lanes, and D is stored as 16-byte pieces
// of its rows.  Few tokens (split kernel) put the weight's columns on the
// lanes, as the linear layer does: there the weight's stream is all that
// counts, and the statistics of 16 tokens meet over a warp's lanes.
#pragma once

#include <cstdint>
#include <type_traits>

#include <cuda_runtime.h>

#include "device_util.cuh"
#include "gemm_f16.cuh"
#include "layers.h"
#include "linear.cuh"
#include "row_util.cuh"

namespace mt {
namespace head {

using linear::FINISH_ROWS;
using linear::Rows;

constexpr float LOG2E = 1.4426950408889634f;
constexpr int LANE_SLOT = 32;    // columns of the vocabulary behind one entry of `parts`:
constexpr int PAIR_SLOT = 128;   // a warp's lanes, or half a pair's tile

// 2^x on the special-function unit (2^-22 of the result; what would be
// subnormal is 0).
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Some logits' part of a softmax, in base 2: top = max(z) * log2(e), rounded
// once and then taken as it is, and sum of 2^(z * log2(e) - top), each exponent
// rounded once.  Joining parts of one top multiplies by exactly 1, so parts
// without number may be joined.  No logits: -inf and 0.
struct Softmax {
  float top, sum;

  // What exponents are taken against: top, or 0 where there is none.
  static __device__ __forceinline__ float base(float top) {
    return top == -INFINITY ? 0.0f : top;
  }
  __device__ __forceinline__ void join(const Softmax& o) {
    const float t = fmaxf(top, o.top), b = base(t);
    sum = sum * exp2_approx(top - b) + o.sum * exp2_approx(o.top - b);
    top = t;
  }
};

// Token t's logits of slot s of the vocabulary leave parts[s * T + t] and,
// where wanted, their plain sum in sums[s * T + t]; the logit of its target
// goes to target_logit[t].
struct HeadStats {
  int T, C;
  const int64_t* target;
  float2* parts;
  float* sums;  // nullptr: not wanted
  float* target_logit;
  int64_t slots;
  BoundsRecord* bounds;

  __device__ __forceinline__ void store(int slot, int t, const Softmax& s, float sum) const {
    const int64_t at = static_cast<int64_t>(slot) * T + t;
    if (!bounds_ok(bounds, SITE_PARTIAL, at, 1, slots * T)) return;
    parts[at] = make_float2(s.top, s.sum);
    if (sums) sums[at] = sum;
  }
  // The target of token t as a column (negative: none).
  __device__ __forceinline__ int target_of(int t) const {
    if (t >= T || !bounds_ok(bounds, SITE_ROWS, t, 1, T)) return -1;
    const int64_t v = target[t];
    return v >= 0 && v < C ? static_cast<int>(v) : -1;
  }
  __device__ __forceinline__ void store_target(int t, float z) const {
    if (bounds_ok(bounds, SITE_ROWS, t, 1, T)) target_logit[t] = z;
  }
};

// A token's factors of D: D = exp2(z * log2(e) - x) * p - all - (its target: hit).
struct __align__(16) HeadRow {
  static constexpr int DEAD = -2;  // no target: a row of zeros

  float x, p, all, hit;
  int target;  // column of the vocabulary; -1: outside it, and the factors are NaN
};

// What they are made of.
struct HeadSource {
  const float* dloss;
  const float* lse;
  const int64_t* target;
  int64_t ignore_index;
  float smoothing, z_loss;
  int V;

  __device__ __forceinline__ HeadRow row(int64_t t, float scale) const {
    const int64_t column = target[t];
    HeadRow r{0.0f, 0.0f, 0.0f, 0.0f, HeadRow::DEAD};
    if (column != ignore_index) {
      const bool inside = column >= 0 && column < V;
      const float l = lse[t], g = inside ? dloss[t] * scale : NAN;
      r.x = l * LOG2E;
      r.p = g * (1.0f + 2.0f * z_loss * l);
      r.all = g * (smoothing / static_cast<float>(V));
      r.hit = g * (1.0f - smoothing);
      r.target = inside ? static_cast<int>(column) : -1;
    }
    return r;
  }
};

// D of columns first .. first + C - 1 of the vocabulary, to a T x C matrix of
// rows of ldd 16-bit values, or to boxes of 64 columns x 32 rows of its map.
struct HeadGrad {
  CUtensorMap map;
  int T, C;
  const HeadRow* rows;  // with fp16's scale; null: from the source
  HeadSource source;
  int first;
  void* D;
  int64_t ldd;
  int dtype;
  BoundsRecord* bounds;

  // Token t's factors, those of no target where there is no such token.
  __device__ __forceinline__ HeadRow row(int t, int end) const {
    if (t >= end || !bounds_ok(bounds, SITE_ROWS, t, 1, T))
      return HeadRow{0.0f, 0.0f, 0.0f, 0.0f, HeadRow::DEAD};
    return rows ? rows[t] : source.row(t, 1.0f);
  }
};

// --- few tokens: the weight's columns on the lanes ----------------------------

struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// Reduces FINISH_ROWS values over the lanes: lanes 2 r and 2 r + 1 get row
// r's.  Each step halves the rows a lane still holds.
template <class Op>
__device__ __forceinline__ float over_lanes(const Rows& v, Op op) {
  static_assert(FINISH_ROWS == 16, "four halvings");
  const int lane = threadIdx.x % 32;
  float a[FINISH_ROWS];
#pragma unroll
  for (int i = 0; i < FINISH_ROWS; ++i) a[i] = v[i];
#pragma unroll
  for (int n = 8, off = 16; n > 0; n /= 2, off /= 2) {
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float give = upper ? a[i] : a[i + n], keep = upper ? a[i + n] : a[i];
      a[i] = op(keep, __shfl_xor_sync(0xffffffffu, give, off));
    }
  }
  return op(a[0], __shfl_xor_sync(0xffffffffu, a[0], 1));
}

// Column c's logits of tokens t_begin .. t_end - 1, the whole warp together
// (c: 32 neighbouring columns, those at or past e.C are none).
template <class Sums>
__device__ __forceinline__ void finish(const HeadStats& e, int c, int t_begin, int t_end,
                                       Sums&& logits) {
  const bool live = c < e.C;
  const int lane = threadIdx.x % 32, slot = (c - lane) / LANE_SLOT;
#pragma unroll 1
  for (int t = t_begin; t < t_end; t += FINISH_ROWS) {
    const int mine = t + lane / 2;  // the row whose results this lane gets
    const int target = mine < t_end ? e.target_of(mine) : -1;
    Rows v;
    __syncwarp();
    logits(t, v);
    float sum = 0.0f;
    if (e.sums) {
      Rows z;
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) z[i] = live ? v[i] : 0.0f;
      sum = over_lanes(z, Sum{});
    }
    const int at = target - (c - lane);  // the lane that holds row `mine`'s target
    const bool here = at >= 0 && at < 32;
    if (__any_sync(0xffffffffu, here)) {
#pragma unroll
      for (int i = 0; i < FINISH_ROWS; ++i) {
        const float z = __shfl_sync(0xffffffffu, v[i], here ? at : 0);
        if (here && lane == 2 * i) e.store_target(mine, z);
      }
    }
#pragma unroll
    for (int i = 0; i < FINISH_ROWS; ++i) v[i] = live ? v[i] : -INFINITY;
    Softmax s;
    s.top = over_lanes(v, Max{}) * LOG2E;
    const float base = Softmax::base(s.top);
#pragma unroll
    for (int i = 0; i < FINISH_ROWS; ++i)
      v[i] = exp2_approx(fmaf(v[i], LOG2E, -__shfl_sync(0xffffffffu, base, 2 * i)));
    s.sum = over_lanes(v, Sum{});
    if (mine < t_end && lane % 2 == 0) e.store(slot, mine, s, sum);
  }
}

// The tokens' factors are read 16 rows ahead, a row a lane, and handed round.
template <class T, class Sums>
__device__ __forceinline__ void finish_typed(const HeadGrad& e, int c, int t_begin, int t_end,
                                             Sums&& logits) {
  T* const D = static_cast<T*>(e.D);
  const int lane = threadIdx.x % 32, column = e.first + c;
  auto load = [&](int t) { return e.row(t + lane, lane < FINISH_ROWS ? t_end : 0); };
  HeadRow next = load(t_begin);
#pragma unroll 1
  for (int t = t_begin; t < t_end; t += FINISH_ROWS) {
    const HeadRow now = next;
    if (t + FINISH_ROWS < t_end) next = load(t + FINISH_ROWS);
    Rows v;
    __syncwarp();
    logits(t, v);
    T* to = D + t * e.ldd + c;
#pragma unroll
    for (int i = 0; i < FINISH_ROWS; ++i, to += e.ldd) {
      auto of = [&](float f) { return __shfl_sync(0xffffffffu, f, i); };
      const int target = __shfl_sync(0xffffffffu, now.target, i);
      const float p = exp2_approx(fmaf(v[i], LOG2E, -of(now.x)));
      const float hit = of(now.hit);
      const float d = fmaf(p, of(now.p), -of(now.all)) - (target == column ? hit : 0.0f);
      if (c < e.C && t + i < t_end &&
          bounds_ok(e.bounds, SITE_C_STORE, (t + i) * e.ldd + c, 1, e.T * e.ldd))
        *to = row::from_f32<T>(target == HeadRow::DEAD ? 0.0f : d);
    }
  }
}

template <class Sums>
__device__ __forceinline__ void finish(const HeadGrad& e, int c, int t_begin, int t_end,
                                       Sums&& logits) {
  if (e.dtype == DT_F16) finish_typed<__half>(e, c, t_begin, t_end, logits);
  else finish_typed<__nv_bfloat16>(e, c, t_begin, t_end, logits);
}

}  // namespace head

// The product of `a` (its Y and what goes with it unused) with one of the
// epilogues above; plan and workspace as launch_linear (linear.cu).
template <class Ep>
cudaError_t launch_head(const LinearArgs& a, const LinearPlan& p, void* workspace, const Ep& ep,
                        cudaStream_t stream, int fault_inject = 0);

// The kernels with these epilogues (head_pair.cu, head_split.cu).
template <class Ep>
cudaError_t launch_head_pair(const CUtensorMap& map_x, const CUtensorMap& map_w, uint32_t idesc,
                             const Ep& ep, bool w_mn, int kt, int clusters, int fault_inject,
                             cudaStream_t stream);
template <class Ep>
linear::LinearKernel head_split_kernel_for(int bt);
cudaError_t head_pair_read_and_clear_status(unsigned int* status);
cudaError_t head_split_read_and_clear_status(unsigned int* status);

}  // namespace mt
