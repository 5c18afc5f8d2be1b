// The vocabulary loss and its gradient on the host's side, and their small
// kernels: the join of the softmax statistics, the tokens' factors of D, and
// the rounding of dX's sums.
//
// Bound by the tensor cores for batches (2 T K V operations forwards, 6 back,
// of which a third computes the logits again), by the weight's stream for a
// few tokens.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "head.cuh"
#include "model.h"
#include "row_util.cuh"

namespace mt {
namespace {

using namespace head;
using row::Matrix;
using row::warp_max;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t up256(int64_t bytes) { return ceil_div(bytes, 256) * 256; }

// --- forwards -----------------------------------------------------------------

constexpr int kJoinThreads = 1024;

struct JoinArgs {
  int64_t T, V, slots;
  const float2* parts;
  const float* sums;  // nullptr: no smoothing
  const float* target_logit;
  const int64_t* target;
  int64_t ignore_index;
  float smoothing, z_loss;
  float* loss;
  float* lse;
  BoundsRecord* bounds;
};

// Joins the entries of `across` tokens (a power of two up to 32) a CTA: a
// thread takes every (1024 / across)th of a token's, and the threads' meet in
// a fixed tree.  Logarithm and difference in fp64: one a token, and lse is some
// 12 while the loss may be a thousandth of it.
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const JoinArgs a, int across) {
  __shared__ Softmax soft[kJoinThreads];
  __shared__ float plain[kJoinThreads];
  grid_launch_dependents();
  grid_wait();
  const int lanes = kJoinThreads / across, me = threadIdx.x / across;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * across + threadIdx.x % across;
  Softmax s{-INFINITY, 0.0f};
  float sum = 0.0f;
  if (t < a.T) {
#pragma unroll 4
    for (int64_t i = me; i < a.slots; i += lanes) {
      const int64_t at = i * a.T + t;
      if (!bounds_ok(a.bounds, SITE_PARTIAL, at, 1, a.slots * a.T)) continue;
      const float2 p = a.parts[at];
      s.join(Softmax{p.x, p.y});
      if (a.sums) sum += a.sums[at];
    }
  }
  soft[threadIdx.x] = s;
  plain[threadIdx.x] = sum;
  for (int n = kJoinThreads / 2; n >= across; n /= 2) {
    __syncthreads();
    if (threadIdx.x < n) {
      soft[threadIdx.x].join(soft[threadIdx.x + n]);
      plain[threadIdx.x] += plain[threadIdx.x + n];
    }
  }
  if (me > 0 || t >= a.T || !bounds_ok(a.bounds, SITE_ROWS, t, 1, a.T)) return;
  s = soft[threadIdx.x];
  const double lse = s.top * 0.69314718055994531 + log(static_cast<double>(s.sum));
  a.lse[t] = static_cast<float>(lse);
  const int64_t target = a.target[t];
  float loss = 0.0f;
  if (target != a.ignore_index) {
    if (target >= 0 && target < a.V) {
      double z = a.target_logit[t];
      if (a.sums)
        z += static_cast<double>(a.smoothing) *
             (plain[threadIdx.x] / static_cast<double>(a.V) - z);
      loss = static_cast<float>(lse - z + static_cast<double>(a.z_loss) * lse * lse);
    } else {
      loss = NAN;
    }
  }
  a.loss[t] = loss;
}

// The product whose logits either pass takes, columns first .. first + n - 1.
LinearArgs logits_of(const HeadLossArgs& a, int64_t first, int64_t n) {
  LinearArgs l{};
  l.T = a.T;
  l.C = n;
  l.K = a.K;
  l.X = a.X;
  l.ldx = a.ldx;
  l.W = static_cast<const char*>(a.W) + 2 * (a.w_mn ? first : first * a.ldw);
  l.ldw = a.ldw;
  l.w_mn = a.w_mn;
  l.dtype = l.out_dtype = a.dtype;
  l.act = ACT_NONE;
  l.bounds = a.bounds;
  return l;
}

}  // namespace

HeadLossPlan plan_head_loss(const HeadLossArgs& a, int sms) {
  HeadLossPlan p{};
  p.product = plan_linear(logits_of(a, 0, a.V), sms);
  p.slots = p.product.pair ? ceil_div(a.V, 2 * PAIR_SLOT) * 2
                           : ceil_div(a.V, linear::LINEAR_BC) * (linear::LINEAR_BC / LANE_SLOT);
  p.parts_bytes = up256(p.slots * a.T * 8);
  p.sums_bytes = a.smoothing != 0.0f ? up256(p.slots * a.T * 4) : 0;
  p.target_bytes = up256(a.T * 4);
  p.workspace_bytes =
      p.parts_bytes + p.sums_bytes + p.target_bytes + p.product.workspace_bytes;
  return p;
}

cudaError_t launch_head_loss(const HeadLossArgs& a, const HeadLossPlan& p, float* loss, float* lse,
                             void* workspace, int sms, int fault_inject, cudaStream_t stream) {
  char* ws = static_cast<char*>(workspace);
  float2* parts = reinterpret_cast<float2*>(ws);
  float* sums = p.sums_bytes ? reinterpret_cast<float*>(ws + p.parts_bytes) : nullptr;
  float* target_logit = reinterpret_cast<float*>(ws + p.parts_bytes + p.sums_bytes);
  const HeadStats stats{static_cast<int>(a.T), static_cast<int>(a.V), a.target, parts, sums,
                        target_logit, p.slots, a.bounds};
  const cudaError_t e =
      launch_head(logits_of(a, 0, a.V), p.product,
                  ws + p.parts_bytes + p.sums_bytes + p.target_bytes, stats, stream, fault_inject);
  if (e != cudaSuccess) return e;
  // As many tokens side by side as leave a CTA for every SM.
  int across = 1;
  while (across < 32 && a.T >= 2 * across * static_cast<int64_t>(sms)) across *= 2;
  const JoinArgs j{a.T, a.V, p.slots, parts, sums, target_logit, a.target, a.ignore_index,
                   a.smoothing, a.z_loss, loss, lse, a.bounds};
  return launch_dependent(join_kernel, static_cast<unsigned>(ceil_div(a.T, across)), kJoinThreads,
                          stream, j, across);
}

// --- backwards ----------------------------------------------------------------

namespace {

struct RowArgs {
  int64_t T, V;
  const float* dloss;
  const float* lse;
  const int64_t* target;
  int64_t ignore_index;
  float smoothing, z_loss;
  HeadRow* rows;
  int* column;
  // fp16 only (null otherwise): per-CTA maxima of |dloss| (amax), and what the
  // products' results are multiplied with to undo D's scale: n factors for
  // their rows, n ones for their columns.
  float* amax;
  float* undo;
  float* ones;
  int64_t n;
  BoundsRecord* bounds;
};

constexpr int kRowThreads = 256;
constexpr int kMaxCtas = 256;  // CTAs that leave a maximum

// The largest factor of a token's D: |dloss| (1 + 2 c |lse|); 0 for what does
// not count (no target, not finite).
__device__ __forceinline__ float size_of(const RowArgs& a, int64_t t) {
  if (a.target[t] == a.ignore_index) return 0.0f;
  const float v = fabsf(a.dloss[t]) * (1.0f + 2.0f * a.z_loss * fabsf(a.lse[t]));
  return v < INFINITY ? v : 0.0f;
}

// Maximum over the CTA, in thread 0's warp.
__device__ __forceinline__ float cta_max(float v) {
  __shared__ float part[kRowThreads / 32];
  v = warp_max(v);
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  return warp_max(threadIdx.x % 32 < kRowThreads / 32 ? part[threadIdx.x % 32] : 0.0f);
}

__global__ void __launch_bounds__(kRowThreads) size_kernel(const RowArgs a) {
  grid_launch_dependents();
  grid_wait();
  float v = 0.0f;
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kRowThreads)
    if (bounds_ok(a.bounds, SITE_ROWS, t, 1, a.T)) v = fmaxf(v, size_of(a, t));
  v = cta_max(v);
  if (threadIdx.x == 0) a.amax[blockIdx.x] = v;
}

// The tokens' factors of D; with `ctas` maxima, D's scale is the power of two
// that brings the largest to [2^13, 2^14): fp16 then keeps ten digits of a
// probability down to 2^-27 of the largest factor, and 65504 is not reached.
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowArgs a, int ctas) {
  grid_launch_dependents();
  grid_wait();
  float scale = 1.0f;
  if (a.amax) {
    const float top = cta_max(static_cast<int>(threadIdx.x) < ctas ? a.amax[threadIdx.x] : 0.0f);
    const int e = top > 0.0f ? max(-126, min(126, 13 - ilogbf(top))) : 0;
    scale = ldexpf(1.0f, e);
  }
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
       i < max(a.T, a.n); i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
    if (i < a.n) {
      a.undo[i] = 1.0f / scale;
      a.ones[i] = 1.0f;
    }
    if (i >= a.T || !bounds_ok(a.bounds, SITE_ROWS, i, 1, a.T)) continue;
    const int64_t target = a.target[i];
    HeadRow r{0.0f, 0.0f, 0.0f, 0.0f};
    int column = HeadGrad::DEAD;
    if (target != a.ignore_index) {
      const bool inside = target >= 0 && target < a.V;
      const float lse = a.lse[i], g = inside ? a.dloss[i] * scale : NAN;
      r.x = lse * LOG2E;
      r.p = g * (1.0f + 2.0f * a.z_loss * lse);
      r.all = g * (a.smoothing / static_cast<float>(a.V));
      r.hit = g * (1.0f - a.smoothing);
      column = inside ? static_cast<int>(target) : -1;
    }
    a.rows[i] = r;
    a.column[i] = column;
  }
}

// dX in its type from its sums over the pieces of the vocabulary.
template <class T>
__global__ void __launch_bounds__(kRowThreads)
    round_rows_kernel(const Matrix<const float> acc, const Matrix<T> to, int64_t rows, int cols) {
  grid_launch_dependents();
  grid_wait();
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int c = threadIdx.x; c < cols; c += kRowThreads) to.store(r, c, acc.load(r, c));
}

// A piece of D: large enough that its products fill the GPU for several rounds
// of tiles, small enough to stay near the chip between the kernel that writes
// it and the two that read it.
constexpr int64_t kPieceBytes = int64_t(256) << 20;

// The two products of a piece of n columns from `first` on.
struct Products {
  LinearArgs x, w;
};
Products products_of(const HeadGradArgs& a, const void* d, int64_t ldd, int64_t first, int64_t n) {
  const HeadLossArgs& l = a.loss;
  Products p{};
  p.x.dtype = p.w.dtype = l.dtype;
  p.x.act = p.w.act = ACT_NONE;
  p.x.bounds = p.w.bounds = l.bounds;
  // dX = D * W^T: contracted over the piece.
  p.x.T = l.T;
  p.x.C = l.K;
  p.x.K = n;
  p.x.X = d;
  p.x.ldx = ldd;
  p.x.W = static_cast<const char*>(l.W) + 2 * (l.w_mn ? first : first * l.ldw);
  p.x.ldw = l.ldw;
  p.x.w_mn = !l.w_mn;
  p.x.out_dtype = l.dtype;
  p.x.Y = a.dX;
  p.x.ldy = a.lddx;
  // dW as W is stored, contracted over the tokens.
  const int64_t elem = dtype_bytes(a.dw_dtype);
  p.w.T = l.w_mn ? l.K : n;
  p.w.C = l.w_mn ? n : l.K;
  p.w.K = l.T;
  p.w.X = l.w_mn ? l.X : d;
  p.w.ldx = l.w_mn ? l.ldx : ldd;
  p.w.W = l.w_mn ? d : l.X;
  p.w.ldw = l.w_mn ? ldd : l.ldx;
  p.w.x_mn = p.w.w_mn = 1;
  p.w.out_dtype = a.dw_dtype;
  p.w.Y = a.dW ? static_cast<char*>(a.dW) + elem * (l.w_mn ? first : first * a.lddw) : nullptr;
  p.w.ldy = a.lddw;
  return p;
}

// Plans of a piece's launches.
struct PiecePlan {
  LinearPlan logits, x, w;
  int64_t bytes(const HeadGradArgs& a) const {
    return std::max(up256(logits.workspace_bytes),
                    (a.dX ? up256(x.workspace_bytes) : 0) + (a.dW ? up256(w.workspace_bytes) : 0));
  }
};
PiecePlan plan_piece(const HeadGradArgs& a, int64_t ldd, int64_t first, int64_t n, int sms) {
  PiecePlan p{};
  const Products m = products_of(a, nullptr, ldd, first, n);
  p.logits = plan_linear(logits_of(a.loss, first, n), sms);
  // Planned as if both were wanted: a gradient's bits do not depend on which
  // others are asked for.
  plan_linear_two(m.x, m.w, sms, &p.x, &p.w);
  return p;
}

}  // namespace

HeadGradPlan plan_head_grad(const HeadGradArgs& a, int sms) {
  const HeadLossArgs& l = a.loss;
  HeadGradPlan p{};
  if (l.T == 0) {  // one launch that writes zeros
    p.too_large = plan_linear(products_of(a, nullptr, ceil_div(l.V, 64) * 64, 0, l.V).w, sms).grid >
                  INT32_MAX;
    return p;
  }
  const int64_t most = std::max<int64_t>(256, kPieceBytes / (2 * l.T) / 256 * 256);
  // Pieces of about one size.
  p.pieces = ceil_div(l.V, most);
  p.piece = std::min(most, ceil_div(ceil_div(l.V, p.pieces), 256) * 256);
  p.pieces = ceil_div(l.V, p.piece);
  const int64_t widest = std::min(l.V, p.piece);
  p.ldd = ceil_div(widest, 64) * 64;
  p.d_bytes = up256(l.T * p.ldd * 2);
  p.rows_bytes = up256(l.T * static_cast<int64_t>(sizeof(HeadRow))) + up256(l.T * 4);
  p.acc_bytes = a.dX && p.pieces > 1 ? up256(l.T * l.K * 4) : 0;
  if (l.dtype == DT_F16)
    p.scale_bytes = kMaxCtas * 4 + 2 * up256(4 * std::max({l.T, l.K, widest}));
  // The last piece is narrower, and may take other kernels.
  for (int64_t first : {int64_t(0), (p.pieces - 1) * p.piece}) {
    const PiecePlan q = plan_piece(a, p.ldd, first, std::min(p.piece, l.V - first), sms);
    p.product_bytes = std::max(p.product_bytes, q.bytes(a));
    p.too_large |= q.logits.grid > INT32_MAX || q.x.grid > INT32_MAX || q.w.grid > INT32_MAX;
  }
  p.workspace_bytes = p.d_bytes + p.rows_bytes + p.acc_bytes + p.scale_bytes + p.product_bytes;
  return p;
}

cudaError_t launch_head_grad(const HeadGradArgs& a, const HeadGradPlan& p, void* workspace,
                             int sms, cudaStream_t stream) {
  const HeadLossArgs& l = a.loss;
  if (l.T == 0) {
    const Products m = products_of(a, nullptr, ceil_div(l.V, 64) * 64, 0, l.V);
    return launch_linear(m.w, plan_linear(m.w, sms), nullptr, stream);  // a sum of nothing
  }
  char* ws = static_cast<char*>(workspace);
  void* const D = ws;
  HeadRow* const rows = reinterpret_cast<HeadRow*>(ws + p.d_bytes);
  int* const column = reinterpret_cast<int*>(
      ws + p.d_bytes + up256(l.T * static_cast<int64_t>(sizeof(HeadRow))));
  float* const acc = reinterpret_cast<float*>(ws + p.d_bytes + p.rows_bytes);
  char* const scales = ws + p.d_bytes + p.rows_bytes + p.acc_bytes;
  char* const products = scales + p.scale_bytes;
  RowArgs r{l.T, l.V, a.dloss, a.lse, l.target, l.ignore_index, l.smoothing, l.z_loss, rows,
            column, nullptr, nullptr, nullptr, 0, l.bounds};
  int ctas = 0;
  cudaError_t e = cudaSuccess;
  if (p.scale_bytes) {
    r.n = std::max({l.T, l.K, std::min(l.V, p.piece)});
    r.amax = reinterpret_cast<float*>(scales);
    r.undo = reinterpret_cast<float*>(scales + kMaxCtas * 4);
    r.ones = r.undo + up256(4 * r.n) / 4;
    ctas = static_cast<int>(std::min<int64_t>(kMaxCtas, ceil_div(l.T, kRowThreads)));
    e = launch_dependent(size_kernel, static_cast<unsigned>(ctas), kRowThreads, stream, r);
  }
  if (e == cudaSuccess)
    e = launch_dependent(
        rows_kernel,
        static_cast<unsigned>(std::min<int64_t>(8 * static_cast<int64_t>(sms),
                                                ceil_div(std::max(l.T, r.n), kRowThreads))),
        kRowThreads, stream, r, ctas);
  for (int64_t i = 0; i < p.pieces && e == cudaSuccess; ++i) {
    const int64_t first = i * p.piece, n = std::min(p.piece, l.V - first);
    const PiecePlan q = plan_piece(a, p.ldd, first, n, sms);
    const HeadGrad grad{static_cast<int>(l.T), static_cast<int>(n), rows, column,
                        static_cast<int>(first), D, p.ldd, l.dtype, l.bounds};
    e = launch_head(logits_of(l, first, n), q.logits, products, grad, stream);
    if (e != cudaSuccess) break;
    Products m = products_of(a, D, p.ldd, first, n);
    m.x.row_scale = m.w.row_scale = r.undo;
    m.x.col_scale = m.w.col_scale = r.ones;
    if (p.acc_bytes) {
      m.x.out_dtype = DT_F32;
      m.x.Y = acc;
      m.x.ldy = l.K;
      m.x.residual = i > 0 ? acc : nullptr;
      m.x.ldr = l.K;
    }
    char* const wx = products;
    char* const ww = products + (a.dX ? up256(q.x.workspace_bytes) : 0);
    if (a.dX && a.dW) e = launch_linear_two(m.x, q.x, wx, m.w, q.w, ww, stream);
    else if (a.dX) e = launch_linear(m.x, q.x, wx, stream);
    else e = launch_linear(m.w, q.w, ww, stream);
  }
  if (e != cudaSuccess || !p.acc_bytes) return e;
  const Matrix<const float> from{acc, l.K, l.T * l.K, l.bounds};
  const unsigned grid = static_cast<unsigned>(std::min<int64_t>(l.T, 16 * sms));
  const int64_t extent = view_extent(l.T, l.K, a.lddx);
  const int cols = static_cast<int>(l.K);
  if (l.dtype == DT_F16)
    return launch_dependent(
        round_rows_kernel<__half>, grid, kRowThreads, stream, from,
        Matrix<__half>{static_cast<__half*>(a.dX), a.lddx, extent, l.bounds}, l.T, cols);
  return launch_dependent(
      round_rows_kernel<__nv_bfloat16>, grid, kRowThreads, stream, from,
      Matrix<__nv_bfloat16>{static_cast<__nv_bfloat16*>(a.dX), a.lddx, extent, l.bounds}, l.T,
      cols);
}

}  // namespace mt
