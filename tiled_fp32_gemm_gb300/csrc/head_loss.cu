// The vocabulary loss and its gradient on the host's side, and their small
// kernels: the join of the softmax statistics, the tokens' factors of D, and
// the rounding of dX's sums.
//
// Bound by the tensor cores for batches (2 T K V operations forwards, 6 back,
// of which a third computes the logits again): bf16, V x K weight, calls back to back
// for a second, 8192 x 4096 x 131072 forwards 4.9 to 5.0 ms, 1765 to 1782 TFLOP/s, 4096
// x 4096 x 131072 back 7.8 ms, 1698 TFLOP/s.  Few tokens are bound by the weight's
// stream: one token x 4096 x 131072 162 us, 0.98 of the copy rate; back 571 us, the
// weight read twice and its gradient written.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <type_traits>

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

constexpr int kJoinBatch = 8;  // entries a thread has in flight

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
// thread takes every (THREADS / across)th of a token's, and the threads' meet in
// a fixed tree.  Logarithm and difference in fp64: one a token, and lse is some
// 12 while the loss may be a thousandth of it.
template <int THREADS>
__global__ void __launch_bounds__(THREADS) join_kernel(const JoinArgs a, int across) {
  __shared__ Softmax soft[THREADS];
  __shared__ float plain[THREADS];
  grid_launch_dependents();
  grid_wait();
  const int lanes = THREADS / across, me = threadIdx.x / across;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * across + threadIdx.x % across;
  Softmax s{-INFINITY, 0.0f};
  float sum = 0.0f;
  if (t < a.T) {
    for (int64_t i0 = me; i0 < a.slots; i0 += kJoinBatch * lanes) {
      float2 part[kJoinBatch];
      float add[kJoinBatch];
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        const int64_t i = i0 + k * lanes, at = i * a.T + t;
        const bool there =
            i < a.slots && bounds_ok(a.bounds, SITE_PARTIAL, at, 1, a.slots * a.T);
        part[k] = there ? a.parts[at] : make_float2(-INFINITY, 0.0f);
        add[k] = there && a.sums ? a.sums[at] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < kJoinBatch; ++k) {
        s.join(Softmax{part[k].x, part[k].y});
        sum += add[k];
      }
    }
  }
  soft[threadIdx.x] = s;
  plain[threadIdx.x] = sum;
  for (int n = THREADS / 2; n >= across; n /= 2) {
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

// A piece of the weight: columns `first` .. first + n - 1 of the vocabulary, as
// they are stored at p.
struct Piece {
  const void* p;
  int64_t ld, first, n;
};
Piece piece_of(const HeadLossArgs& a, int64_t first, int64_t n) {
  return Piece{static_cast<const char*>(a.W) + 2 * (a.w_mn ? first : first * a.ldw), a.ldw, first,
               n};
}

// The product whose logits either pass takes.
LinearArgs logits_of(const HeadLossArgs& a, const Piece& w) {
  LinearArgs l{};
  l.T = a.T;
  l.C = w.n;
  l.K = a.K;
  l.X = a.X;
  l.ldx = a.ldx;
  l.W = w.p;
  l.ldw = w.ld;
  l.w_mn = a.w_mn;
  l.dtype = l.out_dtype = a.dtype;
  l.act = ACT_NONE;
  l.bounds = a.bounds;
  return l;
}

// Pairs from one tile on (and more than 128 tokens) up to 1280 values of K, from
// a seventh as many tiles as SMs on past that: half as many as for the linear
// layer, whose epilogue costs the split kernel less (there 16 tokens' statistics
// meet over a warp's lanes, here a thread walks over one token's).  Of a long K few
// tiles want the split kernel's slices.  Measured (bf16, the loss after a flush of
// L2, us for the split kernel against pairs, steps of 2 us, by tiles of 256 x 256):
//   K     256: 4 tiles 22 / 18, 16 tiles 22 / 18, 32 tiles 22 / 18, 128 tiles 35 / 22
//   K    1280: 4 tiles 22 / 22, 16 tiles 24 / 22, 32 tiles 28 / 24
//   K    1536: 4 tiles 22 / 24, 16 tiles 25 / 24, 32 tiles 28 / 24
//   K    2048: 4 tiles 23 / 26, 16 tiles 26 / 26, 32 tiles 32 / 28, 128 tiles 56 / 36
//   K    4096: 4 tiles 26 / 35, 16 tiles 31 / 35, 32 tiles 43 / 39, 128 tiles 82 / 57
//   K    8192: 4 tiles 32 / 51, 16 tiles 43 / 55, 32 tiles 61 / 61, 128 tiles 133 / 96
LinearPlan plan_logits(const LinearArgs& l, int sms) {
  return plan_linear(l, sms, l.K <= 1280 ? 7 : sms);
}

}  // namespace

HeadLossPlan plan_head_loss(const HeadLossArgs& a, int sms) {
  HeadLossPlan p{};
  p.product = plan_logits(logits_of(a, piece_of(a, 0, a.V)), sms);
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
      launch_head(logits_of(a, piece_of(a, 0, a.V)), p.product,
                  ws + p.parts_bytes + p.sums_bytes + p.target_bytes, stats, stream, fault_inject);
  if (e != cudaSuccess) return e;
  // As many tokens side by side as leave a CTA for every SM.
  int across = 1;
  while (across < 32 && a.T >= 2 * across * static_cast<int64_t>(sms)) across *= 2;
  const JoinArgs j{a.T, a.V, p.slots, parts, sums, target_logit, a.target, a.ignore_index,
                   a.smoothing, a.z_loss, loss, lse, a.bounds};
  // Few tokens: the threads that a CTA for every SM would have.
  const unsigned ctas = static_cast<unsigned>(ceil_div(a.T, across));
  return a.T < sms ? launch_dependent(join_kernel<1024>, ctas, 1024, stream, j, across)
                   : launch_dependent(join_kernel<256>, ctas, 256, stream, j, across);
}

// --- backwards ----------------------------------------------------------------

namespace {

// Where D is held times a scale, the tokens' factors with the scale in them are made
// beforehand.
struct RowArgs {
  int64_t T;
  HeadSource source;
  HeadRow* rows;
  // Per-CTA maxima (amax, kMaxCtas of a token's largest factor and as many of
  // |dloss|), and what the products' results are multiplied with to undo D's scale: n
  // factors for their rows, n ones for their columns.
  float* amax;
  float* undo;
  float* ones;
  int64_t n;
  BoundsRecord* bounds;
};

constexpr int kRowThreads = 256;
constexpr int kMaxCtas = 256;  // CTAs that leave maxima

// What counts of a value's size: 0 unless it is finite.
__device__ __forceinline__ float finite(float v) { return v < INFINITY ? v : 0.0f; }

// Maxima over the CTA, in every warp.
__device__ __forceinline__ float2 cta_max(float2 v) {
  __shared__ float2 part[kRowThreads / 32];
  v = make_float2(warp_max(v.x), warp_max(v.y));
  if (threadIdx.x % 32 == 0) part[threadIdx.x / 32] = v;
  __syncthreads();
  v = threadIdx.x % 32 < kRowThreads / 32 ? part[threadIdx.x % 32] : make_float2(0.0f, 0.0f);
  return make_float2(warp_max(v.x), warp_max(v.y));
}

__global__ void __launch_bounds__(kRowThreads) size_kernel(const RowArgs a) {
  grid_launch_dependents();
  grid_wait();
  const HeadSource& s = a.source;
  float2 v = make_float2(0.0f, 0.0f);  // |dloss| (1 + 2 c |lse|), |dloss|
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x; t < a.T;
       t += static_cast<int64_t>(gridDim.x) * kRowThreads) {
    if (!bounds_ok(a.bounds, SITE_ROWS, t, 1, a.T) || s.target[t] == s.ignore_index) continue;
    const float g = fabsf(s.dloss[t]);
    v.x = fmaxf(v.x, finite(g * (1.0f + 2.0f * s.z_loss * fabsf(s.lse[t]))));
    v.y = fmaxf(v.y, finite(g));
  }
  v = cta_max(v);
  if (threadIdx.x == 0) {
    a.amax[blockIdx.x] = v.x;
    a.amax[kMaxCtas + blockIdx.x] = v.y;
  }
}

// D's scale, and what undoes it, from the largest factor of the call and its
// largest |dloss| times 1 - s, the size of a D's entry at its target.  The scale makes
// the latter a power of two, so that a dloss that all tokens have (a mean's 1 / T)
// is not rounded with D, alike everywhere, and brings the largest factor to
// [2^13, 2^14).  Both are good to 2^-24.
struct Scale {
  float scale, undo;
};
__device__ __forceinline__ Scale scale_of(float top, float hit) {
  if (!(top > 0.0f)) return Scale{1.0f, 1.0f};
  const float m = hit > 0.0f ? ldexpf(hit, -ilogbf(hit)) : 1.0f;  // in [1, 2)
  const int e = max(-126, min(126, 13 - ilogbf(top / m)));
  return Scale{ldexpf(1.0f / m, e), ldexpf(m, -e)};
}

// The tokens' factors of D, with its scale from `ctas` CTAs' maxima.  With the largest
// factor in [2^13, 2^14) fp16 keeps its eleven bits down to
// 2^-27 (7.5e-9) of the largest factor and one fewer for each half of that (1e-9: eight
// or nine), and 65504 is not reached.
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const RowArgs a, int ctas) {
  grid_launch_dependents();
  grid_wait();
  const bool there = static_cast<int>(threadIdx.x) < ctas;
  const float2 top = cta_max(there ? make_float2(a.amax[threadIdx.x], a.amax[kMaxCtas + threadIdx.x])
                                   : make_float2(0.0f, 0.0f));
  const float at_target = 1.0f - a.source.smoothing;
  const Scale s = scale_of(top.x, top.y * (at_target > 0.0f ? at_target : 1.0f));
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
       i < max(a.T, a.n); i += static_cast<int64_t>(gridDim.x) * kRowThreads) {
    if (i < a.n) {
      a.undo[i] = s.undo;
      a.ones[i] = 1.0f;
    }
    if (i >= a.T || !bounds_ok(a.bounds, SITE_ROWS, i, 1, a.T)) continue;
    a.rows[i] = a.source.row(i, s.scale);
  }
}

// dX in its type from its planes of sums.  A CTA takes 32 groups of four values;
// its warps take every eighth plane each, and the warps' sums are added in order.
constexpr int kPlaneWarps = kRowThreads / 32;

template <class T>
__global__ void __launch_bounds__(kRowThreads)
    round_planes_kernel(const float* sums, int planes, int64_t plane, int64_t pitch,
                        int64_t extent, const Matrix<T> to, int64_t rows, int cols) {
  __shared__ float4 part[kPlaneWarps][32];
  grid_launch_dependents();
  grid_wait();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const int64_t per_row = pitch / 4, total = rows * per_row;
  for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * 32; i0 < total;
       i0 += static_cast<int64_t>(gridDim.x) * 32) {
    const int64_t i = i0 + lane, r = i / per_row;
    const int c = static_cast<int>(i % per_row) * 4;
    float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i < total) {
#pragma unroll 4
      for (int p = warp; p < planes; p += kPlaneWarps) {
        const int64_t at = p * plane + r * pitch + c;
        if (!bounds_ok(to.rec, SITE_PARTIAL, at, 4, extent)) continue;
        const float4 v = *reinterpret_cast<const float4*>(sums + at);
        s.x += v.x;
        s.y += v.y;
        s.z += v.z;
        s.w += v.w;
      }
    }
    part[warp][lane] = s;
    __syncthreads();
    // Warp w finishes value w of the groups (four of the warps).
    if (warp < 4 && i < total && c + warp < cols) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kPlaneWarps; ++w)
        t += reinterpret_cast<const float*>(&part[w][lane])[warp];
      to.store(r, c + warp, t);
    }
    __syncthreads();
  }
}

// A piece of D: large enough that its products fill the GPU for many rounds of
// tiles and dX's sums seldom wait in memory, 0.4 % of this GPU's.  What counts is
// one piece instead of two (mostly 3 to 5 %, up to 20); of several pieces 1 GiB ones
// are as fast as 512 MiB ones or up to 4 % faster.  Measured (bf16, us for a gradient
// by itself, by limits of 128 / 256 / 512 / 1024 / 2048 MiB, the same form again
// within 2 %):
//   D of  512 MiB   8192 x 1024 x 32768   1316 / 1249 / 1007 / 1003 / 1002
//   D of 1024 MiB   8192 x 2048 x 65536   4593 / 4114 / 4159 / 3949 / 4016
//                   4096 x 4096 x 131072  7834 / 7806 / 7934 / 7672 / 7834
//   D of 1144 MiB   6000 x 2048 x 100000  4969 / 4540 / 4655 / 4501 / 4495
//   D of 2048 MiB   8192 x 512 x 131072   3169 / 2461 / 2399 / 2293 / 2289
//                   8192 x 1024 x 131072  4181 / 4211 / 4107 / 4102 / 3992
//                   16384 x 2048 x 65536  8518 / 8354 / 8225 / 8233 / 7898
//                   4096 x 1024 x 262144  4645 / 3971 / 4150 / 4162 / 4121
//                   32768 x 1024 x 32768  5530 / 4333 / 4336 / 4407 / 3869
constexpr int64_t kPieceBytes = int64_t(1) << 30;

// Whether D is held times a scale: fp16's range wants it, and in both types dloss's
// own digits are then not rounded away (see Scale): 1 / 1021 for all of 1021 tokens in
// bf16, dB in fp32 off by 2.9e-3 of its norm without.  bf16 goes without where the two
// small kernels that make it would show, in gradients of less than some 280 us: the
// weight's passes take as long as 256 tokens' products.  Measured (bf16, us without and
// with): 16 x 1024 x 8192 28.9 / 33, 256 x 1024 x 8192 38 / 43, 1024 x 4096 x 9000 156 / 159,
// 256 x 4096 x 32768 205 / 213, 8192 x 1024 x 8192 274 / 276, 64 x 4096 x 131072 608 / 613,
// 8192 x 2048 x 65536 4088 / 4098, 4096 x 4096 x 131072 7700 / 7790 (under the power cap).
constexpr double kScaledWork = 68719476736.0;  // 2^36

bool scaled(const HeadLossArgs& l) {
  return l.dtype == DT_F16 || (l.T + 256.0) * l.K * l.V >= kScaledWork;
}

// The two products of a piece of the vocabulary.
struct Products {
  LinearArgs x, w;
};
Products products_of(const HeadGradArgs& a, const void* d, int64_t ldd, const Piece& w) {
  const HeadLossArgs& l = a.loss;
  Products p{};
  p.x.dtype = p.w.dtype = l.dtype;
  p.x.act = p.w.act = ACT_NONE;
  p.x.bounds = p.w.bounds = l.bounds;
  // dX = D * W^T: contracted over the piece.
  p.x.T = l.T;
  p.x.C = l.K;
  p.x.K = w.n;
  p.x.X = d;
  p.x.ldx = ldd;
  p.x.W = w.p;
  p.x.ldw = w.ld;
  p.x.w_mn = !l.w_mn;
  p.x.out_dtype = l.dtype;
  p.x.Y = a.dX;
  p.x.ldy = a.lddx;
  // dW as W is stored, contracted over the tokens.
  const int64_t elem = dtype_bytes(a.dw_dtype);
  p.w.T = l.w_mn ? l.K : w.n;
  p.w.C = l.w_mn ? w.n : l.K;
  p.w.K = l.T;
  p.w.X = l.w_mn ? l.X : d;
  p.w.ldx = l.w_mn ? l.ldx : ldd;
  p.w.W = l.w_mn ? d : l.X;
  p.w.ldw = l.w_mn ? ldd : l.ldx;
  p.w.x_mn = p.w.w_mn = 1;
  p.w.out_dtype = a.dw_dtype;
  p.w.Y = a.dW ? static_cast<char*>(a.dW) + elem * (l.w_mn ? w.first : w.first * a.lddw) : nullptr;
  p.w.ldy = a.lddw;
  return p;
}

// Plans of a piece's launches.  Their operands are in a form that TMA reads:
// the three products share the copies of those that are not.
struct PiecePlan {
  LinearPlan logits, x, w;
  bool planes;  // dX's sums are kept in planes of fp32
};
PiecePlan plan_piece(const HeadGradArgs& a, const Piece& piece, int64_t pieces, int64_t ldd,
                     int sms) {
  PiecePlan p{};
  const Products m = products_of(a, nullptr, ldd, piece);
  p.logits = plan_logits(logits_of(a.loss, piece), sms);
  // Planned as if both were wanted: a gradient's bits do not depend on which
  // others are asked for.
  plan_linear_two(m.x, m.w, sms, &p.x, &p.w);
  // dX's sums are kept over several pieces of the vocabulary, and where too few
  // tiles of dX for pairs leave a contraction of 8192 columns or more to be cut into
  // slices of pairs.  The planes and their rounding cost 5 to 10 us, which shorter
  // contractions seldom give back; at 8192 it is about even, from 16384 on a gain
  // but for a few percent past 2048 values of K.  Measured (bf16, the whole gradient
  // after a flush of L2, us without / with slices, T x K by columns):
  //                     4096          8192         16384         65536
  //   16 x 256        24 / 34       29 / 36       42 / 32       83 / 51
  //   16 x 1024       30 / 34       41 / 38       52 / 46      125 / 105
  //   16 x 4096       50 / 48       65 / 66      103 / 105     306 / 308
  //   256 x 256       27 / 40       34 / 41       45 / 38       99 / 64
  //   256 x 1024      36 / 43       45 / 46       68 / 56      199 / 131
  //   256 x 4096      60 / 66       83 / 91      126 / 130     398 / 380
  //   1024 x 256      38 / 43       49 / 52       76 / 56      215 / 144
  //   1024 x 1024     76 / 56      118 / 70      103 / 106     309 / 290
  p.planes = pieces > 1 || (!p.x.pair && piece.n >= 8192);
  if (p.planes) p.w = plan_linear(m.w, sms);
  return p;
}

PaddedCopy copy_of_x(const HeadLossArgs& l) { return PaddedCopy{l.X, l.T, l.K, l.ldx, nullptr}; }
PaddedCopy copy_of_w(const HeadLossArgs& l, const Piece& w) {
  return l.w_mn ? PaddedCopy{w.p, l.K, w.n, w.ld, nullptr}
                : PaddedCopy{w.p, w.n, l.K, w.ld, nullptr};
}

}  // namespace

HeadGradPlan plan_head_grad(const HeadGradArgs& a, int sms) {
  const HeadLossArgs& l = a.loss;
  HeadGradPlan p{};
  if (l.T == 0) {  // one launch that writes zeros
    const Products m = products_of(a, nullptr, ceil_div(l.V, 64) * 64, piece_of(l, 0, l.V));
    p.too_large = plan_linear(m.w, sms).grid > INT32_MAX;
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
  if (scaled(l)) {
    p.rows_bytes = up256(l.T * static_cast<int64_t>(sizeof(HeadRow)));
    p.scale_bytes = 2 * kMaxCtas * 4 + 2 * up256(4 * std::max({l.T, l.K, widest}));
  }
  const Piece first = piece_of(l, 0, widest);
  p.x_bytes = up256(padded_bytes(copy_of_x(l), 2));
  p.w_bytes = up256(padded_bytes(copy_of_w(l, first), 2));
  const PiecePlan q = plan_piece(a, first, p.pieces, p.ldd, sms);
  if (q.planes && a.dX) {
    p.dx = plan_planes(products_of(a, nullptr, p.ldd, first).x, sms);
    p.acc_bytes = up256(p.dx.bytes);
  }
  p.too_large =
      q.logits.grid > INT32_MAX || q.x.grid > INT32_MAX || q.w.grid > INT32_MAX;
  p.workspace_bytes =
      p.d_bytes + p.rows_bytes + p.acc_bytes + p.scale_bytes + p.x_bytes + p.w_bytes;
  return p;
}

cudaError_t launch_head_grad(const HeadGradArgs& args, const HeadGradPlan& p, void* workspace,
                             int sms, cudaStream_t stream) {
  HeadGradArgs a = args;
  HeadLossArgs& l = a.loss;
  if (l.T == 0) {
    const Products m = products_of(a, nullptr, ceil_div(l.V, 64) * 64, piece_of(l, 0, l.V));
    return launch_linear(m.w, plan_linear(m.w, sms), nullptr, stream);  // a sum of nothing
  }
  char* ws = static_cast<char*>(workspace);
  void* const D = ws;
  HeadRow* const rows = p.rows_bytes ? reinterpret_cast<HeadRow*>(ws + p.d_bytes) : nullptr;
  float* const acc = reinterpret_cast<float*>(ws + p.d_bytes + p.rows_bytes);
  char* const scales = ws + p.d_bytes + p.rows_bytes + p.acc_bytes;
  char* const x_copy = scales + p.scale_bytes;
  char* const w_copy = x_copy + p.x_bytes;
  const HeadSource source{a.dloss, a.lse, l.target, l.ignore_index, l.smoothing, l.z_loss,
                          static_cast<int>(l.V)};
  RowArgs r{l.T, source, rows, nullptr, nullptr, nullptr, 0, l.bounds};
  cudaError_t e = cudaSuccess;
  if (p.scale_bytes) {
    r.n = std::max({l.T, l.K, std::min(l.V, p.piece)});
    r.amax = reinterpret_cast<float*>(scales);
    r.undo = reinterpret_cast<float*>(scales + 2 * kMaxCtas * 4);
    r.ones = r.undo + up256(4 * r.n) / 4;
    const int ctas = static_cast<int>(std::min<int64_t>(kMaxCtas, ceil_div(l.T, kRowThreads)));
    e = launch_dependent(size_kernel, static_cast<unsigned>(ctas), kRowThreads, stream, r);
    const int64_t most = 8 * static_cast<int64_t>(sms);
    if (e == cudaSuccess)
      e = launch_dependent(
          rows_kernel,
          static_cast<unsigned>(std::min(most, ceil_div(std::max(l.T, r.n), kRowThreads))),
          kRowThreads, stream, r, ctas);
  }
  for (int64_t i = 0; i < p.pieces && e == cudaSuccess; ++i) {
    Piece piece = piece_of(l, i * p.piece, std::min(p.piece, l.V - i * p.piece));
    PaddedCopy cx = copy_of_x(l), cw = copy_of_w(l, piece);
    cx.dst = i == 0 && p.x_bytes ? x_copy : nullptr;
    cw.dst = p.w_bytes ? w_copy : nullptr;
    e = launch_padded_copies({&cx, &cw}, 2, l.bounds, stream);
    if (e != cudaSuccess) break;
    l.X = cx.p;
    l.ldx = cx.ld;
    piece.p = cw.p;
    piece.ld = cw.ld;
    const PiecePlan q = plan_piece(a, piece, p.pieces, p.ldd, sms);
    const HeadGrad grad{{}, static_cast<int>(l.T), static_cast<int>(piece.n), rows, source,
                        static_cast<int>(piece.first), D, p.ldd, l.dtype, l.bounds};
    e = launch_head(logits_of(l, piece), q.logits, nullptr, grad, stream);
    if (e != cudaSuccess) break;
    Products m = products_of(a, D, p.ldd, piece);
    m.x.row_scale = m.w.row_scale = m.x.scale = m.w.scale = r.undo;
    m.x.col_scale = m.w.col_scale = r.ones;
    m.x.plain = m.w.plain = 1;
    if (a.dX && q.planes) {
      e = launch_linear_planes(m.x, p.dx, acc, i > 0, sms, stream);
      if (e == cudaSuccess && a.dW) e = launch_linear(m.w, q.w, nullptr, stream);
    } else if (a.dX && a.dW) {
      e = launch_linear_two(m.x, q.x, nullptr, m.w, q.w, nullptr, stream);
    } else {
      e = a.dX ? launch_linear(m.x, q.x, nullptr, stream)
               : launch_linear(m.w, q.w, nullptr, stream);
    }
  }
  if (e != cudaSuccess || !a.dX || !p.acc_bytes) return e;
  const int64_t plane = p.dx.rows * p.dx.pitch, all = p.dx.planes * plane;
  const unsigned grid = static_cast<unsigned>(
      std::min<int64_t>(32 * static_cast<int64_t>(sms), ceil_div(l.T * p.dx.pitch / 4, 32)));
  const int64_t extent = view_extent(l.T, l.K, a.lddx);
  const int cols = static_cast<int>(l.K);
  auto go = [&](auto* kernel, auto* to) {
    using V = std::remove_pointer_t<decltype(to)>;
    return launch_dependent(kernel, grid, kRowThreads, stream, static_cast<const float*>(acc),
                            p.dx.planes, plane, p.dx.pitch, all,
                            Matrix<V>{to, a.lddx, extent, l.bounds}, l.T, cols);
  };
  return l.dtype == DT_F16 ? go(round_planes_kernel<__half>, static_cast<__half*>(a.dX))
                           : go(round_planes_kernel<__nv_bfloat16>,
                                static_cast<__nv_bfloat16*>(a.dX));
}

}  // namespace mt
