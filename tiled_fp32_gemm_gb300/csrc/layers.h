// Internal interface between the host side of the feed-forward operators
// (layers_api.cu) and their kernels.  Not part of the C ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "kernels.h"

namespace mt {

// Storage types, as mt_dtype.
enum DType { DT_F16 = 1, DT_BF16 = 2, DT_F32 = 3, DT_E4M3 = 4 };

inline int dtype_bytes(int t) { return t == DT_F32 ? 4 : t == DT_E4M3 ? 1 : 2; }

// launch_dependent with typed arguments, no cluster and no dynamic shared
// memory.
template <class... P>
cudaError_t launch_dependent(void (*kernel)(P...), dim3 grid, int block, cudaStream_t stream,
                             P... args) {
  void* list[] = {&args...};
  return launch_dependent(reinterpret_cast<const void*>(kernel), grid, block, 0, 1, stream, list);
}

// rms_norm.cu.  See mt_rms_norm_args for the operator.
struct RmsNormArgs {
  int64_t rows;
  int d;
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  void* h;
  int64_t ldh;
  void* y;
  int64_t ldy;
  float* scale;
  float* rstd;
  float eps;
  int dtype;
  int e4m3;        // y in 8 bits with scales
  int weight_f32;  // weight in fp32, else in dtype
  BoundsRecord* bounds;
};

cudaError_t launch_rms_norm(const RmsNormArgs& a, cudaStream_t stream);

// rms_norm_grad.cu.  See mt_rms_norm_backward_args for the operator.
struct RmsNormGradArgs {
  int64_t rows;
  int d;
  const void* dy;
  int64_t lddy;
  const void* h;
  int64_t ldh;
  const void* weight;
  const float* rstd;
  const void* dh;
  int64_t lddh;
  void* dx;
  int64_t lddx;
  float* dweight;
  int dtype;
  int weight_f32;
  BoundsRecord* bounds;
  int fault_inject;
};

// Scratch bytes of a call, and the call (workspace of that many bytes).
int64_t rms_norm_grad_workspace(const RmsNormGradArgs& a, int sms);
cudaError_t launch_rms_norm_grad(const RmsNormGradArgs& a, void* workspace, int sms,
                                 cudaStream_t stream);

cudaError_t rms_norm_grad_read_and_clear_status(unsigned int* status);

// Adds `count` rows of `cols` floats (packed, in row order) to out[cols].
cudaError_t launch_add_rows(const float* rows, int count, int cols, float* out,
                            BoundsRecord* bounds, cudaStream_t stream);

// ---------------------------------------------------------------------------
// The fused product of the linear layer and of its gradient:
//
//   z[t][c] = row_scale[t] * col_scale[c] * sum_k X[t][k] * W[k][c] + bias[c]
//   Y[t][c] = act(z[t][c]) + residual[t][c],  Z[t][c] = z[t][c] (optional)
//
// X: T x K, stored K-contiguous, or T-contiguous (K x T) when x_mn.  W: K x C,
// stored K-contiguous (C x K), or C-contiguous (K x C) when w_mn.  On the
// tensor cores the columns of Y are the MMA's 128 lanes and its rows the
// accumulator's columns, so a warp holds 32 consecutive columns of a row of Y
// and its loads and stores are coalesced whatever the row pitch.
enum Activation { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

struct LinearArgs {
  int64_t T, C, K;
  const void* X;
  int64_t ldx;
  const void* W;
  int64_t ldw;
  int x_mn, w_mn;
  void* Y;
  int64_t ldy;
  void* Z;
  int64_t ldz;
  const void* residual;
  int64_t ldr;
  const float* bias;
  const float* row_scale;
  const float* col_scale;
  int dtype;      // X and W: DT_F16, DT_BF16 or DT_E4M3 (then both K-contiguous)
  int out_dtype;  // Y, Z, residual: DT_F16, DT_BF16 or DT_F32
  int act;
  BoundsRecord* bounds;
  // A product of 16-bit operands and no more: Y = scale * X * W (scale: one value
  // on the device, null: 1).  No bias, activation, scales, residual or Z.
  int plain = 0;
  const float* scale = nullptr;
};

// A plain product whose contraction is cut into slices, each with a plane of
// sums of its own: plane s, rows s * rows .. of `sums` (fp32, pitch a multiple of
// 4, `rows` T rounded up to whole tiles), is written, or with `add` added to.
struct PlanesPlan {
  int planes, kt_per_slice;
  int64_t rows, pitch, bytes;
};
PlanesPlan plan_planes(const LinearArgs& a, int sms);
cudaError_t launch_linear_planes(const LinearArgs& a, const PlanesPlan& p, float* sums, bool add,
                                 int sms, cudaStream_t stream);

// What a product launches.  pair: CTA pairs on tiles of 256 columns x 256
// rows of Y (linear_pair.cu); else CTA tiles of bc = 128 columns x bt rows,
// each computed by a cluster of `split` CTAs that take a slice of K each and
// add their sums through distributed shared memory (linear_split.cu).
struct LinearPlan {
  int pair;
  int bt, bc, split, stages, threads;
  int cluster;  // CTAs of the launch's clusters: split, or 1 < cluster with split = 1
  int64_t smem_bytes, grid;
  int64_t copy_x_bytes, copy_w_bytes;  // padded copies of operands TMA cannot read
  int64_t workspace_bytes;
};

LinearPlan plan_linear(const LinearArgs& a, int sms);
// The same with pairs from `sevenths` sevenths of a pair on.
LinearPlan plan_linear(const LinearArgs& a, int sms, int sevenths);
// Two products that do not depend on one another: planned for one launch when
// both take the split kernel.
void plan_linear_two(const LinearArgs& a, const LinearArgs& b, int sms, LinearPlan* pa,
                     LinearPlan* pb);
// Attributes of the kernels, once per device.
cudaError_t linear_prepare();
cudaError_t launch_linear(const LinearArgs& a, const LinearPlan& p, void* workspace,
                          cudaStream_t stream, int fault_inject = 0);
cudaError_t launch_linear_two(const LinearArgs& a, const LinearPlan& pa, void* wa,
                              const LinearArgs& b, const LinearPlan& pb, void* wb,
                              cudaStream_t stream);
cudaError_t linear_read_and_clear_status(unsigned int* status);

// Whether TMA reads a matrix of `elem`-byte values in place: 16-byte aligned
// base, row pitch a multiple of 16 bytes.
bool tma_readable(const void* p, int64_t ld, int elem);

// A stored matrix of `elem`-byte values and where its padded copy goes (dst null:
// nowhere), for operands that several products read: TMA reads the copy in
// place.  padded_bytes: the copy's size, 0 where TMA reads the matrix itself.
struct PaddedCopy {
  const void* p;
  int64_t rows, cols, ld;
  void* dst;
};
int64_t padded_bytes(const PaddedCopy& c, int elem);
// Copies up to two (null: none) in one launch; p and ld become the copies'.
cudaError_t launch_padded_copies(PaddedCopy* const (&copies)[2], int elem, BoundsRecord* bounds,
                                 cudaStream_t stream);

// linear_grad.cu: dz = dY * act'(Z) rounded to `dtype` (dZ null: not written;
// else 16-byte aligned rows of lddz >= N values, lddz a multiple of 8, whose
// last chunk of eight is padded with zeros), and the column sums of the unrounded dz (dbias null: not
// computed), through `partial` (linear_dz_workspace bytes).
struct LinearDzArgs {
  int64_t M;
  int N;
  const void* dY;
  int64_t lddy;
  const void* Z;
  int64_t ldz;
  void* dZ;
  int64_t lddz;
  float* dbias;
  int dtype, act;
  BoundsRecord* bounds;
};
int64_t linear_dz_workspace(const LinearDzArgs& a, int sms);
cudaError_t launch_linear_dz(const LinearDzArgs& a, void* partial, int sms, cudaStream_t stream);

}  // namespace mt
