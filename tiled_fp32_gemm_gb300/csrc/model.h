// Internal interface between the host side of the residual joins and the
// vocabulary's loss (model_api.cu) and their kernels.  Not part of the C ABI.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "layers.h"
#include "philox.cuh"

namespace mt {

// layer_norm.cu.  See mt_layer_norm_args for the operator.
struct LayerNormArgs {
  int64_t rows;
  int d;
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  const void* weight;
  const void* bias;
  void* h;
  int64_t ldh;
  void* y;
  int64_t ldy;
  float* mean;
  float* rstd;
  float eps;
  int dtype;
  int weight_f32;  // weight and bias in fp32, else in dtype
  int drop;        // whether x is dropped from
  DropoutArgs dropout;
  BoundsRecord* bounds;
};

cudaError_t launch_layer_norm(const LayerNormArgs& a, cudaStream_t stream);

// layer_norm_grad.cuh.  See mt_layer_norm_backward_args for the operator.
struct LayerNormGradArgs {
  int64_t rows;
  int d;
  const void* dy;
  int64_t lddy;
  const void* h;
  int64_t ldh;
  const void* weight;
  const float* mean;
  const float* rstd;
  const void* dh;
  int64_t lddh;
  void* dx;
  int64_t lddx;
  void* dres;  // with dropout only
  int64_t lddres;
  float* dweight;
  float* dbias;
  int dtype;
  int weight_f32;
  int drop;
  DropoutArgs dropout;
  BoundsRecord* bounds;
  int fault_inject;
};

int64_t layer_norm_grad_workspace(const LayerNormGradArgs& a, int sms);
cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& a, void* workspace, int sms,
                                   cudaStream_t stream);
cudaError_t layer_norm_grad_read_and_clear_status(unsigned int* status);
// Its parts by storage type.
cudaError_t launch_layer_norm_grad_f16(const LayerNormGradArgs& a, float* partial, int sms,
                                       cudaStream_t stream);
cudaError_t launch_layer_norm_grad_bf16(const LayerNormGradArgs& a, float* partial, int sms,
                                        cudaStream_t stream);
cudaError_t launch_layer_norm_grad_f32(const LayerNormGradArgs& a, float* partial, int sms,
                                       cudaStream_t stream);
cudaError_t layer_norm_grad_f16_read_and_clear_status(unsigned int* status);
cudaError_t layer_norm_grad_bf16_read_and_clear_status(unsigned int* status);
cudaError_t layer_norm_grad_f32_read_and_clear_status(unsigned int* status);

// dropout.cu.  See mt_dropout_args for the operator.
struct DropoutCall {
  int64_t rows;
  int d;
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  void* y;
  int64_t ldy;
  int dtype;
  DropoutArgs dropout;
  BoundsRecord* bounds;
};

cudaError_t launch_dropout(const DropoutCall& a, int sms, cudaStream_t stream);

// head_loss.cu.  See mt_linear_cross_entropy_args for the operator.  The
// product's operands: T tokens of K values, the weight K x V (w_mn) or V x K.
struct HeadLossArgs {
  int64_t T, K, V;
  const void* X;
  int64_t ldx;
  const void* W;
  int64_t ldw;
  int w_mn;
  const int64_t* target;
  int64_t ignore_index;
  float smoothing, z_loss;
  int dtype;
  BoundsRecord* bounds;
};

// Attributes of the loss's kernels and of its plain products', once per device.
cudaError_t head_prepare();

// A forward pass: its scratch, and the launches.
struct HeadLossPlan {
  LinearPlan product;
  int64_t slots;  // entries of softmax statistics a token leaves
  int64_t parts_bytes, sums_bytes, target_bytes, workspace_bytes;
};
HeadLossPlan plan_head_loss(const HeadLossArgs& a, int sms);
cudaError_t launch_head_loss(const HeadLossArgs& a, const HeadLossPlan& p, float* loss, float* lse,
                             void* workspace, int sms, int fault_inject, cudaStream_t stream);

// A backward pass, a piece of the vocabulary at a time.
struct HeadGradArgs {
  HeadLossArgs loss;
  const float* dloss;
  const float* lse;
  void* dX;  // null: not wanted
  int64_t lddx;
  void* dW;  // null: not wanted
  int64_t lddw;
  int dw_dtype;
};
struct HeadGradPlan {
  int64_t piece;   // columns of the vocabulary at a time, a multiple of 256
  int64_t pieces;
  int64_t ldd;     // row pitch of a piece of D
  int64_t d_bytes, rows_bytes, acc_bytes, scale_bytes, x_bytes, w_bytes, workspace_bytes;
  PlanesPlan dx;   // dX's sums, where they are kept (acc_bytes)
  bool too_large;  // a grid past 2^31 - 1
};
HeadGradPlan plan_head_grad(const HeadGradArgs& a, int sms);
cudaError_t launch_head_grad(const HeadGradArgs& a, const HeadGradPlan& p, void* workspace,
                             int sms, cudaStream_t stream);


}  // namespace mt
