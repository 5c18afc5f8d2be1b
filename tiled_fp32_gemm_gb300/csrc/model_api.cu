// C entry points of the residual joins and the vocabulary's loss
// (include/mt_model.h): argument checks, launch choices, scratch.
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include <cuda_runtime.h>

#include "api_util.h"
#include "host.h"
#include "model.h"
#include "mt_model.h"

namespace {

using namespace mt::host;

// Longest row of a norm or of dropout: the kernels step a 32-bit column by up
// to 4096 past the row's last strip of 256.
constexpr int64_t kMaxWidth = INT32_MAX - 8191;

bool float_type(int t) { return half_type(t) || t == MT_DTYPE_F32; }
bool sizes_ok(int64_t rows, int64_t d) {
  return rows >= 0 && d >= 0 && d <= kMaxWidth && rows <= INT32_MAX;
}
bool probability(double p) { return p >= 0.0 && p < 1.0; }

// A matrix that may be missing, and a vector of n values.
View optional(const void* p, int64_t rows, int64_t cols, int64_t ld, int elem) {
  return View{p, p ? rows : 0, cols, p ? ld : INT32_MAX, elem};
}
View vector(const void* p, int64_t n, int elem) { return View{p, p ? 1 : 0, n, INT32_MAX, elem}; }
View seed_view(const int64_t* seed, bool used) { return View{seed, used ? 1 : 0, 1, 1, 8}; }

mt::DropoutArgs dropout_args(const int64_t* seed, uint64_t sequence, double p) {
  return mt::DropoutArgs{seed, static_cast<uint32_t>(sequence),
                         static_cast<uint32_t>(sequence >> 32),
                         static_cast<uint32_t>(std::floor(p * 4294967296.0)),
                         static_cast<float>(1.0 / (1.0 - p))};
}

// The loss's kernels and those of the products it makes.
OncePerDevice g_loss_ready;

mt_status prepare_loss(int dev) {
  const mt_status st = prepare_linear(dev);
  return st == MT_OK ? g_loss_ready.run(dev, mt::head_prepare) : st;
}

mt_status launched(cudaError_t e) {
  if (e == cudaSuccess) return MT_OK;
  cudaGetLastError();
  return MT_ERR_LAUNCH;
}

}  // namespace

extern "C" {

mt_status mt_layer_norm(const mt_layer_norm_args* g, cudaStream_t stream) {
  if (!g || !sizes_ok(g->rows, g->d) || !float_type(g->dtype) || g->reserved)
    return MT_ERR_INVALID_ARG;
  if ((g->weight || g->bias) && g->weight_dtype != g->dtype && g->weight_dtype != MT_DTYPE_F32)
    return MT_ERR_INVALID_ARG;
  if (!(g->eps >= 0.0f) || std::isinf(g->eps) || !probability(g->dropout))
    return MT_ERR_INVALID_ARG;
  const int e = mt::dtype_bytes(g->dtype), ew = g->weight_dtype == MT_DTYPE_F32 ? 4 : e;
  const int64_t rows = g->rows, d = g->d;
  const View x{g->x, rows, d, g->ldx, e}, y{g->y, rows, d, g->ldy, e};
  const View res = optional(g->residual, rows, d, g->ldr, e);
  const View h = optional(g->h, rows, d, g->ldh, e);
  const View w = vector(g->weight, d, ew), b = vector(g->bias, d, ew);
  const View mean = optional(g->mean, rows, 1, 1, 4), rstd = optional(g->rstd, rows, 1, 1, 4);
  const View seed = seed_view(g->seed, g->dropout > 0.0);
  for (const View* v : {&x, &y, &res, &h, &w, &b, &mean, &rstd, &seed})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  if ((h.hits(x) && !h.same(x)) || (h.hits(res) && !h.same(res)) || (y.hits(x) && !y.same(x)) ||
      y.hits(res) || y.hits(h))
    return MT_ERR_ALIAS;
  for (const View* out : {&h, &y, &mean, &rstd})
    for (const View* in : {&w, &b, &seed})
      if (out->hits(*in)) return MT_ERR_ALIAS;
  for (const View* out : {&mean, &rstd})
    for (const View* v : {&x, &res, &h, &y})
      if (out->hits(*v)) return MT_ERR_ALIAS;
  if (mean.hits(rstd)) return MT_ERR_ALIAS;
  if (rows == 0) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  const mt_status st = current_device(&dev, &info);
  if (st != MT_OK) return st;
  const mt::LayerNormArgs a{rows, static_cast<int>(d), g->x, g->ldx, g->residual, g->ldr,
                            g->weight, g->bias, g->h, g->ldh, g->y, g->ldy, g->mean, g->rstd,
                            g->eps, g->dtype, ew == 4 ? 1 : 0, g->dropout > 0.0 ? 1 : 0,
                            dropout_args(g->seed, g->sequence, g->dropout), bounds_record()};
  return launched(mt::launch_layer_norm(a, stream));
}

mt_status mt_layer_norm_backward(const mt_layer_norm_backward_args* g, cudaStream_t stream) {
  if (!g || !sizes_ok(g->rows, g->d) || !float_type(g->dtype) || g->reserved ||
      g->fault_inject < 0 || g->fault_inject > 1 || !probability(g->dropout))
    return MT_ERR_INVALID_ARG;
  if (g->weight && g->weight_dtype != g->dtype && g->weight_dtype != MT_DTYPE_F32)
    return MT_ERR_INVALID_ARG;
  const bool drop = g->dropout > 0.0;
  if (!drop && g->dresidual) return MT_ERR_INVALID_ARG;
  const int e = mt::dtype_bytes(g->dtype), ew = g->weight_dtype == MT_DTYPE_F32 ? 4 : e;
  const int64_t rows = g->rows, d = g->d;
  const View dy{g->dy, rows, d, g->lddy, e}, h{g->h, rows, d, g->ldh, e};
  const View dx{g->dx, rows, d, g->lddx, e};
  const View w = vector(g->weight, d, ew);
  const View mean{g->mean, rows, 1, 1, 4}, rstd{g->rstd, rows, 1, 1, 4};
  const View dh = optional(g->dh, rows, d, g->lddh, e);
  const View dres = optional(g->dresidual, rows, d, g->lddres, e);
  const View dw = vector(g->dweight, d, 4), db = vector(g->dbias, d, 4);
  const View seed = seed_view(g->seed, drop);
  for (const View* v : {&dy, &h, &dx, &w, &mean, &rstd, &dh, &dres, &dw, &db, &seed})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  for (const View* out : {&dx, &dres})
    for (const View* in : {&dy, &dh})
      if (out->hits(*in) && !out->same(*in)) return MT_ERR_ALIAS;
  for (const View* out : {&dx, &dres, &dw, &db})
    for (const View* in : {&h, &w, &mean, &rstd, &seed})
      if (out->hits(*in)) return MT_ERR_ALIAS;
  for (const View* out : {&dw, &db})
    for (const View* v : {&dx, &dres, &dy, &dh})
      if (out->hits(*v)) return MT_ERR_ALIAS;
  if (dx.hits(dres) || dw.hits(db)) return MT_ERR_ALIAS;
  if (d == 0 || (rows == 0 && !g->dweight && !g->dbias)) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  mt_status st = current_device(&dev, &info);
  if (st != MT_OK) return st;
  const mt::LayerNormGradArgs a{
      rows, static_cast<int>(d), g->dy, g->lddy, g->h, g->ldh, g->weight, g->mean, g->rstd, g->dh,
      g->lddh, g->dx, g->lddx, g->dresidual, g->lddres, g->dweight, g->dbias, g->dtype,
      ew == 4 ? 1 : 0, drop ? 1 : 0, dropout_args(g->seed, g->sequence, g->dropout),
      bounds_record(), g->fault_inject};
  Scratch ws(stream);
  st = ws.get(dev, mt::layer_norm_grad_workspace(a, info.sms));
  if (st != MT_OK) return st;
  return launched(mt::launch_layer_norm_grad(a, ws.p, info.sms, stream));
}

mt_status mt_dropout(const mt_dropout_args* g, cudaStream_t stream) {
  if (!g || !sizes_ok(g->rows, g->d) || !float_type(g->dtype) || g->reserved ||
      !probability(g->p))
    return MT_ERR_INVALID_ARG;
  const int e = mt::dtype_bytes(g->dtype);
  const int64_t rows = g->rows, d = g->d;
  const View x{g->x, rows, d, g->ldx, e}, y{g->y, rows, d, g->ldy, e};
  const View res = optional(g->residual, rows, d, g->ldr, e);
  const View seed = seed_view(g->seed, rows > 0 && d > 0);
  for (const View* v : {&x, &y, &res, &seed})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  if ((y.hits(x) && !y.same(x)) || (y.hits(res) && !y.same(res)) || y.hits(seed))
    return MT_ERR_ALIAS;
  if (rows == 0 || d == 0) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  const mt_status st = current_device(&dev, &info);
  if (st != MT_OK) return st;
  const mt::DropoutCall a{rows, static_cast<int>(d), g->x, g->ldx, g->residual, g->ldr, g->y,
                          g->ldy, g->dtype, dropout_args(g->seed, g->sequence, g->p),
                          bounds_record()};
  return launched(mt::launch_dropout(a, info.sms, stream));
}

mt_status mt_linear_cross_entropy(const mt_linear_cross_entropy_args* g, cudaStream_t stream) {
  if (!g || g->T < 0 || g->K < 0 || g->V < 0 || g->T > kMaxSize || g->K > kMaxSize ||
      g->V > kMaxSize || !half_type(g->dtype) || g->trans_b < 0 || g->trans_b > 1 ||
      g->fault_inject < 0 || g->fault_inject > 1 || g->reserved)
    return MT_ERR_INVALID_ARG;
  if (!(g->label_smoothing >= 0.0f && g->label_smoothing <= 1.0f) || !(g->z_loss >= 0.0f) ||
      std::isinf(g->z_loss))
    return MT_ERR_INVALID_ARG;
  const int64_t T = g->T, K = g->K, V = g->V;
  if (T > 0 && V == 0) return MT_ERR_INVALID_ARG;
  const View A{g->A, T, K, g->lda, 2};
  const View B = g->trans_b ? View{g->B, V, K, g->ldb, 2} : View{g->B, K, V, g->ldb, 2};
  const View target{g->target, 1, T, INT32_MAX, 8};
  const View loss{g->loss, 1, T, INT32_MAX, 4}, lse{g->lse, 1, T, INT32_MAX, 4};
  for (const View* v : {&A, &B, &target, &loss, &lse})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  for (const View* v : {&A, &B, &target})
    if (loss.hits(*v) || lse.hits(*v)) return MT_ERR_ALIAS;
  if (loss.hits(lse)) return MT_ERR_ALIAS;
  if (T == 0) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  mt_status st = current_device(&dev, &info);
  if (st == MT_OK) st = prepare_loss(dev);
  if (st != MT_OK) return st;
  const mt::HeadLossArgs a{T, K, V, g->A, g->lda, g->B, g->ldb, g->trans_b ? 0 : 1, g->target,
                           g->ignore_index, g->label_smoothing, g->z_loss, g->dtype,
                           bounds_record()};
  const mt::HeadLossPlan p = mt::plan_head_loss(a, info.sms);
  if (p.product.grid > INT32_MAX) return MT_ERR_UNSUPPORTED;
  Scratch ws(stream);
  st = ws.get(dev, p.workspace_bytes);
  if (st != MT_OK) return st;
  return launched(mt::launch_head_loss(a, p, g->loss, g->lse, ws.p, info.sms, g->fault_inject,
                                       stream));
}

mt_status mt_linear_cross_entropy_backward(const mt_linear_cross_entropy_backward_args* g,
                                           cudaStream_t stream) {
  if (!g || g->T < 0 || g->K < 0 || g->V < 0 || g->T > kMaxSize || g->K > kMaxSize ||
      g->V > kMaxSize || !half_type(g->dtype) || g->trans_b < 0 || g->trans_b > 1 ||
      (g->db_dtype != g->dtype && g->db_dtype != MT_DTYPE_F32) || g->reserved)
    return MT_ERR_INVALID_ARG;
  if (!(g->label_smoothing >= 0.0f && g->label_smoothing <= 1.0f) || !(g->z_loss >= 0.0f) ||
      std::isinf(g->z_loss))
    return MT_ERR_INVALID_ARG;
  const int64_t T = g->T, K = g->K, V = g->V;
  if (T > 0 && V == 0) return MT_ERR_INVALID_ARG;
  // As B is stored.
  auto like_b = [&](const void* p, int64_t ld, int elem, bool there) {
    return g->trans_b ? View{p, there ? V : 0, K, there ? ld : INT32_MAX, elem}
                      : View{p, there ? K : 0, V, there ? ld : INT32_MAX, elem};
  };
  const View dloss{g->dloss, 1, T, INT32_MAX, 4}, lse{g->lse, 1, T, INT32_MAX, 4};
  const View target{g->target, 1, T, INT32_MAX, 8};
  const View A{g->A, T, K, g->lda, 2}, B = like_b(g->B, g->ldb, 2, true);
  const View dA = optional(g->dA, T, K, g->ldda, 2);
  const View dB = like_b(g->dB, g->lddb, mt::dtype_bytes(g->db_dtype), g->dB != nullptr);
  for (const View* v : {&dloss, &lse, &target, &A, &B, &dA, &dB})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  for (const View* out : {&dA, &dB})
    for (const View* in : {&dloss, &lse, &target, &A, &B})
      if (out->hits(*in)) return MT_ERR_ALIAS;
  if (dA.hits(dB)) return MT_ERR_ALIAS;
  const bool want_a = g->dA && T > 0 && K > 0, want_b = g->dB && V > 0 && K > 0;
  if (!want_a && !want_b) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  mt_status st = current_device(&dev, &info);
  if (st == MT_OK) st = prepare_loss(dev);
  if (st != MT_OK) return st;
  const mt::HeadGradArgs a{
      {T, K, V, g->A, g->lda, g->B, g->ldb, g->trans_b ? 0 : 1, g->target, g->ignore_index,
       g->label_smoothing, g->z_loss, g->dtype, bounds_record()},
      g->dloss, g->lse, want_a ? g->dA : nullptr, g->ldda, want_b ? g->dB : nullptr, g->lddb,
      g->db_dtype};
  const mt::HeadGradPlan p = mt::plan_head_grad(a, info.sms);
  if (p.too_large) return MT_ERR_UNSUPPORTED;
  Scratch ws(stream);
  st = ws.get(dev, p.workspace_bytes);
  if (st != MT_OK) return st;
  return launched(mt::launch_head_grad(a, p, ws.p, info.sms, stream));
}

}  // extern "C"
