// C entry points of the feed-forward operators (include/mt_layers.h):
// argument checks, launch choices, scratch.
#include <atomic>
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>

#include <cuda_runtime.h>

#include "host.h"
#include "layers.h"
#include "mt_layers.h"

namespace {

using namespace mt::host;

static_assert(MT_DTYPE_F16 == mt::DT_F16 && MT_DTYPE_BF16 == mt::DT_BF16 &&
                  MT_DTYPE_F32 == mt::DT_F32 && MT_DTYPE_E4M3 == mt::DT_E4M3,
              "storage type codes");
static_assert(MT_ACT_RELU == mt::ACT_RELU && MT_ACT_GELU == mt::ACT_GELU &&
                  MT_ACT_GELU_TANH == mt::ACT_GELU_TANH && MT_ACT_SILU == mt::ACT_SILU,
              "activation codes");

// Largest row, column or contraction count of a product: tile coordinates
// past the edge stay inside 32 bits.
constexpr int64_t kMaxSize = INT32_MAX - 255;
// Longest row of a norm: the row-wise kernels step a 32-bit column by up to
// 512, and round the columns up to whole strips of 32.
constexpr int64_t kMaxRow = INT32_MAX - 511;

// A rows x cols view of `elem`-byte values with row pitch ld, for the checks.
struct View {
  const void* p;
  int64_t rows, cols, ld;
  int elem;

  int64_t bytes() const { return extent_bytes(rows, cols, ld, elem); }
  bool empty() const { return rows == 0 || cols == 0; }
  // The pitch holds a row, the span fits 64-bit offsets, and the pointer is
  // there and aligned to its element unless there is nothing to address.
  bool valid() const {
    if (ld < (cols > 1 ? cols : 1) || ld > INT64_MAX / 64) return false;
    if (rows > 0 && ld > INT64_MAX / 64 / rows) return false;
    if (empty()) return true;
    return p && (reinterpret_cast<uintptr_t>(p) & static_cast<uintptr_t>(elem - 1)) == 0;
  }
  bool same(const View& o) const { return p == o.p && ld == o.ld && elem == o.elem; }
  // Whether the views share a byte.  Columns of one wider buffer (the same
  // pitch) may lie side by side in spans that overlap; other pitches are
  // judged by their spans.
  bool hits(const View& o) const {
    if (!overlaps(p, bytes(), o.p, o.bytes())) return false;
    const int64_t pitch = ld * elem;
    if (rows < 2 || o.rows < 2 || o.ld * o.elem != pitch) return true;
    const int64_t apart = static_cast<const char*>(o.p) - static_cast<const char*>(p);
    const int64_t first = (apart % pitch + pitch) % pitch;  // o's column 0 in a row of this
    return first < cols * elem || first + o.cols * o.elem > pitch;
  }
};

// Scratch from the device's pool for one call; freed on the call's stream.
struct Scratch {
  void* p = nullptr;
  cudaStream_t stream;

  explicit Scratch(cudaStream_t s) : stream(s) {}
  Scratch(const Scratch&) = delete;
  Scratch& operator=(const Scratch&) = delete;
  ~Scratch() {
    if (p) cudaFreeAsync(p, stream);
  }
  mt_status get(int dev, int64_t bytes) {
    if (bytes <= 0) return MT_OK;
    cudaMemPool_t pool = nullptr;
    const mt_status st = pool_for(dev, &pool);
    if (st != MT_OK) return st;
    if (cudaMallocFromPoolAsync(&p, static_cast<size_t>(bytes), pool, stream) != cudaSuccess) {
      cudaGetLastError();
      p = nullptr;
      return MT_ERR_CUDA;
    }
    return MT_OK;
  }
};

bool half_type(int t) { return t == MT_DTYPE_F16 || t == MT_DTYPE_BF16; }

// The product an mt_linear call makes.
mt::LinearArgs product_of(const mt_linear_args& g) {
  mt::LinearArgs a{};
  a.T = g.M;
  a.C = g.N;
  a.K = g.K;
  a.X = g.A;
  a.ldx = g.lda;
  a.W = g.B;
  a.ldw = g.ldb;
  a.w_mn = g.trans_b ? 0 : 1;
  a.Y = g.Y;
  a.ldy = g.ldy;
  a.Z = g.Z;
  a.ldz = g.ldz;
  a.residual = g.residual;
  a.ldr = g.ldr;
  a.bias = g.bias;
  a.row_scale = g.scale_a;
  a.col_scale = g.scale_b;
  a.dtype = g.dtype;
  a.out_dtype = g.out_dtype;
  a.act = g.activation;
  a.bounds = bounds_record();
  return a;
}

bool linear_types_ok(const mt_linear_args& g) {
  const bool e4m3 = g.dtype == MT_DTYPE_E4M3;
  if (!half_type(g.dtype) && !e4m3) return false;
  if (g.out_dtype != MT_DTYPE_F32 && (e4m3 ? !half_type(g.out_dtype) : g.out_dtype != g.dtype))
    return false;
  if (g.trans_b < 0 || g.trans_b > 1 || (e4m3 && !g.trans_b)) return false;
  return g.activation >= MT_ACT_NONE && g.activation <= MT_ACT_SILU;
}

// The product kernels' shared-memory limits, set once per device.
std::mutex g_linear_mutex;
std::atomic<uint8_t> g_linear_ready[kMaxDevices];

mt_status prepare_linear(int dev) {
  if (!mt::tensor_map_encoder_available()) return MT_ERR_CUDA;
  if (g_linear_ready[dev].load(std::memory_order_acquire)) return MT_OK;
  std::lock_guard<std::mutex> lock(g_linear_mutex);
  if (mt::linear_prepare() != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_LAUNCH;
  }
  g_linear_ready[dev].store(1, std::memory_order_release);
  return MT_OK;
}

}  // namespace

extern "C" {

mt_status mt_rms_norm(const mt_rms_norm_args* g, cudaStream_t stream) {
  if (!g || g->rows < 0 || g->d < 0 || g->d > kMaxRow || g->rows > INT32_MAX)
    return MT_ERR_INVALID_ARG;
  if (!half_type(g->dtype) && g->dtype != MT_DTYPE_F32) return MT_ERR_INVALID_ARG;
  if (g->out_dtype != g->dtype && g->out_dtype != MT_DTYPE_E4M3) return MT_ERR_INVALID_ARG;
  if (g->weight && g->weight_dtype != g->dtype && g->weight_dtype != MT_DTYPE_F32)
    return MT_ERR_INVALID_ARG;
  if (!(g->eps >= 0.0f) || std::isinf(g->eps)) return MT_ERR_INVALID_ARG;
  const bool e4m3 = g->out_dtype == MT_DTYPE_E4M3;
  const int e = mt::dtype_bytes(g->dtype);
  const int64_t rows = g->rows, d = g->d;
  const View x{g->x, rows, d, g->ldx, e};
  const View res{g->residual, g->residual ? rows : 0, d, g->residual ? g->ldr : INT32_MAX, e};
  const View w{g->weight, g->weight ? 1 : 0, d, INT32_MAX, mt::dtype_bytes(g->weight_dtype)};
  const View h{g->h, g->h ? rows : 0, d, g->h ? g->ldh : INT32_MAX, e};
  const View y{g->y, rows, d, g->ldy, mt::dtype_bytes(g->out_dtype)};
  const View scale{g->scale, e4m3 ? rows : 0, 1, 1, 4};
  const View rstd{g->rstd, g->rstd ? rows : 0, 1, 1, 4};
  for (const View* v : {&x, &res, &w, &h, &y, &scale, &rstd})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  if (!e4m3 && g->scale) return MT_ERR_INVALID_ARG;
  if ((h.hits(x) && !h.same(x)) || (h.hits(res) && !h.same(res)) || (y.hits(x) && !y.same(x)) ||
      y.hits(res) || y.hits(h) || w.hits(h) || w.hits(y))
    return MT_ERR_ALIAS;
  for (const View* s : {&scale, &rstd})
    for (const View* v : {&x, &res, &w, &h, &y})
      if (s->hits(*v)) return MT_ERR_ALIAS;
  if (scale.hits(rstd)) return MT_ERR_ALIAS;
  if (rows == 0) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  const mt_status st = current_device(&dev, &info);
  if (st != MT_OK) return st;
  const mt::RmsNormArgs a{rows, static_cast<int>(d), g->x, g->ldx, g->residual, g->ldr,
                          g->weight, g->h, g->ldh, g->y, g->ldy, g->scale, g->rstd, g->eps,
                          g->dtype, e4m3 ? 1 : 0, g->weight_dtype == MT_DTYPE_F32 ? 1 : 0,
                          bounds_record()};
  if (mt::launch_rms_norm(a, stream) != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_LAUNCH;
  }
  return MT_OK;
}

mt_status mt_rms_norm_backward(const mt_rms_norm_backward_args* g, cudaStream_t stream) {
  if (!g || g->rows < 0 || g->d < 0 || g->d > kMaxRow || g->rows > INT32_MAX)
    return MT_ERR_INVALID_ARG;
  if (!half_type(g->dtype) && g->dtype != MT_DTYPE_F32) return MT_ERR_INVALID_ARG;
  if (g->reserved || g->fault_inject < 0 || g->fault_inject > 1) return MT_ERR_INVALID_ARG;
  if (g->weight && g->weight_dtype != g->dtype && g->weight_dtype != MT_DTYPE_F32)
    return MT_ERR_INVALID_ARG;
  const int e = mt::dtype_bytes(g->dtype);
  const int64_t rows = g->rows, d = g->d;
  const View dy{g->dy, rows, d, g->lddy, e}, h{g->h, rows, d, g->ldh, e};
  const View w{g->weight, g->weight ? 1 : 0, d, INT32_MAX, mt::dtype_bytes(g->weight_dtype)};
  const View rstd{g->rstd, rows, 1, 1, 4};
  const View dh{g->dh, g->dh ? rows : 0, d, g->dh ? g->lddh : INT32_MAX, e};
  const View dx{g->dx, rows, d, g->lddx, e};
  const View dw{g->dweight, g->dweight ? 1 : 0, d, INT32_MAX, 4};
  for (const View* v : {&dy, &h, &w, &rstd, &dh, &dx, &dw})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  if ((dx.hits(dy) && !dx.same(dy)) || (dx.hits(dh) && !dx.same(dh))) return MT_ERR_ALIAS;
  for (const View* v : {&h, &w, &rstd})
    if (v->hits(dx) || v->hits(dw)) return MT_ERR_ALIAS;
  if (dw.hits(dx) || dw.hits(dy) || dw.hits(dh)) return MT_ERR_ALIAS;
  if (d == 0 || (rows == 0 && !g->dweight)) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  mt_status st = current_device(&dev, &info);
  if (st != MT_OK) return st;
  const mt::RmsNormGradArgs a{rows, static_cast<int>(d), g->dy, g->lddy, g->h, g->ldh, g->weight,
                              g->rstd, g->dh, g->lddh, g->dx, g->lddx, g->dweight, g->dtype,
                              g->weight_dtype == MT_DTYPE_F32 ? 1 : 0, bounds_record(),
                              g->fault_inject};
  Scratch ws(stream);
  st = ws.get(dev, mt::rms_norm_grad_workspace(a, info.sms));
  if (st != MT_OK) return st;
  if (mt::launch_rms_norm_grad(a, ws.p, info.sms, stream) != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_LAUNCH;
  }
  return MT_OK;
}

mt_status mt_linear(const mt_linear_args* g, cudaStream_t stream) {
  if (!g || g->M < 0 || g->N < 0 || g->K < 0 || g->M > kMaxSize || g->N > kMaxSize ||
      g->K > kMaxSize || g->reserved || g->fault_inject < 0 || g->fault_inject > 1 ||
      !linear_types_ok(*g))
    return MT_ERR_INVALID_ARG;
  const bool e4m3 = g->dtype == MT_DTYPE_E4M3;
  const int e = mt::dtype_bytes(g->dtype), eo = mt::dtype_bytes(g->out_dtype);
  const int64_t M = g->M, N = g->N, K = g->K;
  if (!e4m3 && (g->scale_a || g->scale_b)) return MT_ERR_INVALID_ARG;
  const View A{g->A, M, K, g->lda, e};
  const View B = g->trans_b ? View{g->B, N, K, g->ldb, e} : View{g->B, K, N, g->ldb, e};
  const View Y{g->Y, M, N, g->ldy, eo};
  const View Z{g->Z, g->Z ? M : 0, N, g->Z ? g->ldz : INT32_MAX, eo};
  const View res{g->residual, g->residual ? M : 0, N, g->residual ? g->ldr : INT32_MAX, eo};
  const View bias{g->bias, g->bias ? 1 : 0, N, INT32_MAX, 4};
  const View sa{g->scale_a, e4m3 ? 1 : 0, M, INT32_MAX, 4};
  const View sb{g->scale_b, e4m3 ? 1 : 0, N, INT32_MAX, 4};
  for (const View* v : {&A, &B, &Y, &Z, &res, &bias, &sa, &sb})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  for (const View* v : {&A, &B, &bias, &sa, &sb})
    if (Y.hits(*v) || Z.hits(*v)) return MT_ERR_ALIAS;
  if ((Y.hits(res) && !Y.same(res)) || Z.hits(res) || Z.hits(Y)) return MT_ERR_ALIAS;
  if (M == 0 || N == 0) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  mt_status st = current_device(&dev, &info);
  if (st == MT_OK) st = prepare_linear(dev);
  if (st != MT_OK) return st;
  const mt::LinearArgs a = product_of(*g);
  const mt::LinearPlan p = mt::plan_linear(a, info.sms);
  if (p.grid > INT32_MAX) return MT_ERR_UNSUPPORTED;
  Scratch ws(stream);
  st = ws.get(dev, p.workspace_bytes);
  if (st != MT_OK) return st;
  if (mt::launch_linear(a, p, ws.p, stream, g->fault_inject) != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_LAUNCH;
  }
  return MT_OK;
}

mt_status mt_linear_plan(const mt_linear_args* g, int sms, mt_plan* out) {
  if (!g || !out || sms < 1 || g->M < 1 || g->N < 1 || g->K < 0 || g->M > kMaxSize ||
      g->N > kMaxSize || g->K > kMaxSize || !linear_types_ok(*g))
    return MT_ERR_INVALID_ARG;
  const mt::LinearPlan p = mt::plan_linear(product_of(*g), sms);
  if (p.grid > INT32_MAX) return MT_ERR_UNSUPPORTED;
  std::memset(out, 0, sizeof(*out));
  out->variant = MT_VARIANT_TC16;
  out->bm = p.bt;
  out->bn = p.bc;
  out->bk = 128 / mt::dtype_bytes(g->dtype);
  out->stages = p.stages;
  out->threads = p.threads;
  out->vec_ab = p.workspace_bytes == 0;
  out->split_k = p.split;
  out->grid = p.grid;
  out->smem_bytes = p.smem_bytes;
  out->workspace_bytes = p.workspace_bytes;
  return MT_OK;
}

mt_status mt_linear_backward(const mt_linear_backward_args* g, cudaStream_t stream) {
  if (!g || g->M < 0 || g->N < 0 || g->K < 0 || g->M > kMaxSize || g->N > kMaxSize ||
      g->K > kMaxSize || g->trans_b < 0 || g->trans_b > 1 || !half_type(g->dtype) ||
      (g->db_dtype != g->dtype && g->db_dtype != MT_DTYPE_F32) ||
      g->activation < MT_ACT_NONE || g->activation > MT_ACT_SILU)
    return MT_ERR_INVALID_ARG;
  const int64_t M = g->M, N = g->N, K = g->K;
  const bool act = g->activation != MT_ACT_NONE;
  // A B stored K x N, or N x K; rows == 0 for what is not there or not read.
  auto like_b = [&](const void* p, int64_t ld, int elem, bool used) {
    return g->trans_b ? View{p, used ? N : 0, K, used ? ld : INT32_MAX, elem}
                      : View{p, used ? K : 0, N, used ? ld : INT32_MAX, elem};
  };
  const View dY{g->dY, M, N, g->lddy, 2};
  const View Z{g->Z, act ? M : 0, N, act ? g->ldz : INT32_MAX, 2};
  const View A{g->A, g->dB ? M : 0, K, g->dB ? g->lda : INT32_MAX, 2};
  const View B = like_b(g->B, g->ldb, 2, g->dA != nullptr);
  const View dA{g->dA, g->dA ? M : 0, K, g->dA ? g->ldda : INT32_MAX, 2};
  const View dB = like_b(g->dB, g->lddb, mt::dtype_bytes(g->db_dtype), g->dB != nullptr);
  const View db{g->dbias, g->dbias ? 1 : 0, N, INT32_MAX, 4};
  for (const View* v : {&dY, &Z, &A, &B, &dA, &dB, &db})
    if (!v->valid()) return MT_ERR_INVALID_ARG;
  for (const View* out : {&dA, &dB, &db})
    for (const View* in : {&dY, &Z, &A, &B})
      if (out->hits(*in)) return MT_ERR_ALIAS;
  if (dA.hits(dB) || dA.hits(db) || dB.hits(db)) return MT_ERR_ALIAS;
  const bool want_a = g->dA && M > 0 && K > 0, want_b = g->dB && N > 0 && K > 0;
  const bool want_bias = g->dbias && N > 0;
  if (!want_a && !want_b && !want_bias) return MT_OK;
  int dev = 0;
  DeviceInfo info;
  mt_status st = current_device(&dev, &info);
  if (st == MT_OK) st = prepare_linear(dev);
  if (st != MT_OK) return st;

  // dz, in rows of whole 128-byte lines, unless dY serves as it is.
  const bool products = (want_a || want_b) && M > 0 && N > 0;
  const bool make_dz = products && (act || !mt::tma_readable(g->dY, g->lddy, 2));
  const int64_t lddz = ceil_div(N, 64) * 64;
  const int64_t dz_bytes = make_dz ? ceil_div(M * lddz * 2, 256) * 256 : 0;
  mt::LinearDzArgs dz{M, static_cast<int>(N), g->dY, g->lddy, g->Z, g->ldz, nullptr, lddz,
                      want_bias ? g->dbias : nullptr, g->dtype, g->activation, bounds_record()};
  const int64_t sum_bytes = ceil_div(mt::linear_dz_workspace(dz, info.sms), 256) * 256;

  mt::LinearArgs pa{}, pb{};
  pa.dtype = pb.dtype = g->dtype;
  pa.out_dtype = g->dtype;
  pb.out_dtype = g->db_dtype;
  pa.act = pb.act = mt::ACT_NONE;
  pa.bounds = pb.bounds = bounds_record();
  // dA = dz * B^T: rows of dz against B's columns k, contracted over n.
  pa.T = M;
  pa.C = K;
  pa.K = N;
  pa.W = g->B;
  pa.ldw = g->ldb;
  pa.w_mn = g->trans_b;
  pa.Y = g->dA;
  pa.ldy = g->ldda;
  // dB as B is stored, contracted over rows: A^T * dz, or dz^T * A.
  pb.T = g->trans_b ? N : K;
  pb.C = g->trans_b ? K : N;
  pb.K = M;
  pb.x_mn = pb.w_mn = 1;
  pb.Y = g->dB;
  pb.ldy = g->lddb;

  // The scratch of the products follows; the plans look at the operands'
  // alignment, which scratch addresses (256-byte aligned) do not change.
  auto bind = [&](const void* dzp, int64_t ld) {
    pa.X = dzp;
    pa.ldx = ld;
    pb.X = g->trans_b ? dzp : g->A;
    pb.ldx = g->trans_b ? ld : g->lda;
    pb.W = g->trans_b ? g->A : dzp;
    pb.ldw = g->trans_b ? g->lda : ld;
  };
  bind(make_dz ? nullptr : g->dY, make_dz ? lddz : g->lddy);
  mt::LinearPlan plan_a{}, plan_b{};
  // Planned as if both were wanted: a gradient's bits do not depend on which
  // others are asked for.
  if (M > 0 && N > 0 && K > 0) mt::plan_linear_two(pa, pb, info.sms, &plan_a, &plan_b);
  else if (want_a) plan_a = mt::plan_linear(pa, info.sms);
  else if (want_b) plan_b = mt::plan_linear(pb, info.sms);
  if (!want_a) plan_a.workspace_bytes = 0;
  if (!want_b) plan_b.workspace_bytes = 0;
  if (plan_a.grid > INT32_MAX || plan_b.grid > INT32_MAX) return MT_ERR_UNSUPPORTED;
  Scratch ws(stream);
  st = ws.get(dev, dz_bytes + sum_bytes + plan_a.workspace_bytes + plan_b.workspace_bytes);
  if (st != MT_OK) return st;
  char* base = static_cast<char*>(ws.p);
  if (make_dz) {
    dz.dZ = base;
    bind(base, lddz);
  }
  cudaError_t e = cudaSuccess;
  if (make_dz || want_bias) e = mt::launch_linear_dz(dz, base + dz_bytes, info.sms, stream);
  char* wa = base + dz_bytes + sum_bytes;
  char* wb = wa + plan_a.workspace_bytes;
  if (e == cudaSuccess && want_a && want_b)
    e = mt::launch_linear_two(pa, plan_a, wa, pb, plan_b, wb, stream);
  else if (e == cudaSuccess && want_a)
    e = mt::launch_linear(pa, plan_a, wa, stream);
  else if (e == cudaSuccess && want_b)
    e = mt::launch_linear(pb, plan_b, wb, stream);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return MT_ERR_LAUNCH;
  }
  return MT_OK;
}

}  // extern "C"
