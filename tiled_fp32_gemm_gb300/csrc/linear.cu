// Host side of the fused linear layer: padded copies of operands TMA cannot
// read in place, the choice of kernel and its launch.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda.h>
#include <cuda_runtime.h>

#include "head.cuh"
#include "layers.h"
#include "linear.cuh"
#include "tcgen05.cuh"

namespace mt {
namespace {

using namespace linear;

constexpr int kRowBytes = 128;  // K of one staged tile row, in bytes
constexpr int kThreads = 192, kPairThreads = 320;
constexpr int kPair = 256;      // columns and rows of Y per CTA pair

// Padded copies of operands TMA cannot read in place (row pitch not a
// multiple of 16 bytes, or base not 16-byte aligned): rows of `pitch` bytes (a
// multiple of 16), the bytes past `bytes` zero.  Source rows start on any
// element, so an output's 16 bytes straddle two aligned 16-byte words of the
// source: both are read (a neighbour's are found in L1) and shifted into
// place.  Words that reach outside the source are read byte by byte.
struct CopyJob {
  const uint8_t* src;
  int64_t pitch_src, bytes, extent;  // bytes: of a row, of the whole source
  uint8_t* dst;
  int64_t pitch;
  int rows;
  int first_block, blocks, row_threads;  // threads side by side on a row
};
struct CopyJobs {
  CopyJob job[2];
  BoundsRecord* rec;
  int count, blocks;
};

constexpr int kCopyThreads = 256;

template <int BATCH>
__global__ void __launch_bounds__(kCopyThreads) copy_rows_kernel(const CopyJobs jobs) {
  grid_launch_dependents();
  grid_wait();
  const CopyJob& j = jobs.job[static_cast<int>(blockIdx.x) >= jobs.job[1].first_block ? 1 : 0];
  const int x0 = threadIdx.x % j.row_threads, row_step = kCopyThreads / j.row_threads;
  const int chunks = static_cast<int>(j.pitch / 16);
  const int64_t first = static_cast<int64_t>(blockIdx.x - j.first_block) * row_step +
                        threadIdx.x / j.row_threads;
  const int64_t step = static_cast<int64_t>(j.blocks) * row_step;
  // BATCH words, `down` rows and `right` words apart; the loads of all of them
  // are in flight before the first is stored.
  auto batch = [&](int64_t r0, int xw, int64_t down, int right) {
    uint4 lo[BATCH], hi[BATCH];
    int shift[BATCH];  // -1: byte by byte
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int64_t r = r0 + k * down, c0 = 16 * static_cast<int64_t>(xw + k * right);
      const int64_t at = r * j.pitch_src + c0;
      shift[k] = -1;
      if (r >= j.rows || c0 >= j.bytes) continue;
      const int s = static_cast<int>(reinterpret_cast<uintptr_t>(j.src + at) & 15u);
      if (at < s || at - s + 32 > j.extent) continue;
      const uint4* p = reinterpret_cast<const uint4*>(j.src + (at - s));
      lo[k] = p[0];
      hi[k] = p[1];
      shift[k] = s;
    }
#pragma unroll
    for (int k = 0; k < BATCH; ++k) {
      const int64_t r = r0 + k * down, c0 = 16 * static_cast<int64_t>(xw + k * right);
      const int64_t at = r * j.pitch_src + c0, to = r * j.pitch + c0;
      const int left = static_cast<int>(min(int64_t(16), j.bytes - c0));  // of the row, or < 0
      if (r >= j.rows || c0 >= j.pitch) break;
      uint32_t o[4] = {0u, 0u, 0u, 0u};
      if (shift[k] >= 0) {
        const uint4 u = row::shifted(lo[k], hi[k], shift[k]);
        o[0] = u.x, o[1] = u.y, o[2] = u.z, o[3] = u.w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int keep = left - 4 * i;  // bytes of this word inside the row
          if (keep < 4) o[i] = keep <= 0 ? 0u : o[i] & ((1u << (8 * keep)) - 1u);
        }
      } else if (left > 0) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i < left && bounds_ok(jobs.rec, SITE_PREP_SRC, at + i, 1, j.extent))
            o[i / 4] |= static_cast<uint32_t>(j.src[at + i]) << (8 * (i % 4));
      }
      if (bounds_ok(jobs.rec, SITE_PREP_DST, to, 16, j.rows * j.pitch))
        *reinterpret_cast<uint4*>(j.dst + to) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  };
  // A batch goes along a row past 16 KB and from row to row in others, a column of
  // words at a time.  Measured (us for a loss with the copy, along / from row to row):
  // 2160 rows of 60 KB 84 / 114, 110304 of 0.7 KB 79 / 59.
  if (BATCH == 1 || chunks > 1024) {
    for (int64_t r = first; r < j.rows; r += step)
      for (int x = x0; x < chunks; x += BATCH * j.row_threads) batch(r, x, 0, j.row_threads);
  } else {
    for (int x = x0; x < chunks; x += j.row_threads)
      for (int64_t r = first; r < j.rows; r += BATCH * step) batch(r, x, step, 0);
  }
}

// The stored matrix of an operand: rows and columns in memory.
struct Stored {
  const void* p;
  int64_t rows, cols, ld;
};
Stored stored_x(const LinearArgs& a) {
  return a.x_mn ? Stored{a.X, a.K, a.T, a.ldx} : Stored{a.X, a.T, a.K, a.ldx};
}
Stored stored_w(const LinearArgs& a) {
  return a.w_mn ? Stored{a.W, a.K, a.C, a.ldw} : Stored{a.W, a.C, a.K, a.ldw};
}

int64_t copy_pitch_bytes(int64_t cols, int elem) { return (cols * elem + 127) / 128 * 128; }

int64_t copy_bytes(const Stored& m, int elem) {
  if (tma_readable(m.p, m.ld, elem)) return 0;
  return (m.rows * copy_pitch_bytes(m.cols, elem) + 255) / 256 * 256;
}

// The copy of *m into dst, which *m then stands for.
CopyJob copy_job(Stored* m, int elem, void* dst, int first_block) {
  CopyJob j{};
  j.src = static_cast<const uint8_t*>(m->p);
  j.pitch_src = m->ld * elem;
  j.bytes = m->cols * elem;
  j.extent = view_extent(m->rows, m->cols, m->ld) * elem;
  j.dst = static_cast<uint8_t*>(dst);
  j.pitch = copy_pitch_bytes(m->cols, elem);
  j.rows = static_cast<int>(m->rows);
  j.first_block = first_block;
  j.row_threads = 8;
  while (j.row_threads < kCopyThreads && j.row_threads * 16 < j.pitch) j.row_threads *= 2;
  const int64_t rows_per_block = kCopyThreads / j.row_threads;
  j.blocks = static_cast<int>(
      std::min<int64_t>(2432, (m->rows + rows_per_block - 1) / rows_per_block));
  m->p = dst;
  m->ld = j.pitch / elem;
  return j;
}

bool encode(CUtensorMap* map, int dtype, const Stored& m, bool mn, int rows) {
  const CUtensorMapDataType t = dtype == DT_E4M3   ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                : dtype == DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int elem = dtype_bytes(dtype);
  return mn ? encode_tensor_map_2d(map, t, elem, m.p, m.rows, m.cols, m.ld, 64, 64,
                                   CU_TENSOR_MAP_SWIZZLE_128B)
            : encode_tensor_map_2d(map, t, elem, m.p, m.rows, m.cols, m.ld, 128 / elem,
                                   rows, CU_TENSOR_MAP_SWIZZLE_128B);
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// CTAs that share a tile's K, each at least four K tiles.  Two CTAs fit an SM
// (clusters of 3 or 4 reach nine tenths of those places, clusters of 8 three
// quarters); a second round of CTAs costs more than slices gain, and past
// four slices the clusters' barriers cost more than they save unless a CTA
// has an SM to itself.  Measured (bf16, one token, weight N x K, us by
// slices 1 / 2 / 4 / 8): 8192 x 4096 20.3 / 16.2 / 15.2 / 23.5; 4096 x 4096
// 19.9 / 13.5 / 10.9 / 12.1; 19456 x 4096 28.1 / 27.4 / 38.2 / 53.6;
// 1024 x 1024 6.6 / 5.9 / 5.6 / 6.9; 128 x 8192 36.1 / 21.2 / 13.2 / 10.4.
int split_of(int64_t tiles, int64_t ktiles, int sms) {
  const int64_t most = ktiles / 4;
  if (most >= 8 && tiles * 8 <= sms * 3 / 4) return 8;
  for (int s = 4; s > 1; --s)
    if (s <= most && tiles * s <= (s > 2 ? 2 * sms * 9 / 10 : 2 * sms)) return s;
  return 1;
}

int64_t ktiles_of(const LinearArgs& a) {
  return ceil_div(a.K * dtype_bytes(a.dtype), kRowBytes);
}
int64_t split_tiles(const LinearArgs& a, int bt) {
  return ceil_div(a.C, LINEAR_BC) * ceil_div(a.T, bt);
}

// A split-kernel plan with `split` CTAs to a tile in clusters of `cluster`.
void use_split(const LinearArgs& a, int bt, int split, int cluster, LinearPlan* p) {
  const LinearKernel k = linear_split_kernel_for(a.dtype, bt);
  p->pair = 0;
  p->bt = bt;
  p->bc = LINEAR_BC;
  p->threads = kThreads;
  p->split = split;
  p->cluster = cluster;
  p->stages = k.stages;
  p->smem_bytes = k.smem;
  p->grid = ceil_div(split_tiles(a, bt) * split, cluster) * cluster;
}

}  // namespace

bool tma_readable(const void* p, int64_t ld, int elem) {
  return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && ld * elem % 16 == 0 &&
         ld * elem < (int64_t(1) << 39);
}

LinearPlan plan_linear(const LinearArgs& a, int sms) { return plan_linear(a, sms, 2 * sms); }

LinearPlan plan_linear(const LinearArgs& a, int sms, int sevenths) {
  LinearPlan p{};
  const int elem = dtype_bytes(a.dtype);
  const int64_t pairs = ceil_div(a.C, kPair) * ceil_div(a.T, kPair);
  // CTA pairs when their tiles fill two sevenths of the GPU's SMs, and with
  // tokens, not padding (and the kernel's tile indices are 32-bit).  Measured
  // (bf16, gelu, bias and residual, N = K = 4096, us for pairs against the
  // split kernel): 512 tokens (32 pairs) 32.0 / 28.0, 768 (48) 33.1 / 38.5,
  // 1024 (64) 33.2 / 39.0, 2048 (128) 55.1 / 74.7; e4m3 512 tokens 23.9 / 21.5,
  // 768 25.2 / 27.1, 2048 38.8 / 52.4.
  p.pair = a.K > 0 && sms >= 2 && 7 * pairs >= sevenths && a.T > 128 &&
           pairs <= INT32_MAX / 8;
  if (p.pair) {
    const LinearKernel k = linear_pair_kernel_for(a.dtype, a.w_mn, a.x_mn);
    p.threads = kPairThreads;
    p.bt = p.bc = kPair;
    p.split = 1;
    p.cluster = 2;
    p.stages = k.stages;
    p.smem_bytes = k.smem;
    p.grid = 2 * std::min<int64_t>(pairs, sms / 2);
  } else {
    const int bt = a.T <= 16 && !a.x_mn ? 16 : a.T <= 32 && !a.x_mn ? 32 : a.T <= 64 ? 64 : 128;
    const int split = split_of(split_tiles(a, bt), ktiles_of(a), sms);
    use_split(a, bt, split, split, &p);
  }
  p.copy_x_bytes = a.K > 0 ? copy_bytes(stored_x(a), elem) : 0;
  p.copy_w_bytes = a.K > 0 ? copy_bytes(stored_w(a), elem) : 0;
  p.workspace_bytes = p.copy_x_bytes + p.copy_w_bytes;
  return p;
}

void plan_linear_two(const LinearArgs& a, const LinearArgs& b, int sms, LinearPlan* pa,
                     LinearPlan* pb) {
  *pa = plan_linear(a, sms);
  *pb = plan_linear(b, sms);
  // Two products that fill the GPU by pairs run one after the other; one that
  // has fewer pairs than the GPU has SMs joins the other's launch instead
  // (128 x 2048 x 4096, 128 pairs: 29.9 us apart, 26.0 together).
  if (pa->pair && pb->pair) return;
  const LinearArgs& paired = pa->pair ? a : b;
  if ((pa->pair || pb->pair) && ceil_div(paired.C, kPair) * ceil_div(paired.T, kPair) >= sms)
    return;
  const int bt = std::max(pa->pair ? 128 : pa->bt, pb->pair ? 128 : pb->bt);
  const int64_t ta = split_tiles(a, bt), tb = split_tiles(b, bt);
  const int64_t ka = ktiles_of(a), kb = ktiles_of(b);
  // The cluster: the most CTAs (of at least four K tiles each) that the split
  // product or products find places for beside the other, or, where one
  // contraction is four times the other's, beside its own tiles alone: else
  // 527 x 4472 x 512, whose gradients contract over 4472 and over 527, would
  // wait for 20 CTAs with 70 K tiles each.
  auto slices = [](int64_t k, int s) { return k >= 4 * s ? s : 1; };
  int cluster = 1;
  for (int s : {8, 4, 3, 2}) {
    const int64_t places = s == 8 ? sms * 3 / 4 : s > 2 ? 2 * sms * 9 / 10 : 2 * sms;
    const int64_t ca = ta * slices(ka, s), cb = tb * slices(kb, s);
    const bool lone = std::max(ka, kb) >= 4 * std::min(ka, kb) && s < 8;
    if (std::max(ka, kb) >= 4 * s &&
        (ca + cb <= places || (lone && (ka > kb ? ca : cb) <= places))) {
      cluster = s;
      break;
    }
  }
  use_split(a, bt, slices(ka, cluster), cluster, pa);
  use_split(b, bt, slices(kb, cluster), cluster, pb);
}

cudaError_t linear_prepare() {
  auto prepare = [](const LinearKernel& k) {
    if (!k.kernel) return cudaSuccess;
    cudaError_t r =
        cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    // Two CTAs of the split kernel share an SM.
    if (r == cudaSuccess)
      r = cudaFuncSetAttribute(k.kernel, cudaFuncAttributePreferredSharedMemoryCarveout,
                               cudaSharedmemCarveoutMaxShared);
    return r;
  };
  cudaError_t r = cudaSuccess;
  for (int dtype : {DT_F16, DT_E4M3}) {
    for (int bt : {16, 32, 64, 128})
      if (r == cudaSuccess) r = prepare(linear_split_kernel_for(dtype, bt));
    for (int mn = 0; mn < 4; ++mn)
      if (r == cudaSuccess) r = prepare(linear_pair_kernel_for(dtype, mn & 1, mn >> 1));
  }
  return r;
}

namespace {

// A product ready to launch: its operands in a form TMA reads.
struct Ready {
  CUtensorMap map_w, map_x;
  LinearEpilogue ep;
  uint32_t idesc;
};

// Adds the copies of what TMA cannot read in place and encodes the maps.
cudaError_t make_ready(const LinearArgs& a, const LinearPlan& p, void* workspace, CopyJobs* jobs,
                       Ready* out) {
  const int elem = dtype_bytes(a.dtype);
  Stored x = stored_x(a), w = stored_w(a);
  char* ws = static_cast<char*>(workspace);
  jobs->rec = a.bounds;
  auto add = [&](Stored* m, void* dst) {
    jobs->job[jobs->count] = copy_job(m, elem, dst, jobs->blocks);
    jobs->blocks += jobs->job[jobs->count++].blocks;
  };
  if ((p.copy_x_bytes != 0) + (p.copy_w_bytes != 0) + jobs->count > 2)
    return cudaErrorInvalidValue;
  if (p.copy_x_bytes) add(&x, ws);
  if (p.copy_w_bytes) add(&w, ws + p.copy_x_bytes);
  // A pair's CTAs load half a tile of each operand; without a product (K = 0)
  // the maps are not read.
  const int box_w = p.pair ? kPair / 2 : p.bc, box_x = p.pair ? kPair / 2 : p.bt;
  if (a.K > 0 && (!encode(&out->map_w, a.dtype, w, a.w_mn, box_w) ||
                  !encode(&out->map_x, a.dtype, x, a.x_mn, box_x)))
    return cudaErrorInvalidValue;
  const uint32_t fmt = a.dtype == DT_BF16 ? 1u : 0u;  // f16 0, bf16 1; e4m3 0
  out->idesc = tc::instr_desc(p.bc, p.bt, fmt, fmt, a.w_mn ? 1u : 0u, a.x_mn ? 1u : 0u);
  out->ep = LinearEpilogue{a.Y, a.ldy, a.Z, a.ldz, a.residual, a.ldr, a.bias, a.row_scale,
                           a.col_scale, static_cast<int>(a.T), static_cast<int>(a.C),
                           a.out_dtype, a.act, a.bounds};
  return cudaSuccess;
}

cudaError_t launch_copies(CopyJobs* jobs, cudaStream_t stream) {
  if (jobs->count == 0) return cudaSuccess;
  if (jobs->count == 1) jobs->job[1].first_block = INT32_MAX;
  // Eight words a thread and more are loaded four at a time, fewer one by one: the
  // batch's 80 registers let three blocks share an SM, the single word's 38 six.  Measured
  // (us with the product or loss that follows, batched / single): 2 words a thread 73.5 / 64.5
  // (4097 and 2053 fp16 rows of 3001), 5 words 36.0 / 33.6, 8.5 words 59.8 / 65.0, 49 words
  // 240 / 260.
  int64_t words = 0;
  for (int i = 0; i < jobs->count; ++i) words += jobs->job[i].rows * (jobs->job[i].pitch / 16);
  const bool batched = words >= 8 * static_cast<int64_t>(jobs->blocks) * kCopyThreads;
  return launch_dependent(batched ? copy_rows_kernel<4> : copy_rows_kernel<1>,
                          dim3(static_cast<unsigned>(jobs->blocks)), kCopyThreads, stream, *jobs);
}

template <class Ep>
SplitProblemOf<Ep> problem_of(const LinearArgs& a, const LinearPlan& p, const Ready& r,
                              const Ep& ep, int first_cta) {
  return SplitProblemOf<Ep>{r.map_w, r.map_x, ep, r.idesc, static_cast<int>(ktiles_of(a)),
                            static_cast<int>(split_tiles(a, p.bt)),
                            static_cast<int>(ceil_div(a.T, p.bt)), first_cta, p.split, a.w_mn,
                            a.x_mn};
}

template <class Ep>
cudaError_t launch_split(const LinearPlan& p, const LinearKernel& k, int64_t grid,
                         SplitProblemsOf<Ep>* problems, int fault_inject, cudaStream_t stream) {
  void* args[] = {problems, &fault_inject};
  return launch_dependent(k.kernel, dim3(static_cast<unsigned>(grid)), kThreads, p.smem_bytes,
                          p.cluster, stream, args);
}

// The map of a result that is written by boxes of 32 rows x 128 bytes; false
// where TMA cannot write it.
bool encode_boxes(CUtensorMap* map, int dtype, const void* p, int64_t rows, int64_t cols,
                  int64_t ld) {
  const CUtensorMapDataType t = dtype == DT_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : dtype == DT_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                  : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  const int elem = dtype_bytes(dtype);
  return tma_readable(p, ld, elem) &&
         encode_tensor_map_2d(map, t, elem, p, rows, cols, ld, 128 / elem, 32,
                              CU_TENSOR_MAP_SWIZZLE_128B);
}
bool encode_result(CUtensorMap* map, const LinearArgs& a) {
  return encode_boxes(map, a.out_dtype, a.Y, a.T, a.C, a.ldy);
}

// The MMA of pairs whose M side are the rows.
uint32_t pair_rows_idesc(const LinearArgs& a) {
  const uint32_t fmt = a.dtype == DT_BF16 ? 1u : 0u;
  return tc::instr_desc(kPair, kPair, fmt, fmt, a.x_mn ? 1u : 0u, a.w_mn ? 1u : 0u);
}

}  // namespace

int64_t padded_bytes(const PaddedCopy& c, int elem) {
  return copy_bytes(Stored{c.p, c.rows, c.cols, c.ld}, elem);
}

cudaError_t launch_padded_copies(PaddedCopy* const (&copies)[2], int elem, BoundsRecord* bounds,
                                 cudaStream_t stream) {
  CopyJobs jobs{};
  jobs.rec = bounds;
  for (PaddedCopy* c : copies) {
    if (!c || !c->dst) continue;
    Stored m{c->p, c->rows, c->cols, c->ld};
    jobs.job[jobs.count] = copy_job(&m, elem, c->dst, jobs.blocks);
    jobs.blocks += jobs.job[jobs.count++].blocks;
    c->p = m.p;
    c->ld = m.ld;
  }
  return launch_copies(&jobs, stream);
}

cudaError_t launch_linear(const LinearArgs& a, const LinearPlan& p, void* workspace,
                          cudaStream_t stream, int fault_inject) {
  Ready r{};
  CopyJobs jobs{};
  cudaError_t e = make_ready(a, p, workspace, &jobs, &r);
  if (e == cudaSuccess) e = launch_copies(&jobs, stream);
  if (e != cudaSuccess) return e;
  CUtensorMap map_y;
  if (p.pair && a.plain && encode_result(&map_y, a))
    return launch_linear_rows(a, r.map_x, r.map_w, map_y, pair_rows_idesc(a),
                              static_cast<int>(ktiles_of(a)), nullptr, false,
                              static_cast<int>(p.grid / 2), stream);
  if (p.pair)
    return launch_linear_pair(linear_pair_kernel_for(a.dtype, a.w_mn, a.x_mn), r.map_w, r.map_x,
                              r.idesc, r.ep, static_cast<int>(ktiles_of(a)),
                              static_cast<int>(p.grid / 2), fault_inject, stream);
  SplitProblems problems{};
  problems.p[0] = problem_of(a, p, r, r.ep, 0);
  problems.p[1].first_cta = INT32_MAX;
  return launch_split(p, linear_split_kernel_for(a.dtype, p.bt), p.grid, &problems, fault_inject,
                      stream);
}

// Slices of at least eight K tiles, as many as find pairs of SMs beside each
// other.
PlanesPlan plan_planes(const LinearArgs& a, int sms) {
  PlanesPlan p{};
  const int64_t tiles = ceil_div(a.T, kPair) * ceil_div(a.C, kPair), kt = ktiles_of(a);
  const int64_t want = std::min<int64_t>(sms / 2 / std::max<int64_t>(1, tiles), kt / 8);
  p.planes = static_cast<int>(std::max<int64_t>(1, want));
  p.kt_per_slice = static_cast<int>(ceil_div(kt, p.planes));
  p.planes = static_cast<int>(ceil_div(kt, p.kt_per_slice));
  p.rows = ceil_div(a.T, kPair) * kPair;
  p.pitch = ceil_div(a.C, 4) * 4;
  p.bytes = p.planes * p.rows * p.pitch * 4;
  return p;
}

cudaError_t launch_linear_planes(const LinearArgs& a, const PlanesPlan& p, float* sums, bool add,
                                 int sms, cudaStream_t stream) {
  Ready r{};
  CopyJobs jobs{};
  LinearPlan pairs{};
  pairs.pair = 1;
  CUtensorMap map_y;
  cudaError_t e = make_ready(a, pairs, nullptr, &jobs, &r);
  if (e == cudaSuccess &&
      !encode_boxes(&map_y, DT_F32, sums, p.planes * p.rows, a.C, p.pitch))
    e = cudaErrorInvalidValue;
  if (e != cudaSuccess) return e;
  const int64_t units = ceil_div(a.T, kPair) * ceil_div(a.C, kPair) * p.planes;
  return launch_linear_rows(a, r.map_x, r.map_w, map_y, pair_rows_idesc(a),
                            static_cast<int>(ktiles_of(a)), &p, add,
                            static_cast<int>(std::min<int64_t>(units, sms / 2)), stream);
}

template <class Ep>
cudaError_t launch_head(const LinearArgs& a, const LinearPlan& p, void* workspace, const Ep& ep,
                        cudaStream_t stream, int fault_inject) {
  Ready r{};
  CopyJobs jobs{};
  cudaError_t e = make_ready(a, p, workspace, &jobs, &r);
  if (e == cudaSuccess) e = launch_copies(&jobs, stream);
  if (e != cudaSuccess) return e;
  if (p.pair) {
    Ep with = ep;
    if constexpr (std::is_same<Ep, head::HeadGrad>::value)
      if (!encode_boxes(&with.map, ep.dtype, ep.D, ep.T, ep.C, ep.ldd))
        return cudaErrorInvalidValue;
    return launch_head_pair(r.map_x, r.map_w, pair_rows_idesc(a), with, a.w_mn != 0,
                            static_cast<int>(ktiles_of(a)), static_cast<int>(p.grid / 2),
                            fault_inject, stream);
  }
  SplitProblemsOf<Ep> problems{};
  problems.p[0] = problem_of(a, p, r, ep, 0);
  problems.p[1].first_cta = INT32_MAX;
  return launch_split(p, head_split_kernel_for<Ep>(p.bt), p.grid, &problems, fault_inject,
                      stream);
}
template cudaError_t launch_head(const LinearArgs&, const LinearPlan&, void*,
                                 const head::HeadStats&, cudaStream_t, int);
template cudaError_t launch_head(const LinearArgs&, const LinearPlan&, void*,
                                 const head::HeadGrad&, cudaStream_t, int);

cudaError_t launch_linear_two(const LinearArgs& a, const LinearPlan& pa, void* wa,
                              const LinearArgs& b, const LinearPlan& pb, void* wb,
                              cudaStream_t stream) {
  if (pa.pair || pb.pair || pa.bt != pb.bt || pa.cluster != pb.cluster || a.dtype != b.dtype ||
      pa.grid + pb.grid > INT32_MAX) {
    const cudaError_t e = launch_linear(a, pa, wa, stream);
    return e != cudaSuccess ? e : launch_linear(b, pb, wb, stream);
  }
  // At most two copies: dz is made for TMA to read.
  Ready ra{}, rb{};
  CopyJobs jobs{};
  cudaError_t e = make_ready(a, pa, wa, &jobs, &ra);
  if (e == cudaSuccess) e = make_ready(b, pb, wb, &jobs, &rb);
  if (e == cudaSuccess) e = launch_copies(&jobs, stream);
  if (e != cudaSuccess) return e;
  SplitProblems problems{};
  // The longer contraction's CTAs start first.
  if (ktiles_of(a) >= ktiles_of(b)) {
    problems.p[0] = problem_of(a, pa, ra, ra.ep, 0);
    problems.p[1] = problem_of(b, pb, rb, rb.ep, static_cast<int>(pa.grid));
  } else {
    problems.p[0] = problem_of(b, pb, rb, rb.ep, 0);
    problems.p[1] = problem_of(a, pa, ra, ra.ep, static_cast<int>(pb.grid));
  }
  return launch_split(pa, linear_split_kernel_for(a.dtype, pa.bt), pa.grid + pb.grid, &problems,
                      0, stream);
}

cudaError_t linear_read_and_clear_status(unsigned int* status) {
  unsigned int split = 0, pair = 0, rows = 0, head_split = 0, head_pair = 0;
  cudaError_t e = linear_split_read_and_clear_status(&split);
  if (e == cudaSuccess) e = linear_pair_read_and_clear_status(&pair);
  if (e == cudaSuccess) e = linear_rows_read_and_clear_status(&rows);
  if (e == cudaSuccess) e = head_split_read_and_clear_status(&head_split);
  if (e == cudaSuccess) e = head_pair_read_and_clear_status(&head_pair);
  *status = split | pair | rows | head_split | head_pair;
  return e;
}

}  // namespace mt
