// Products without an epilogue but a scale on CTA pairs, for results that TMA
// writes: 256 rows x 256 columns of Y a tile (the pair kernel of gemm_f16.cuh with
// the rows' operand as its A), drained a row a lane through boxes in shared
// memory (store_box.cuh).  A product of few tiles cuts its contraction into
// slices, whose sums go to a plane of fp32 each, or are added to what is there.  The loss's
// weight gradient of a few tokens is all result: 65536 x 4096 bf16 from 16 tokens
// takes 118 us so, 231 us with the linear layer's drain.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "gemm_f16.cuh"
#include "layers.h"
#include "store_box.cuh"

namespace mt {
namespace f16tc {

struct RowsDrain {
  static constexpr bool DEPENDENT_LAUNCH = true;
  static constexpr int WARPS = 8, STORE_BYTES = WARPS * STORE_BOX_BYTES;
  CUtensorMap map;
  const float* scale;  // one value; null: 1
  int T, C, dtype, add;
  int64_t plane_rows;  // slices: rows of a plane

  template <class V>
  __device__ __forceinline__ void typed(uint32_t t_row, int lane, uint8_t* box, int x0,
                                        int y, int row) const {
    constexpr int COLS = STORE_ROW_BYTES / static_cast<int>(sizeof(V)), CHUNK = 32;
    const float s = scale ? *scale : 1.0f;
#pragma unroll 1
    for (int c = 0; c < PAIR_HALF; c += COLS) {
      store_begin(lane);
#pragma unroll
      for (int i = 0; i < COLS; i += CHUNK) {
        float v[CHUNK];
        __syncwarp();
        tmem_ld32(t_row + c + i, v);
        if (scale) {
#pragma unroll
          for (int k = 0; k < CHUNK; ++k) v[k] *= s;
        }
        store_fill<V>(box, lane, i, v);
      }
      store_end(&map, box, lane, x0 + c, row, x0 + c < C && y < T, add != 0);
    }
  }

  __device__ __forceinline__ void operator()(uint32_t t_row, const Unit& w, int q, int half,
                                             int lane, const Sched& sched, float* square,
                                             int rank) const {
    uint8_t* const box = store_staging<RowsDrain>(square, q, half);
    const int y = w.tm * PAIR_TILE + rank * PAIR_HALF + q * 32;
    const int row =
        y + (w.pidx >= 0 ? static_cast<int>(w.pidx % sched.split * plane_rows) : 0);
    const int x = w.tn * PAIR_TILE + half * PAIR_HALF;
    const uint32_t from = t_row + half * PAIR_HALF;
    if (dtype == DT_F16) typed<__half>(from, lane, box, x, y, row);
    else if (dtype == DT_BF16) typed<__nv_bfloat16>(from, lane, box, x, y, row);
    else typed<float>(from, lane, box, x, y, row);
  }
};

constexpr int ACC_BUFS = 2;

const void* rows_kernel_for(bool x_mn, bool w_mn) {
  if (x_mn)
    return w_mn ? reinterpret_cast<const void*>(pair_kernel<Half, true, true, ACC_BUFS, RowsDrain>)
                : nullptr;
  return w_mn ? reinterpret_cast<const void*>(pair_kernel<Half, false, true, ACC_BUFS, RowsDrain>)
              : reinterpret_cast<const void*>(
                    pair_kernel<Half, false, false, ACC_BUFS, RowsDrain>);
}

}  // namespace f16tc

using namespace f16tc;

cudaError_t linear_rows_prepare() {
  for (int mn : {0, 2, 3}) {
    const cudaError_t e = cudaFuncSetAttribute(rows_kernel_for(mn & 1, mn & 2),
                                               cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               pair_smem<RowsDrain, ACC_BUFS>());
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_linear_rows(const LinearArgs& a, const CUtensorMap& map_x,
                               const CUtensorMap& map_w, const CUtensorMap& map_y,
                               uint32_t idesc, int kt, const PlanesPlan* planes, bool add,
                               int clusters, cudaStream_t stream) {
  RowsDrain drain{map_y,
                  a.scale,
                  static_cast<int>(a.T),
                  static_cast<int>(a.C),
                  planes ? DT_F32 : a.out_dtype,
                  add ? 1 : 0,
                  planes ? planes->rows : 0};
  int tiles_t = static_cast<int>((a.T + PAIR_TILE - 1) / PAIR_TILE);
  int tiles_c = static_cast<int>((a.C + PAIR_TILE - 1) / PAIR_TILE);
  int group = 8, fault_inject = 0;
  Sched sched{tiles_t * tiles_c, 1, kt, nullptr, 0, 0};
  if (planes) {
    sched.full_tiles = 0;
    sched.kt_per_slice = (kt + planes->planes - 1) / planes->planes;
    sched.split = (kt + sched.kt_per_slice - 1) / sched.kt_per_slice;  // none empty
  }
  CUtensorMap x = map_x, w = map_w;
  void* args[] = {&x,       &w,       &idesc, &drain, &kt,
                  &tiles_t, &tiles_c, &group, &sched, &fault_inject};
  return launch_dependent(rows_kernel_for(a.x_mn, a.w_mn),
                          dim3(2 * static_cast<unsigned>(clusters)), pair_threads<RowsDrain>(),
                          pair_smem<RowsDrain, ACC_BUFS>(), 2, stream, args);
}

cudaError_t linear_rows_read_and_clear_status(unsigned int* status) {
  return f16tc::read_and_clear_status(status);
}

}  // namespace mt
