// The fused linear layer on CTA pairs: 256 columns x 256 rows of Y per pair,
// persistent, for products with enough such tiles to fill the GPU.  The pair
// kernel of gemm_f16.cuh with the weight as its A operand (its rows are the
// columns of Y) and the tokens as its B operand.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "gemm_f16.cuh"
#include "layers.h"
#include "linear.cuh"

namespace mt {
namespace linear {

using namespace f16tc;

// Takes warp q's 32 columns of Y from tensor memory to Y while the next
// tile's MMAs run on the other accumulator; two warps share the 256 rows of
// a column block.
struct PairDrain {
  static constexpr bool DEPENDENT_LAUNCH = true;
  static constexpr int WARPS = 8, STORE_BYTES = 0;
  LinearEpilogue ep;
  __device__ __forceinline__ void operator()(uint32_t t_row, const Unit& w, int q, int half,
                                             int lane, const Sched&, float*, int rank) const {
    const int c = w.tm * PAIR_TILE + rank * PAIR_HALF + q * 32 + lane;
    const int t0 = w.tn * PAIR_TILE, first = t0 + half * PAIR_HALF;
    const int last = min(ep.T, first + PAIR_HALF);
    if (first < last)
      finish(ep, c, first, last, [&](int row, Rows& v) { tmem_ld16(t_row + (row - t0), v); });
  }
};

constexpr int PAIR_ACC_BUFS = 2;
using Geometry = PairGeometry<PAIR_ACC_BUFS>;

template <class E, bool W_MN, bool X_MN>
LinearKernel entry() {
  return LinearKernel{
      reinterpret_cast<const void*>(pair_kernel<E, W_MN, X_MN, PAIR_ACC_BUFS, PairDrain>),
      Geometry::SMEM_BYTES - EPI_STAGE_BYTES, Geometry::STAGES};
}

}  // namespace linear

using namespace linear;

LinearKernel linear_pair_kernel_for(int dtype, bool w_mn, bool x_mn) {
  if (dtype == DT_E4M3)
    return w_mn || x_mn ? LinearKernel{} : entry<E4m3, false, false>();
  if (x_mn) return w_mn ? entry<Half, true, true>() : LinearKernel{};
  return w_mn ? entry<Half, true, false>() : entry<Half, false, false>();
}

cudaError_t launch_linear_pair(const LinearKernel& k, const CUtensorMap& map_w,
                               const CUtensorMap& map_x, uint32_t idesc,
                               const LinearEpilogue& ep, int kt, int clusters,
                               int fault_inject, cudaStream_t stream) {
  PairDrain drain{ep};
  int tiles_c = (ep.C + PAIR_TILE - 1) / PAIR_TILE, tiles_t = (ep.T + PAIR_TILE - 1) / PAIR_TILE;
  int group = 8;
  Sched sched{tiles_c * tiles_t, 1, kt, nullptr, 0, 0};
  CUtensorMap w = map_w, x = map_x;
  void* args[] = {&w,       &x,       &idesc, &drain, &kt,
                  &tiles_c, &tiles_t, &group, &sched, &fault_inject};
  return launch_dependent(k.kernel, dim3(2 * static_cast<unsigned>(clusters)),
                          pair_threads<PairDrain>(), k.smem, 2,
                          stream, args);
}

cudaError_t linear_pair_read_and_clear_status(unsigned int* status) {
  return f16tc::read_and_clear_status(status);
}

}  // namespace mt
