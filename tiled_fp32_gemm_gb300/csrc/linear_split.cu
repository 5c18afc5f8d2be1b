// The fused linear layer on one CTA tile per cluster: the split kernel
// (linear_split.cuh) with the linear layer's epilogue.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "linear_split.cuh"

namespace mt {
namespace linear {

template <class E, int BT>
LinearKernel entry() {
  return LinearKernel{reinterpret_cast<const void*>(linear_split_kernel<E, BT, LinearEpilogue>),
                      SplitGeometry<BT>::SMEM_BYTES, SplitGeometry<BT>::STAGES};
}

template <class E>
LinearKernel entry_for(int bt) {
  switch (bt) {
    case 16: return entry<E, 16>();
    case 32: return entry<E, 32>();
    case 64: return entry<E, 64>();
    default: return entry<E, 128>();
  }
}

}  // namespace linear

using namespace linear;

LinearKernel linear_split_kernel_for(int dtype, int bt) {
  return dtype == DT_E4M3 ? entry_for<E4m3>(bt) : entry_for<Half>(bt);
}

cudaError_t linear_split_read_and_clear_status(unsigned int* status) {
  return f16tc::read_and_clear_status(status);
}

}  // namespace mt
