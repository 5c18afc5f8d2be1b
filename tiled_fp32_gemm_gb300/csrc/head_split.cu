// The vocabulary loss's logits of few tokens: the split kernel
// (linear_split.cuh) with the loss's epilogues.
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "head.cuh"
#include "linear_split.cuh"

namespace mt {

using namespace head;

template <class Ep>
linear::LinearKernel head_split_kernel_for(int bt) {
  using linear::linear_split_kernel;  // its finish() is found by the epilogue's namespace
  using linear::SplitGeometry;
  auto of = [](auto kernel, int smem, int stages) {
    return linear::LinearKernel{reinterpret_cast<const void*>(kernel), smem, stages};
  };
  switch (bt) {
    case 16: return of(linear_split_kernel<f16tc::Half, 16, Ep>, SplitGeometry<16>::SMEM_BYTES,
                       SplitGeometry<16>::STAGES);
    case 32: return of(linear_split_kernel<f16tc::Half, 32, Ep>, SplitGeometry<32>::SMEM_BYTES,
                       SplitGeometry<32>::STAGES);
    case 64: return of(linear_split_kernel<f16tc::Half, 64, Ep>, SplitGeometry<64>::SMEM_BYTES,
                       SplitGeometry<64>::STAGES);
    default: return of(linear_split_kernel<f16tc::Half, 128, Ep>,
                       SplitGeometry<128>::SMEM_BYTES, SplitGeometry<128>::STAGES);
  }
}
template linear::LinearKernel head_split_kernel_for<HeadStats>(int);
template linear::LinearKernel head_split_kernel_for<HeadGrad>(int);

cudaError_t head_split_read_and_clear_status(unsigned int* status) {
  return f16tc::read_and_clear_status(status);
}

}  // namespace mt
