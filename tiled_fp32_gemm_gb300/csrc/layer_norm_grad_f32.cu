// The layer norm's gradient in fp32, and the choice among the types.
#include "layer_norm_grad.cuh"

namespace mt {

MT_LAYER_NORM_GRAD_TYPE(f32, float)

int64_t layer_norm_grad_workspace(const LayerNormGradArgs& a, int sms) {
  Staging g{};
  int parts = 0;
  path_of(a, sms, &g, &parts);
  return static_cast<int64_t>(parts) * a.d * 4 * ((a.dweight != nullptr) + (a.dbias != nullptr));
}

cudaError_t launch_layer_norm_grad(const LayerNormGradArgs& a, void* workspace, int sms,
                                   cudaStream_t stream) {
  float* partial = static_cast<float*>(workspace);
  switch (a.dtype) {
    case DT_F16: return launch_layer_norm_grad_f16(a, partial, sms, stream);
    case DT_BF16: return launch_layer_norm_grad_bf16(a, partial, sms, stream);
    default: return launch_layer_norm_grad_f32(a, partial, sms, stream);
  }
}

cudaError_t layer_norm_grad_read_and_clear_status(unsigned int* status) {
  unsigned int f16 = 0, bf16 = 0, f32 = 0;
  cudaError_t e = layer_norm_grad_f16_read_and_clear_status(&f16);
  if (e == cudaSuccess) e = layer_norm_grad_bf16_read_and_clear_status(&bf16);
  if (e == cudaSuccess) e = layer_norm_grad_f32_read_and_clear_status(&f32);
  *status = f16 | bf16 | f32;
  return e;
}

}  // namespace mt
