// The layer norm's gradient in fp16: a translation unit of its own for the build's
// sake.
#include "layer_norm_grad.cuh"

namespace mt {

MT_LAYER_NORM_GRAD_TYPE(f16, __half)

}  // namespace mt
