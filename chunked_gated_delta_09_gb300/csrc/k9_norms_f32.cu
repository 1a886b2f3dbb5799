// k9_norms_f32.cu -- the norms around a block for f32 activations (kernels in k9_norms.cuh).
#include "k9_norms.cuh"

namespace gdr {
NORM_INSTANTIATE(float)
}  // namespace gdr
