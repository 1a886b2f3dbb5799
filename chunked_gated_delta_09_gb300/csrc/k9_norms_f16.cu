// k9_norms_f16.cu -- the norms around a block for f16 activations (kernels in k9_norms.cuh).
#include "k9_norms.cuh"

namespace gdr {
NORM_INSTANTIATE(__half)
NORM_INSTANTIATE_F32_STREAM(__half)
}  // namespace gdr
