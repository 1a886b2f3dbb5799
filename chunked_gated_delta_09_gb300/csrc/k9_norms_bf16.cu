// k9_norms_bf16.cu -- the norms around a block for bf16 activations (kernels in k9_norms.cuh).
#include "k9_norms.cuh"

namespace gdr {
NORM_INSTANTIATE(__nv_bfloat16)
NORM_INSTANTIATE_F32_STREAM(__nv_bfloat16)
}  // namespace gdr
