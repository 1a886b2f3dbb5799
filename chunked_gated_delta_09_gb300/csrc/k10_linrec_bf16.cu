// k10_linrec_bf16.cu -- the gated linear recurrence for bf16 activations (kernels in k10_linrec.cuh).
#include "k10_linrec.cuh"

namespace gdr {
LINREC_INSTANTIATE(__nv_bfloat16, __nv_bfloat16)
LINREC_INSTANTIATE(__nv_bfloat16, float)
}  // namespace gdr
