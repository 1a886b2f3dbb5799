// k10_linrec_f32.cu -- the gated linear recurrence for f32 activations (kernels in k10_linrec.cuh).
#include "k10_linrec.cuh"

namespace gdr {
LINREC_INSTANTIATE(float, float)
}  // namespace gdr
