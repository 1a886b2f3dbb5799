// k10_linrec_f16.cu -- the gated linear recurrence for f16 activations (kernels in k10_linrec.cuh).
#include "k10_linrec.cuh"

namespace gdr {
LINREC_INSTANTIATE(__half, __half)
LINREC_INSTANTIATE(__half, float)
}  // namespace gdr
