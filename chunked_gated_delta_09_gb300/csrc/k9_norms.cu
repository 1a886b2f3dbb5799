// k9_norms.cu -- the norms around a block: choice by type, and the sum of the partial column sums (dweight, dscale).
#include "block_common.cuh"

namespace gdr {

// Rows of partial sums that a backward may write: as many CTAs as its grid can have.
int norm_parts(int64_t rows, int64_t dim) {
    const int64_t most = dim <= 512 ? NORM_MAX_PARTS : NORM_MAX_PARTS / 2;
    return (int)(rows < most ? (rows < 1 ? 1 : rows) : most);
}

// out[col] = sum over the partial rows, in a fixed order: a CTA takes 32 columns, its 32 warps take every 32nd row
// each, and the warps' sums are added in order.
__global__ void __launch_bounds__(1024) k9_colsum(const float *part, int parts, int dim, void *out, int dtype) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float a = 0.f;
    if (col < dim)
        for (int r = wid; r < parts; r += 32) a += part[(size_t)r * dim + col];
    s[wid][lane] = a;
    __syncthreads();
    if (wid == 0 && col < dim) {
        float t = 0.f;
        for (int i = 0; i < 32; ++i) t += s[i][lane];
        store_scalar(out, col, t, dtype);
    }
}

cudaError_t launch_colsum(const float *part, int parts, int dim, void *out, int dtype, cudaStream_t stream) {
    k9_colsum<<<(dim + 31) / 32, 1024, 0, stream>>>(part, parts, dim, out, dtype);
    return cudaGetLastError();
}

template <typename T> cudaError_t gated_norm_fwd_t(const GatedNormParams &, cudaStream_t);
template <typename T> cudaError_t gated_norm_bwd_t(const GatedNormParams &, cudaStream_t);
template <typename T, typename R> cudaError_t add_norm_fwd_t(const AddNormParams &, cudaStream_t);
template <typename T, typename R> cudaError_t add_norm_bwd_t(const AddNormParams &, cudaStream_t);

cudaError_t launch_gated_norm_fwd(const GatedNormParams &p, cudaStream_t s) {
    if (p.dtype == F32) return gated_norm_fwd_t<float>(p, s);
    return p.dtype == BF16 ? gated_norm_fwd_t<__nv_bfloat16>(p, s) : gated_norm_fwd_t<__half>(p, s);
}
cudaError_t launch_gated_norm_bwd(const GatedNormParams &p, cudaStream_t s) {
    if (p.dtype == F32) return gated_norm_bwd_t<float>(p, s);
    return p.dtype == BF16 ? gated_norm_bwd_t<__nv_bfloat16>(p, s) : gated_norm_bwd_t<__half>(p, s);
}
cudaError_t launch_add_norm_fwd(const AddNormParams &p, cudaStream_t s) {
    if (p.dtype == F32) return add_norm_fwd_t<float, float>(p, s);
    if (p.residual_dtype == F32)
        return p.dtype == BF16 ? add_norm_fwd_t<__nv_bfloat16, float>(p, s) : add_norm_fwd_t<__half, float>(p, s);
    return p.dtype == BF16 ? add_norm_fwd_t<__nv_bfloat16, __nv_bfloat16>(p, s) : add_norm_fwd_t<__half, __half>(p, s);
}
cudaError_t launch_add_norm_bwd(const AddNormParams &p, cudaStream_t s) {
    if (p.dtype == F32) return add_norm_bwd_t<float, float>(p, s);
    if (p.residual_dtype == F32)
        return p.dtype == BF16 ? add_norm_bwd_t<__nv_bfloat16, float>(p, s) : add_norm_bwd_t<__half, float>(p, s);
    return p.dtype == BF16 ? add_norm_bwd_t<__nv_bfloat16, __nv_bfloat16>(p, s) : add_norm_bwd_t<__half, __half>(p, s);
}

}  // namespace gdr
