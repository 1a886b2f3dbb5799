// k9_norms.cu -- the norms around a block: choice by type, and the sum of the partial column sums (dweight, dscale).
#include <map>
#include <mutex>
#include <tuple>

#include "block_common.cuh"

namespace gdr {

namespace {
std::mutex g_mu;
// per device, by kernel, warps of a CTA and CTAs of a cluster: CTAs (clusters) that it holds
std::map<std::tuple<const void *, int, int>, int> g_resident[64];
}  // namespace

// CTAs of a persistent grid, or its clusters of `ctas`: as many as the device holds at a time, no more than there are rows for,
// and at most `most`.
// max_smem: with the most threads that the kernel is launched with.
cudaError_t norm_grid(const void *kernel, int threads, int ctas, int smem, int max_smem, int64_t rows, int rows_per_cta, int most,
                      int &grid) {
    int dev = 0, n = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    {
        std::lock_guard<std::mutex> lock(g_mu);
        int fresh = 0;
        int &held = dev >= 0 && dev < 64 ? g_resident[dev][{kernel, threads / 32, ctas}] : fresh;
        if (!held) {
            int sms = 0, per_sm = 0;
            if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, max_smem)) != cudaSuccess)
                return e;
            if (ctas > 1) {
                ClusterLaunch l(ctas, threads, smem, ctas, nullptr);
                if ((e = cudaOccupancyMaxActiveClusters(&held, kernel, &l.cfg)) != cudaSuccess) return e;
            } else {
                if ((e = device_sm_count(&sms)) != cudaSuccess) return e;
                if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kernel, threads, smem)) != cudaSuccess) return e;
                held = sms * per_sm;
            }
            if (held < 1) return cudaErrorInvalidConfiguration;
        }
        n = held;
    }
    const int64_t need = (rows + rows_per_cta - 1) / rows_per_cta;
    if (n > need) n = (int)need;
    if (n > most) n = most;
    grid = n < 1 ? 1 : n;
    return cudaSuccess;
}

// Rows of partial sums that a backward may write: as many CTAs as its grid can have.
int norm_parts(int64_t rows, int64_t dim) {
    const int64_t most = dim <= 512 ? NORM_MAX_PARTS : NORM_MAX_PARTS / 2;
    return (int)(rows < most ? (rows < 1 ? 1 : rows) : most);
}

// out[col] = sum over the partial rows, in a fixed order: a CTA takes 32 columns of one of the sums, its 32 warps take every
// 32nd row each, and the warps' sums are added in order.
__global__ void __launch_bounds__(1024) k9_colsum(const float *part, int parts, int dim, void *out0, int dtype0, void *out1,
                                                  int dtype1) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    part += (size_t)blockIdx.y * parts * dim;
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the kernel before has ended, its partial rows are there
    float a = 0.f;
    if (col < dim)
        for (int r0 = wid; r0 < parts; r0 += 32 * 10) {
            float v[10];  // all under way at once
#pragma unroll
            for (int i = 0; i < 10; ++i) v[i] = r0 + 32 * i < parts ? part[(size_t)(r0 + 32 * i) * dim + col] : 0.f;
#pragma unroll
            for (int i = 0; i < 10; ++i) a += v[i];
        }
    s[wid][lane] = a;
    __syncthreads();
    if (wid == 0 && col < dim) {
        float t = 0.f;
#pragma unroll
        for (int i = 0; i < 32; ++i) t += s[i][lane];
        store_scalar(blockIdx.y ? out1 : out0, col, t, blockIdx.y ? dtype1 : dtype0);
    }
}

cudaError_t launch_colsum(const float *part, int parts, int dim, int sums, void *out0, int dtype0, void *out1, int dtype1,
                          cudaStream_t stream) {
    // its CTAs are set up while the kernel before ends (65536 x 128 after a block, backward 22.1 -> 20.4 us)
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((dim + 31) / 32, sums);
    cfg.blockDim = dim3(1024);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k9_colsum, part, parts, dim, out0, dtype0, out1, dtype1);
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
