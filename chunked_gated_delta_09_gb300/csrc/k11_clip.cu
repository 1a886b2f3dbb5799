// k11_clip.cu -- the global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum of all squares) ;  out_i = grad_i min(1, max_norm / (norm + eps))
//
// The tensors are cut into pieces of CLIP_PIECE elements, numbered through all of them; a CTA takes every
// gridDim-th piece.  The table of tensors travels as a kernel argument, so the call copies nothing to the device
// and can be captured in a graph.  A first kernel leaves one partial sum per CTA; the second adds them in order in
// every CTA (a few KB from L2), which saves a launch and a counter between the two, and scales.
#include "block_clip.h"
#include "block_common.cuh"

namespace gdr {
namespace {

constexpr int CLIP_THREADS = 512;

__device__ __forceinline__ int find_tensor(const ClipTable &t, int64_t piece) {
    int lo = 0, hi = t.count;  // first[lo] <= piece < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (t.first[mid] <= piece) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ double block_sum(double v, double *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int i = 0; i < CLIP_THREADS / 32; ++i) v += red[i];
    return v;
}

__global__ void __launch_bounds__(CLIP_THREADS) k11_sumsq(const __grid_constant__ ClipTable t, double *part) {
    __shared__ double red[CLIP_THREADS / 32];
    double total = 0.0;
    for (int64_t piece = blockIdx.x; piece < t.pieces; piece += gridDim.x) {
        const int k = find_tensor(t, piece);
        const int64_t start = (piece - t.first[k]) * CLIP_PIECE, end = min(start + CLIP_PIECE, t.size[k]);
        float s = 0.f;
        for (int64_t i = start + threadIdx.x; i < end; i += CLIP_THREADS) {
            const float x = load_scalar(t.grad[k], i, t.dtype[k]);
            s = fmaf(x, x, s);
        }
        total += s;
    }
    total = block_sum(total, red);
    if (threadIdx.x == 0) part[blockIdx.x] = total;
}

__device__ __forceinline__ float norm_of(const double *part, int parts, double *red) {
    double v = 0.0;
    for (int i = threadIdx.x; i < parts; i += CLIP_THREADS) v += part[i];
    return (float)sqrt(block_sum(v, red));
}

__global__ void __launch_bounds__(CLIP_THREADS) k11_norm(const double *part, int parts, float *norm) {
    __shared__ double red[CLIP_THREADS / 32];
    const float n = norm_of(part, parts, red);
    if (threadIdx.x == 0) *norm = n;
}

__global__ void __launch_bounds__(CLIP_THREADS)
    k11_scale(const __grid_constant__ ClipTable t, const double *part, int parts, float *norm, float max_norm, float eps) {
    __shared__ double red[CLIP_THREADS / 32];
    const float n = norm_of(part, parts, red);
    if (norm && blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    float f = max_norm / (n + eps);
    f = f > 1.f ? 1.f : f;  // (a nan stays one)
    for (int64_t piece = blockIdx.x; piece < t.pieces; piece += gridDim.x) {
        const int k = find_tensor(t, piece);
        const int64_t start = (piece - t.first[k]) * CLIP_PIECE, end = min(start + CLIP_PIECE, t.size[k]);
        for (int64_t i = start + threadIdx.x; i < end; i += CLIP_THREADS)
            store_scalar(t.out[k], i, f * load_scalar(t.grad[k], i, t.dtype[k]), t.out_dtype[k]);
    }
}

}  // namespace

cudaError_t launch_clip_sumsq(const ClipTable &t, double *part, int parts, cudaStream_t stream) {
    k11_sumsq<<<parts, CLIP_THREADS, 0, stream>>>(t, part);
    return cudaGetLastError();
}
cudaError_t launch_clip_norm(const double *part, int parts, float *norm, cudaStream_t stream) {
    k11_norm<<<1, CLIP_THREADS, 0, stream>>>(part, parts, norm);
    return cudaGetLastError();
}
cudaError_t launch_clip_scale(const ClipTable &t, const double *part, int parts, float *norm, float max_norm, float eps,
                              cudaStream_t stream) {
    const int64_t grid = t.pieces < CLIP_CTAS ? t.pieces : CLIP_CTAS;
    k11_scale<<<(int)(grid < 1 ? 1 : grid), CLIP_THREADS, 0, stream>>>(t, part, parts, norm, max_norm, eps);
    return cudaGetLastError();
}

}  // namespace gdr
