// k11_clip.cu -- the global gradient norm over many tensors, and clipping.
//
//   norm = sqrt(sum of all squares) ;  out_i = grad_i min(1, max_norm / (norm + eps))
//
// The tensors are cut into pieces of CLIP_PIECE elements, numbered through all of them; a CTA takes every gridDim-th
// piece, in 16-byte loads that are all under way before the first is used.  The table of tensors travels as a kernel
// argument, so the call copies nothing to the device and can be captured in a graph.  A first kernel leaves one partial
// sum per CTA; the second adds them in order in every CTA (a few KB from L2), which saves a launch and a counter between
// the two, and scales.  Both are bound by HBM: the gradients have to be read twice, since all of them decide on the
// factor.  The second kernel goes through the pieces from the last to the first, whose end is then still in L2.
// 393 million bf16 gradients clipped into fp32: 0.484 ms, 6.5 TB/s (6.8 is a plain copy's).  A few small tensors are one
// launch (k11_small).
//
// Squares are summed in fp32 within a thread's part of a piece (at most 32 of them to a sum) and in fp64 from there on.
#include "block_clip.h"
#include "block_common.cuh"

namespace gdr {
namespace {

constexpr int CLIP_THREADS = 512, CLIP_CLUSTER = 8;

template <int N> __device__ __forceinline__ int find_tensor(const ClipTable<N> &t, int64_t piece) {
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
#pragma unroll
    for (int i = 0; i < CLIP_THREADS / 32; ++i) v += red[i];
    return v;
}

// The sum of a thread's squares in a piece of n elements.
template <typename T> __device__ __forceinline__ float piece_sumsq(const T *x, int n) {
    constexpr int V = 16 / (int)sizeof(T), P = CLIP_PIECE / (V * CLIP_THREADS);
    float s = 0.f;
    if (n == CLIP_PIECE && (uintptr_t)x % 16 == 0) {
        Pack<T, V> v[P];
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = load_pack<T, V>(x + (k * CLIP_THREADS + threadIdx.x) * V);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            float f[V];
            unpack<T, V>(v[k], f);
#pragma unroll
            for (int j = 0; j < V; ++j) s = fmaf(f[j], f[j], s);
        }
    } else {
        for (int i = threadIdx.x; i < n; i += CLIP_THREADS) {
            const float f = to_f32(x[i]);
            s = fmaf(f, f, s);
        }
    }
    return s;
}

template <int N> __device__ __forceinline__ float one_sumsq(const ClipTable<N> &t, int64_t piece) {
    const int k = find_tensor(t, piece);
    const int64_t start = (piece - t.first[k]) * CLIP_PIECE;
    const int n = (int)min((int64_t)CLIP_PIECE, t.size[k] - start);
    if (t.dtype[k] == F32) return piece_sumsq(reinterpret_cast<const float *>(t.grad[k]) + start, n);
    if (t.dtype[k] == BF16) return piece_sumsq(reinterpret_cast<const __nv_bfloat16 *>(t.grad[k]) + start, n);
    return piece_sumsq(reinterpret_cast<const __half *>(t.grad[k]) + start, n);
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS, 4) k11_sumsq(const __grid_constant__ ClipTable<N> t, double *part) {
    __shared__ double red[CLIP_THREADS / 32];
    double total = 0.0;
    for (int64_t piece = blockIdx.x; piece < t.pieces; piece += gridDim.x) total += one_sumsq(t, piece);
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

template <typename T, typename O> __device__ __forceinline__ void piece_scale(const T *x, O *o, int n, float f) {
    // 16 bytes of the wider type at a time: a warp's accesses are then contiguous on both sides (8 elements, whose fp32
    // results leave as two halves 32 bytes apart, took 0.48 ms instead of 0.36 ms for 393 M bf16 gradients)
    constexpr int V = 16 / (int)(sizeof(T) > sizeof(O) ? sizeof(T) : sizeof(O)), P = CLIP_PIECE / (V * CLIP_THREADS);
    if (n == CLIP_PIECE && (uintptr_t)x % (V * sizeof(T)) == 0 && (uintptr_t)o % (V * sizeof(O)) == 0) {
        Pack<T, V> v[P];
#pragma unroll
        for (int k = 0; k < P; ++k) v[k] = load_pack<T, V>(x + (k * CLIP_THREADS + threadIdx.x) * V);
#pragma unroll
        for (int k = 0; k < P; ++k) {
            float y[V];
            unpack<T, V>(v[k], y);
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] *= f;
            store_pack<O, V>(o + (k * CLIP_THREADS + threadIdx.x) * V, y);
        }
    } else {
        for (int i = threadIdx.x; i < n; i += CLIP_THREADS) o[i] = to_out_t<O>(f * to_f32(x[i]));
    }
}
template <typename T> __device__ __forceinline__ void piece_scale(const T *x, void *o, int64_t start, int n, int dt, float f) {
    if (dt == F32) piece_scale(x + start, reinterpret_cast<float *>(o) + start, n, f);
    else if (dt == BF16) piece_scale(x + start, reinterpret_cast<__nv_bfloat16 *>(o) + start, n, f);
    else piece_scale(x + start, reinterpret_cast<__half *>(o) + start, n, f);
}

template <int N> __device__ __forceinline__ void one_scale(const ClipTable<N> &t, int64_t piece, float f) {
    const int k = find_tensor(t, piece);
    const int64_t start = (piece - t.first[k]) * CLIP_PIECE;
    const int n = (int)min((int64_t)CLIP_PIECE, t.size[k] - start);
    if (t.dtype[k] == F32) piece_scale(reinterpret_cast<const float *>(t.grad[k]), t.out[k], start, n, t.out_dtype[k], f);
    else if (t.dtype[k] == BF16)
        piece_scale(reinterpret_cast<const __nv_bfloat16 *>(t.grad[k]), t.out[k], start, n, t.out_dtype[k], f);
    else piece_scale(reinterpret_cast<const __half *>(t.grad[k]), t.out[k], start, n, t.out_dtype[k], f);
}
__device__ __forceinline__ float factor_of(float norm, float max_norm, float eps) {
    const float f = max_norm / (norm + eps);
    return f > 1.f ? 1.f : f;  // (a nan stays one)
}

template <int N>
__global__ void __launch_bounds__(CLIP_THREADS, 3) k11_scale(const __grid_constant__ ClipTable<N> t, const double *part,
                                                             int parts, float *norm, float max_norm, float eps) {
    __shared__ double red[CLIP_THREADS / 32];
    const float n = norm_of(part, parts, red);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    const float f = factor_of(n, max_norm, eps);
    for (int64_t piece = t.pieces - 1 - blockIdx.x; piece >= 0; piece -= gridDim.x) one_scale(t, piece, f);
}

__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Both steps in one launch, by one cluster whose CTAs tell each other their partial sums: for small totals, where a second
// launch costs more than the work (20 fp32 tensors of 4096: 9 us of a call less; it takes 35 to 40, nearly all of it the host's
// work on the list).
template <int N, bool SCALE>
__global__ void __launch_bounds__(CLIP_THREADS) k11_small(const __grid_constant__ ClipTable<N> t, float *norm, float max_norm,
                                                          float eps) {
    __shared__ double red[CLIP_THREADS / 32], part[CLIP_CLUSTER];
    double total = 0.0;
    for (int64_t piece = blockIdx.x; piece < t.pieces; piece += CLIP_CLUSTER) total += one_sumsq(t, piece);
    total = block_sum(total, red);
    cluster_meet();  // (every CTA runs: its shared memory may be written)
    if (threadIdx.x < CLIP_CLUSTER) {
        uint32_t at;
        asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(&part[blockIdx.x])), "r"(threadIdx.x));
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(total) : "memory");
    }
    cluster_meet();
    double v = 0.0;
#pragma unroll
    for (int i = 0; i < CLIP_CLUSTER; ++i) v += part[i];
    const float n = (float)sqrt(v);
    if (blockIdx.x == 0 && threadIdx.x == 0) *norm = n;
    if (SCALE) {
        const float f = factor_of(n, max_norm, eps);
        for (int64_t piece = blockIdx.x; piece < t.pieces; piece += CLIP_CLUSTER) one_scale(t, piece, f);
    }
}

// A short list takes a short table: the argument is copied with every launch.
template <int N> void shorten(const ClipTable<CLIP_TENSORS> &t, ClipTable<N> &s) {
    for (int i = 0; i < t.count; ++i) {
        s.grad[i] = t.grad[i], s.out[i] = t.out[i], s.size[i] = t.size[i], s.first[i] = t.first[i];
        s.dtype[i] = t.dtype[i], s.out_dtype[i] = t.out_dtype[i];
    }
    s.first[t.count] = t.first[t.count];
    s.pieces = t.pieces, s.count = t.count;
}
constexpr int CLIP_SHORT = 64;

// Pieces up to which one cluster does both steps: 4 for each of its CTAs.
constexpr int64_t CLIP_SMALL_PIECES = 4 * CLIP_CLUSTER;

}  // namespace

cudaError_t launch_clip_sumsq(const ClipTable<CLIP_TENSORS> &t, double *part, int parts, cudaStream_t stream) {
    if (t.count <= CLIP_SHORT) {
        ClipTable<CLIP_SHORT> s;
        shorten(t, s);
        k11_sumsq<<<parts, CLIP_THREADS, 0, stream>>>(s, part);
    } else {
        k11_sumsq<<<parts, CLIP_THREADS, 0, stream>>>(t, part);
    }
    return cudaGetLastError();
}
bool clip_is_small(const ClipTable<CLIP_TENSORS> &t) { return t.count <= CLIP_SHORT && t.pieces <= CLIP_SMALL_PIECES; }

cudaError_t launch_clip_small(const ClipTable<CLIP_TENSORS> &t, float *norm, bool scale, float max_norm, float eps,
                              cudaStream_t stream) {
    ClipTable<CLIP_SHORT> s;
    shorten(t, s);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CLIP_CLUSTER);
    cfg.blockDim = dim3(CLIP_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = CLIP_CLUSTER;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (scale) return cudaLaunchKernelEx(&cfg, k11_small<CLIP_SHORT, true>, s, norm, max_norm, eps);
    return cudaLaunchKernelEx(&cfg, k11_small<CLIP_SHORT, false>, s, norm, max_norm, eps);
}

cudaError_t launch_clip_norm(const double *part, int parts, float *norm, cudaStream_t stream) {
    k11_norm<<<1, CLIP_THREADS, 0, stream>>>(part, parts, norm);
    return cudaGetLastError();
}
cudaError_t launch_clip_scale(const ClipTable<CLIP_TENSORS> &t, const double *part, int parts, float *norm, float max_norm,
                              float eps, cudaStream_t stream) {
    const int64_t most = t.pieces < CLIP_CTAS ? t.pieces : CLIP_CTAS;
    const int grid = (int)(most < 1 ? 1 : most);
    if (t.count <= CLIP_SHORT) {
        ClipTable<CLIP_SHORT> s;
        shorten(t, s);
        k11_scale<<<grid, CLIP_THREADS, 0, stream>>>(s, part, parts, norm, max_norm, eps);
    } else {
        k11_scale<<<grid, CLIP_THREADS, 0, stream>>>(t, part, parts, norm, max_norm, eps);
    }
    return cudaGetLastError();
}

}  // namespace gdr
