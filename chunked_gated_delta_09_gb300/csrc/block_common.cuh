// block_common.cuh -- device-side pieces of the operators around the delta rule (include/gdr_block.h) and the
// host-side launchers that block_api.cu calls.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "gdr_common.cuh"
#include "gdr_kernels.h"

namespace gdr {

// N consecutive elements moved as one access (two when they exceed 16 bytes).
template <typename T, int N> struct alignas(sizeof(T) * N < 16 ? sizeof(T) * N : 16) Pack {
    T v[N];
};
template <typename T, int N> __device__ __forceinline__ Pack<T, N> load_pack(const T *p) {
    return *reinterpret_cast<const Pack<T, N> *>(p);
}
template <typename T, int N> __device__ __forceinline__ void unpack(const Pack<T, N> &a, float (&o)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = to_f32(a.v[i]);
}
// Two values rounded by one instruction.
template <typename T> struct Pair;
template <> struct Pair<__nv_bfloat16> {
    static __device__ __forceinline__ uint32_t of(float x, float y) {
        const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <> struct Pair<__half> {
    static __device__ __forceinline__ uint32_t of(float x, float y) {
        const __half2 v = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
};
template <typename T, int N> __device__ __forceinline__ void store_pack(T *p, const float (&x)[N]) {
    Pack<T, N> a;
    if constexpr (sizeof(T) == 2 && N % 2 == 0) {
        uint32_t *w = reinterpret_cast<uint32_t *>(&a);
#pragma unroll
        for (int i = 0; i < N / 2; ++i) w[i] = Pair<T>::of(x[2 * i], x[2 * i + 1]);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) a.v[i] = to_out_t<T>(x[i]);
    }
    *reinterpret_cast<Pack<T, N> *>(p) = a;
}

// ---------------------------------------------------------------- pairs of fp32 values, one instruction for both
struct F2 {
    uint64_t v;
    __device__ __forceinline__ F2() {}
    __device__ __forceinline__ F2(float x, float y) { asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(x), "f"(y)); }
    __device__ __forceinline__ explicit F2(float x) : F2(x, x) {}
    __device__ __forceinline__ void get(float &x, float &y) const { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
};
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return d;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
    return d;
}

// 16 bytes from global to shared memory without waiting; zeros where `on` is false.  For long contiguous rows: L2 fetches
// 256 bytes at a time.
__device__ __forceinline__ void copy16(void *dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global.L2::256B [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
template <int BYTES> __device__ __forceinline__ void copy_piece(void *dst, const void *src) {  // 4, 8 or 16
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(smem_u32(dst)), "l"(src), "n"(BYTES) : "memory");
}
__device__ __forceinline__ void copies_issued() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most LEFT of the thread's groups of copies are under way.
template <int LEFT> __device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// n / d for n < 2^31 by one multiplication: with s = ceil(log2 d) and m = ceil(2^(31 + s) / d) the error
// m d - 2^(31 + s) is below d <= 2^s, so n m / 2^(31 + s) exceeds n / d by less than 1 / d.
struct FastDiv {
    uint32_t d, m, s;
    static FastDiv of(uint32_t d) {
        uint32_t s = 0;
        while ((1ull << s) < d) ++s;
        return {d, (uint32_t)(((1ull << (31 + s)) + d - 1) / d), 31 + s};
    }
    __device__ __forceinline__ uint32_t div(uint32_t n) const { return (uint32_t)(((uint64_t)n * m) >> s); }
};

// Where row (token, head) of a strided tensor starts, rows counted token by token.
struct RowMap {
    int64_t ts, hs;
    __device__ __forceinline__ int64_t at(uint32_t row, const FastDiv &heads) const {
        if (heads.d == 1) return (int64_t)row * ts;
        const uint32_t t = heads.div(row);
        return (int64_t)t * ts + (int64_t)(row - t * heads.d) * hs;
    }
};

struct GatedNormParams {
    const void *dy, *x, *z, *weight;
    void *y, *dx, *dz, *dweight;
    float *part;  // backward: [CTAs][dim] column sums
    RowMap dym, xm, zm;
    FastDiv heads;
    uint32_t rows;
    int dim, dtype, weight_dtype, act;
    float eps;
    bool vec;  // rows are moved in 16-byte pieces
};

struct AddNormParams {
    const void *dy, *dres, *x, *residual, *weight, *scale_vec;
    void *y, *residual_out, *dx, *dresidual, *dweight, *dscale;
    float *part;  // backward: [CTAs][1 or 2][dim] column sums
    int64_t dy_ts, dres_ts, x_ts, r_ts, ro_ts;
    uint32_t rows;
    int dim, dtype, residual_dtype, weight_dtype, scale_dtype;
    float scale, eps;
    bool vec;
};

// Rows of the recurrence between saved states; channels of a tile; CTAs of a cluster, at most.
constexpr int LR_SAVE = 16, LR_CH = 32, LR_MAX_CLUSTER = 16;

struct LinrecParams {
    const void *x, *g, *dh;
    const float *h0, *dht;
    const int32_t *cu;
    void *h, *dx, *dg;
    float *ht, *dh0, *states;
    int64_t x_ts, g_ts, dh_ts;
    int rows, tokens, dim, N, complement;  // rows = batch * tokens; N sequences
    int dtype, gate_dtype;
    bool vec;    // rows can be moved by tensor maps
    int x_piece, g_piece;  // else: elements moved together in rows of activations and of gates, 4, 2 or 1
    bool clear;  // the kernel's first CTA sets the status word
    uint32_t spin;
    int *status;
    int tiles, cluster, supers;  // tiles of rows, CTAs of a cluster, clusters' worth of rows
    FastDiv per_seq;             // divides by tokens
};

struct LinrecMaps {
    CUtensorMap g, x, dh;
};

// A launch of a kernel of the recurrence: what is known of it beforehand, and the configuration that linrec_plan makes.
struct LinrecLaunch {
    const void *kernel;
    int threads, smem;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    LinrecLaunch(const void *k, int t, int s) : kernel(k), threads(t), smem(s) {}
};

struct StepParams {
    const void *x, *g;
    const int32_t *slots;
    float *state;
    void *y;
    int64_t x_ts, g_ts, batch, num_slots;
    int dim, dtype, gate_dtype, complement;
    bool vec;
    FastDiv pieces;
};

// CTAs that write partial column sums, at most (the workspace is sized for it).
constexpr int NORM_MAX_PARTS = 152 * 8;
int norm_parts(int64_t rows, int64_t dim);
cudaError_t norm_grid(const void *kernel, int threads, int ctas, int smem, int max_smem, int64_t rows, int rows_per_cta,
                      int most, int &grid);
// A launch whose CTAs form clusters of `ctas`.
struct ClusterLaunch {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr = {};
    ClusterLaunch(int grid, int threads, int smem, int ctas, cudaStream_t stream) {
        cfg.gridDim = dim3((unsigned)grid);
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = (size_t)smem;
        cfg.stream = stream;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = (unsigned)ctas;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
    }
    ClusterLaunch(const ClusterLaunch &) = delete;
};

cudaError_t launch_gated_norm_fwd(const GatedNormParams &p, cudaStream_t stream);
cudaError_t launch_gated_norm_bwd(const GatedNormParams &p, cudaStream_t stream);
cudaError_t launch_add_norm_fwd(const AddNormParams &p, cudaStream_t stream);
cudaError_t launch_add_norm_bwd(const AddNormParams &p, cudaStream_t stream);
cudaError_t linrec_plan(LinrecParams &p, LinrecLaunch &l, int rows_per_tile, bool *narrow, cudaStream_t stream);
cudaError_t linrec_maps(const LinrecParams &p, LinrecMaps &maps, int rows_per_tile);
// Tensor map of rows [rows][dim] at a distance of `stride` elements, for boxes of box_rows x box_cols; what lies outside
// reads as zero.  Base, stride and box_cols in bytes must be multiples of 16.
cudaError_t encode_matrix_map(CUtensorMap *map, const void *base, int dtype, int64_t rows, int64_t dim, int64_t stride,
                              int box_rows, int box_cols);
cudaError_t launch_linrec_fwd(LinrecParams p, cudaStream_t stream);
cudaError_t launch_linrec_bwd(LinrecParams p, cudaStream_t stream);
cudaError_t launch_linrec_step(StepParams p, cudaStream_t stream);

}  // namespace gdr
