// k9_norms.cuh -- the norms on both sides of a block, forward and backward (included once per activation type):
//
//   after, over each head of D channels      y = w x rs act(z)            rs = (mean(x^2) + eps)^-1/2
//     t = dy act(z) w ;  dx = rs t - x rs^3 mean(t x) ;  dz = dy x rs w act'(z) ;  dw = sum over rows of dy act(z) x rs
//   before, over the residual stream         r = res + s x ;  y = w r rs  rs = (mean(r^2) + eps)^-1/2
//     t = dy w ;  dr = rs t - r rs^3 mean(t r) + dres ;  dx = s dr ;  dw = sum of dy r rs ;  ds = sum of dr x
//
// Both row sums of a backward (of squares and of t x) come from one pass over values that stay in registers, so
// every input is read once and every output written once: the kernels are bound by HBM.  A row belongs to a group
// of G threads, each holding NV pieces of VEC elements; groups of up to 32 threads sum by shuffles, larger ones
// (one row per CTA) through shared memory.  The grid is persistent, so the weights are read once per thread and the
// column sums of a backward (dw, ds) stay in registers until the CTA writes its partial row; k9_colsum adds the
// partial rows in a fixed order.
#pragma once

#include "block_common.cuh"

namespace gdr {
namespace {

constexpr int NORM_THREADS = 256;  // of a CTA whose groups are warps or parts of one

template <typename T> __device__ __forceinline__ float sigmoid_t(float z) {
    // 16-bit results: the fast exponential and reciprocal are 3e-7 off, far below the result's 4e-3 or 5e-4
    if constexpr (sizeof(T) == 2) return __fdividef(1.f, 1.f + __expf(-z));
    return 1.f / (1.f + expf(-z));
}

// Sums of two values over the group's G threads, in the same order whatever the row.
template <int G> struct GroupSum {
    static constexpr int NW = G > 32 ? G / 32 : 1;
    float2 *red;  // [2][NW] in shared memory (G > 32)
    int buf;
    __device__ __forceinline__ explicit GroupSum(float2 *r) : red(r), buf(0) {}
    __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int o = (G < 32 ? G : 32) / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if constexpr (G > 32) {
            // two buffers in turn: a warp can only be back at this one after the next row's barrier
            if ((threadIdx.x & 31) == 0) red[buf * NW + (threadIdx.x >> 5)] = make_float2(a, b);
            __syncthreads();
            a = b = 0.f;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                const float2 x = red[buf * NW + i];
                a += x.x;
                b += x.y;
            }
            buf ^= 1;
        }
        return make_float2(a, b);
    }
};

// The gradient of x rs with respect to x along t: rs t - x rs^3 mean(t x).  A row of one channel has t x for its mean and
// the terms cancel to eps rs^3 t, which is formed directly.
struct NormGrad {
    float t, x;
    __device__ __forceinline__ NormGrad(float rs, float mean, int dim, float eps)
        : t(dim == 1 ? rs * rs * rs * eps : rs), x(dim == 1 ? 0.f : rs * rs * rs * mean) {}
    __device__ __forceinline__ float operator()(float tv, float xv) const { return fmaf(tv, t, -xv * x); }
};

// The thread's columns: piece i starts at column (t + i G) VEC.
template <int VEC, int G, int NV> struct Cols {
    int t;
    bool on[NV];
    __device__ __forceinline__ Cols(int t_, int dim) : t(t_) {
#pragma unroll
        for (int i = 0; i < NV; ++i) on[i] = (t + i * G) * VEC < dim;
    }
    __device__ __forceinline__ int at(int i) const { return (t + i * G) * VEC; }
};

template <int VEC, int G, int NV>
__device__ __forceinline__ void load_cols(const void *p, int dt, const Cols<VEC, G, NV> &c, float fill,
                                          float (&o)[NV][VEC]) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < VEC; ++j) o[i][j] = p && c.on[i] ? load_scalar(p, c.at(i) + j, dt) : fill;
}

// The CTA's column sums to its partial row: the groups of a CTA are added in order.
template <int VEC, int G, int NV>
__device__ __forceinline__ void write_part(float *part, float *smem, const Cols<VEC, G, NV> &c, int dim,
                                           const float (&acc)[NV][VEC]) {
    constexpr int RPC = G > 32 ? 1 : NORM_THREADS / G;
    if constexpr (RPC == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (c.on[i])
#pragma unroll
                for (int j = 0; j < VEC; ++j) part[c.at(i) + j] = acc[i][j];
    } else {
        constexpr int W = G * NV * VEC;  // columns held by a group
        const int gi = threadIdx.x / G;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) smem[gi * W + c.at(i) + j] = acc[i][j];
        __syncthreads();
        for (int col = threadIdx.x; col < dim; col += NORM_THREADS) {
            float s = 0.f;
            for (int r = 0; r < RPC; ++r) s += smem[r * W + col];
            part[col] = s;
        }
    }
}

template <int VEC, int G, int NV> constexpr int norm_threads() { return G > 32 ? G : NORM_THREADS; }
template <int VEC, int G, int NV> constexpr int part_smem() {
    return G > 32 ? 1 : NORM_THREADS / G * G * NV * VEC;  // floats
}

// ---------------------------------------------------------------- after a block
template <typename T, int VEC, int G, int NV>
__global__ void __launch_bounds__(norm_threads<VEC, G, NV>()) k9_gated_fwd(const GatedNormParams p) {
    constexpr int RPC = G > 32 ? 1 : NORM_THREADS / G;
    __shared__ float2 red[2 * GroupSum<G>::NW];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(threadIdx.x % G, p.dim);
    float w[NV][VEC];
    load_cols<VEC, G, NV>(p.weight, p.weight_dtype, c, 1.f, w);
    const float inv_dim = 1.f / (float)p.dim;
    for (int64_t base = (int64_t)blockIdx.x * RPC; base < p.rows; base += (int64_t)gridDim.x * RPC) {
        const uint32_t row = (uint32_t)base + threadIdx.x / G;
        const bool live = row < p.rows;
        const T *x = reinterpret_cast<const T *>(p.x) + (live ? p.xm.at(row, p.heads) : 0);
        const T *z = reinterpret_cast<const T *>(p.z) + (live ? p.zm.at(row, p.heads) : 0);
        float xv[NV][VEC], zv[NV][VEC], s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<T, VEC> a = {}, b = {};
            if (live && c.on[i]) {
                a = load_pack<T, VEC>(x + c.at(i));
                if (p.z) b = load_pack<T, VEC>(z + c.at(i));
            }
            unpack<T, VEC>(a, xv[i]);
            unpack<T, VEC>(b, zv[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) s1 = fmaf(xv[i][j], xv[i][j], s1);
        const float rs = rsqrtf(sum(s1, 0.f).x * inv_dim + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float y[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                float a = 1.f;
                if (p.z) {
                    a = sigmoid_t<T>(zv[i][j]);
                    if (p.act == 0) a *= zv[i][j];
                }
                y[j] = xv[i][j] * rs * w[i][j] * a;
            }
            if (live && c.on[i])
                store_pack<T, VEC>(reinterpret_cast<T *>(p.y) + (size_t)row * p.dim + c.at(i), y);
        }
    }
}

template <typename T, int VEC, int G, int NV>
__global__ void __launch_bounds__(norm_threads<VEC, G, NV>()) k9_gated_bwd(const GatedNormParams p) {
    constexpr int RPC = G > 32 ? 1 : NORM_THREADS / G;
    __shared__ float2 red[2 * GroupSum<G>::NW];
    __shared__ float psm[part_smem<VEC, G, NV>()];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(threadIdx.x % G, p.dim);
    float w[NV][VEC], dw[NV][VEC] = {};
    load_cols<VEC, G, NV>(p.weight, p.weight_dtype, c, 1.f, w);
    const float inv_dim = 1.f / (float)p.dim;
    for (int64_t base = (int64_t)blockIdx.x * RPC; base < p.rows; base += (int64_t)gridDim.x * RPC) {
        const uint32_t row = (uint32_t)base + threadIdx.x / G;
        const bool live = row < p.rows;
        const T *x = reinterpret_cast<const T *>(p.x) + (live ? p.xm.at(row, p.heads) : 0);
        const T *z = reinterpret_cast<const T *>(p.z) + (live ? p.zm.at(row, p.heads) : 0);
        const T *dy = reinterpret_cast<const T *>(p.dy) + (live ? p.dym.at(row, p.heads) : 0);
        float xv[NV][VEC], up[NV][VEC], dzv[NV][VEC], s1 = 0.f, s2 = 0.f;  // up = dy act(z), dzv = dy act'(z)
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<T, VEC> a = {}, b = {}, d = {};
            if (live && c.on[i]) {
                a = load_pack<T, VEC>(x + c.at(i));
                d = load_pack<T, VEC>(dy + c.at(i));
                if (p.z) b = load_pack<T, VEC>(z + c.at(i));
            }
            unpack<T, VEC>(a, xv[i]);
            unpack<T, VEC>(d, up[i]);
            unpack<T, VEC>(b, dzv[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                if (p.z) {
                    const float z1 = dzv[i][j], d = up[i][j], sg = sigmoid_t<T>(z1), rest = sg * (1.f - sg);
                    up[i][j] = d * (p.act == 0 ? z1 * sg : sg);
                    dzv[i][j] = d * (p.act == 0 ? fmaf(z1, rest, sg) : rest);
                }
                s1 = fmaf(xv[i][j], xv[i][j], s1);
                s2 = fmaf(up[i][j] * w[i][j], xv[i][j], s2);
            }
        const float2 s = sum(s1, s2);
        const float rs = rsqrtf(s.x * inv_dim + p.eps);
        const NormGrad q(rs, s.y * inv_dim, p.dim, p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float dx[VEC], dz[VEC];
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const float xr = xv[i][j] * rs;
                dx[j] = q(up[i][j] * w[i][j], xv[i][j]);
                dz[j] = dzv[i][j] * xr * w[i][j];
                dw[i][j] = fmaf(up[i][j], xr, dw[i][j]);  // (rows past the end hold zeros)
            }
            if (live && c.on[i]) {
                const size_t o = (size_t)row * p.dim + c.at(i);
                store_pack<T, VEC>(reinterpret_cast<T *>(p.dx) + o, dx);
                if (p.z) store_pack<T, VEC>(reinterpret_cast<T *>(p.dz) + o, dz);
            }
        }
    }
    if (p.dweight) write_part<VEC, G, NV>(p.part + (size_t)blockIdx.x * p.dim, psm, c, p.dim, dw);
}

// ---------------------------------------------------------------- before a block
template <typename T, typename R, int VEC, int G, int NV>
__global__ void __launch_bounds__(norm_threads<VEC, G, NV>()) k9_add_fwd(const AddNormParams p) {
    constexpr int RPC = G > 32 ? 1 : NORM_THREADS / G;
    __shared__ float2 red[2 * GroupSum<G>::NW];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(threadIdx.x % G, p.dim);
    float w[NV][VEC], sc[NV][VEC];
    load_cols<VEC, G, NV>(p.weight, p.weight_dtype, c, 1.f, w);
    load_cols<VEC, G, NV>(p.scale_vec, p.scale_dtype, c, p.scale, sc);
    const float inv_dim = 1.f / (float)p.dim;
    for (int64_t base = (int64_t)blockIdx.x * RPC; base < p.rows; base += (int64_t)gridDim.x * RPC) {
        const uint32_t row = (uint32_t)base + threadIdx.x / G;
        const bool live = row < p.rows;
        const T *x = reinterpret_cast<const T *>(p.x) + (int64_t)row * p.x_ts;
        const R *res = reinterpret_cast<const R *>(p.residual) + (int64_t)row * p.r_ts;
        float rv[NV][VEC], s1 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<T, VEC> a = {};
            Pack<R, VEC> b = {};
            if (live && c.on[i]) {
                a = load_pack<T, VEC>(x + c.at(i));
                if (p.residual) b = load_pack<R, VEC>(res + c.at(i));
            }
            float xv[VEC];
            unpack<T, VEC>(a, xv);
            unpack<R, VEC>(b, rv[i]);
#pragma unroll
            for (int j = 0; j < VEC; ++j) rv[i][j] = fmaf(sc[i][j], xv[j], rv[i][j]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) s1 = fmaf(rv[i][j], rv[i][j], s1);
        const float rs = rsqrtf(sum(s1, 0.f).x * inv_dim + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (live && c.on[i]) {
                float y[VEC];
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[j] = rv[i][j] * rs * w[i][j];
                store_pack<T, VEC>(reinterpret_cast<T *>(p.y) + (size_t)row * p.dim + c.at(i), y);
                if (p.residual_out)
                    store_pack<R, VEC>(reinterpret_cast<R *>(p.residual_out) + (int64_t)row * p.ro_ts + c.at(i), rv[i]);
            }
    }
}

template <typename T, typename R, int VEC, int G, int NV>
__global__ void __launch_bounds__(norm_threads<VEC, G, NV>()) k9_add_bwd(const AddNormParams p) {
    constexpr int RPC = G > 32 ? 1 : NORM_THREADS / G;
    __shared__ float2 red[2 * GroupSum<G>::NW];
    __shared__ float psm[part_smem<VEC, G, NV>()];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(threadIdx.x % G, p.dim);
    float w[NV][VEC], sc[NV][VEC], dw[NV][VEC] = {}, ds[NV][VEC] = {};
    load_cols<VEC, G, NV>(p.weight, p.weight_dtype, c, 1.f, w);
    load_cols<VEC, G, NV>(p.scale_vec, p.scale_dtype, c, p.scale, sc);
    const float inv_dim = 1.f / (float)p.dim;
    for (int64_t base = (int64_t)blockIdx.x * RPC; base < p.rows; base += (int64_t)gridDim.x * RPC) {
        const uint32_t row = (uint32_t)base + threadIdx.x / G;
        const bool live = row < p.rows;
        const T *dy = reinterpret_cast<const T *>(p.dy) + (int64_t)row * p.dy_ts;
        const T *x = reinterpret_cast<const T *>(p.x) + (int64_t)row * p.x_ts;
        const R *r = reinterpret_cast<const R *>(p.residual_out) + (int64_t)row * p.ro_ts;
        const R *dres = reinterpret_cast<const R *>(p.dres) + (int64_t)row * p.dres_ts;
        float rv[NV][VEC], up[NV][VEC], s1 = 0.f, s2 = 0.f;
        Pack<R, VEC> dr[NV] = {};
        Pack<T, VEC> xp[NV] = {};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            Pack<T, VEC> a = {};
            Pack<R, VEC> b = {};
            if (live && c.on[i]) {
                a = load_pack<T, VEC>(dy + c.at(i));
                b = load_pack<R, VEC>(r + c.at(i));
                if (p.dres) dr[i] = load_pack<R, VEC>(dres + c.at(i));
                if (p.dscale) xp[i] = load_pack<T, VEC>(x + c.at(i));
            }
            unpack<T, VEC>(a, up[i]);
            unpack<R, VEC>(b, rv[i]);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                s1 = fmaf(rv[i][j], rv[i][j], s1);
                s2 = fmaf(up[i][j] * w[i][j], rv[i][j], s2);
            }
        const float2 s = sum(s1, s2);
        const float rs = rsqrtf(s.x * inv_dim + p.eps);
        const NormGrad q(rs, s.y * inv_dim, p.dim, p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            float d[VEC], dx[VEC], xv[VEC];
            unpack<R, VEC>(dr[i], d);
            unpack<T, VEC>(xp[i], xv);
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                d[j] += q(up[i][j] * w[i][j], rv[i][j]);
                dx[j] = sc[i][j] * d[j];
                dw[i][j] = fmaf(up[i][j], rv[i][j] * rs, dw[i][j]);
                ds[i][j] = fmaf(d[j], xv[j], ds[i][j]);
            }
            if (live && c.on[i]) {
                const size_t o = (size_t)row * p.dim + c.at(i);
                if (p.dresidual) store_pack<R, VEC>(reinterpret_cast<R *>(p.dresidual) + o, d);
                if (p.dx) store_pack<T, VEC>(reinterpret_cast<T *>(p.dx) + o, dx);
            }
        }
    }
    float *part = p.part + (size_t)blockIdx.x * p.dim;
    if (p.dweight) write_part<VEC, G, NV>(part, psm, c, p.dim, dw);
    if (p.dweight) part += (size_t)gridDim.x * p.dim;
    if (p.dscale) write_part<VEC, G, NV>(part, psm, c, p.dim, ds);
}

// ---------------------------------------------------------------- choice of the group
// The fewest threads that hold a row in at most 4 pieces (16 single elements), up to 1024 threads.
#define NORM_DISPATCH(T, vec, dim, CALL)                              \
    do {                                                              \
        if (vec) {                                                    \
            constexpr int VE = 16 / (int)sizeof(T);                   \
            const int n = (dim) / VE;                                 \
            if (n <= 8) { CALL(VE, 8, 1); }                           \
            else if (n <= 16) { CALL(VE, 16, 1); }                    \
            else if (n <= 32) { CALL(VE, 32, 1); }                    \
            else if (n <= 64) { CALL(VE, 32, 2); }                    \
            else if (n <= 256) { CALL(VE, 128, 2); }                  \
            else if (n <= 512) { CALL(VE, 256, 2); }                  \
            else if (n <= 1024) { CALL(VE, 512, 2); }                 \
            else if (n <= 2048) { CALL(VE, 512, 4); }                 \
            else { CALL(VE, 1024, 4); }                               \
        } else {                                                      \
            if ((dim) <= 128) { CALL(1, 32, 4); }                     \
            else if ((dim) <= 512) { CALL(1, 32, 16); }               \
            else if ((dim) <= 2048) { CALL(1, 256, 8); }              \
            else { CALL(1, 1024, 16); }                               \
        }                                                             \
    } while (0)

// CTAs of a persistent grid: `threads_per_sm` threads on each of the device's SMs, no more than there are rows for.
inline int norm_grid(int64_t rows, int threads, int rows_per_cta, int threads_per_sm, int most) {
    int sms = 152;
    if (device_sm_count(&sms) != cudaSuccess || sms < 1) sms = 152;
    int64_t grid = (int64_t)sms * (threads_per_sm / threads > 0 ? threads_per_sm / threads : 1);
    const int64_t need = (rows + rows_per_cta - 1) / rows_per_cta;
    if (grid > need) grid = need;
    if (grid > most) grid = most;
    return (int)(grid < 1 ? 1 : grid);
}

}  // namespace

cudaError_t launch_colsum(const float *part, int parts, int dim, void *out, int dtype, cudaStream_t stream);

template <typename T> cudaError_t gated_norm_fwd_t(const GatedNormParams &p, cudaStream_t stream) {
#define CALL(V, G, NV)                                                                                              \
    k9_gated_fwd<T, V, G, NV><<<norm_grid(p.rows, norm_threads<V, G, NV>(), norm_threads<V, G, NV>() / G, 2048, 1 << 30), \
                                norm_threads<V, G, NV>(), 0, stream>>>(p)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
    return cudaGetLastError();
}

template <typename T> cudaError_t gated_norm_bwd_t(const GatedNormParams &p, cudaStream_t stream) {
    const int most = norm_parts(p.rows, p.dim);
    int grid = 0;
#define CALL(V, G, NV)                                                                                    \
    grid = norm_grid(p.rows, norm_threads<V, G, NV>(), norm_threads<V, G, NV>() / G, 1024, most),         \
    k9_gated_bwd<T, V, G, NV><<<grid, norm_threads<V, G, NV>(), 0, stream>>>(p)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
    cudaError_t e = cudaGetLastError();
    if (e == cudaSuccess && p.dweight) e = launch_colsum(p.part, grid, p.dim, p.dweight, p.weight_dtype, stream);
    return e;
}

template <typename T, typename R> cudaError_t add_norm_fwd_t(const AddNormParams &p, cudaStream_t stream) {
#define CALL(V, G, NV)                                                                                                \
    k9_add_fwd<T, R, V, G, NV><<<norm_grid(p.rows, norm_threads<V, G, NV>(), norm_threads<V, G, NV>() / G, 2048, 1 << 30), \
                                 norm_threads<V, G, NV>(), 0, stream>>>(p)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
    return cudaGetLastError();
}

template <typename T, typename R> cudaError_t add_norm_bwd_t(const AddNormParams &p, cudaStream_t stream) {
    const int most = norm_parts(p.rows, p.dim);
    int grid = 0;
#define CALL(V, G, NV)                                                                                    \
    grid = norm_grid(p.rows, norm_threads<V, G, NV>(), norm_threads<V, G, NV>() / G, 1024, most),         \
    k9_add_bwd<T, R, V, G, NV><<<grid, norm_threads<V, G, NV>(), 0, stream>>>(p)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
    cudaError_t e = cudaGetLastError();
    const float *part = p.part;
    if (e == cudaSuccess && p.dweight) {
        e = launch_colsum(part, grid, p.dim, p.dweight, p.weight_dtype, stream);
        part += (size_t)grid * p.dim;
    }
    if (e == cudaSuccess && p.dscale) e = launch_colsum(part, grid, p.dim, p.dscale, p.scale_dtype, stream);
    return e;
}

// what a translation unit instantiates for its activation type
#define NORM_INSTANTIATE(T)                                                                \
    template cudaError_t gated_norm_fwd_t<T>(const GatedNormParams &, cudaStream_t);       \
    template cudaError_t gated_norm_bwd_t<T>(const GatedNormParams &, cudaStream_t);       \
    template cudaError_t add_norm_fwd_t<T, T>(const AddNormParams &, cudaStream_t);        \
    template cudaError_t add_norm_bwd_t<T, T>(const AddNormParams &, cudaStream_t);
#define NORM_INSTANTIATE_F32_STREAM(T)                                                     \
    template cudaError_t add_norm_fwd_t<T, float>(const AddNormParams &, cudaStream_t);    \
    template cudaError_t add_norm_bwd_t<T, float>(const AddNormParams &, cudaStream_t);

}  // namespace gdr
