// k15_ffn_rows.cu -- what surrounds the feed-forward's large products: its forward pass for few tokens, the element-wise part of
// its backward pass, and rows brought to 16-byte boundaries for the tensor maps.
#include "ffn.h"
#include "ffn_act.cuh"

namespace gdr {
namespace {

// ---------------------------------------------------------------- few tokens
// The weights' bytes bound it: 4 inner dim of them for 4 tokens inner dim operations.  A CTA has 8 or 16 rows of both weights, its
// warps a part of the summed axis each; the weights go from global memory to the registers of the products (mma.sync: rows 0
// to 7 of a product are gates, 8 to 15 the values beside them, tokens its 8 columns) without a stop in shared memory.  The
// summed axis may be taken in any order, so each lane's 16 bytes of a row, eight neighbours, stand for the pairs of both halves
// of two products, and x is read the same way, from L1: with more than 8 tokens each piece of x meets two eights of rows.
constexpr int FEW_ROWS = 8;

template <typename T> __device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                                uint32_t b0, uint32_t b1) {
    if constexpr (sizeof(T) == 2 && __is_same(T, __nv_bfloat16))
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight neighbours of a row from k on, zeros past the row's end or where the row is none.
template <bool VEC, bool STREAM> __device__ __forceinline__ uint4 eight(const uint16_t *row, int k, int dim, bool on) {
    uint4 r = make_uint4(0, 0, 0, 0);
    if constexpr (VEC) {
        if (on && k < dim) {
            if constexpr (STREAM)
                asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
                             : "l"(row + k));
            else
                r = __ldg(reinterpret_cast<const uint4 *>(row + k));
        }
    } else {
        uint32_t e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = on && k + i < dim ? __ldg(row + k + i) : 0;
        r = make_uint4(e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16);
    }
    return r;
}

// NT: eights of tokens; NR: eights of rows; AHEAD: steps of 64 of the summed axis of which a warp has the weights under way at
// a time; CTAS: of a processor, at least.
template <int NT, int NR, int AHEAD, int WARPS, int CTAS, int ACT, bool VEC, typename T>
__global__ void __launch_bounds__(WARPS * 32, CTAS) k15_few(const FfnFew p) {
    __shared__ float sums[WARPS][NR * NT * 4][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, row0 = blockIdx.x * FEW_ROWS * NR + r;
    const uint16_t *x = static_cast<const uint16_t *>(p.x), *wg = static_cast<const uint16_t *>(p.wg), *wu = static_cast<const uint16_t *>(p.wu);
    bool live[NR];
    int64_t g_at[NR], u_at[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
        live[i] = row0 + i * FEW_ROWS < p.inner;
        g_at[i] = live[i] ? (row0 + i * FEW_ROWS) * p.wg_rs : 0, u_at[i] = live[i] ? (row0 + i * FEW_ROWS) * p.wu_rs : 0;
    }
    float acc[NR][NT][4] = {};
    constexpr int STEP = WARPS * 64;
#pragma unroll 1
    for (int k0 = warp * 64 + c * 8; k0 - c * 8 < p.dim; k0 += STEP * AHEAD) {
        uint4 g[AHEAD][2][NR], u[AHEAD][2][NR];
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < NR; ++i) {
                    g[s][j][i] = eight<VEC, true>(wg + g_at[i], k0 + s * STEP + j * 32, p.dim, live[i]);
                    u[s][j][i] = eight<VEC, true>(wu + u_at[i], k0 + s * STEP + j * 32, p.dim, live[i]);
                }
#pragma unroll
        for (int s = 0; s < AHEAD; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int token = t * 8 + r;
                    const bool there = token < p.tokens;
                    const uint4 b = eight<VEC, false>(x + (there ? token * p.x_ts : 0), k0 + s * STEP + j * 32, p.dim, there);
#pragma unroll
                    for (int i = 0; i < NR; ++i) {
                        mma16816<T>(acc[i][t], g[s][j][i].x, u[s][j][i].x, g[s][j][i].y, u[s][j][i].y, b.x, b.y);
                        mma16816<T>(acc[i][t], g[s][j][i].z, u[s][j][i].z, g[s][j][i].w, u[s][j][i].w, b.z, b.w);
                    }
                }
    }
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int j = 0; j < 4; ++j) sums[warp][(i * NT + t) * 4 + j][lane] = acc[i][t][j];
    __syncthreads();
    for (int n = threadIdx.x; n < FEW_ROWS * NR * 8 * NT; n += WARPS * 32) {
        const int row = n % (FEW_ROWS * NR), i = blockIdx.x * FEW_ROWS * NR + row, token = n / (FEW_ROWS * NR);
        if (token >= p.tokens || i >= p.inner) continue;
        const int at = row % FEW_ROWS * 4 + token % 8 / 2, j = (row / FEW_ROWS * NT + token / 8) * 4 + token % 2;
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) a += sums[w][j][at], b += sums[w][j + 2][at];
        const int64_t to = (int64_t)token * p.inner + i;
        if (p.gate) p.gate[to] = a, p.up[to] = b;
        if (p.h) static_cast<T *>(p.h)[to] = to_out_t<T>(activate<ACT>(a) * b);
    }
}

template <int NT, int NR, int AHEAD, int WARPS, int CTAS, int ACT, bool VEC, typename T> cudaError_t few_launch(const FfnFew &p, cudaStream_t stream) {
    const unsigned grid = (unsigned)((p.inner + FEW_ROWS * NR - 1) / (FEW_ROWS * NR));
    k15_few<NT, NR, AHEAD, WARPS, CTAS, ACT, VEC, T><<<grid, WARPS * 32, 0, stream>>>(p);
    return cudaGetLastError();
}
template <int ACT, bool VEC, typename T> cudaError_t few_t(const FfnFew &p, cudaStream_t stream) {
    // Few rows of long ones: 16 warps share a CTA's (4096 x 1024, 8 tokens: 10.6 us with 4 warps, 5.5 with 16).
    if (p.inner <= 16 * 152 && p.dim > 512) {
        if (p.tokens <= 8) return few_launch<1, 1, 2, 16, 1, ACT, VEC, T>(p, stream);
        if (p.tokens <= 16) return few_launch<2, 1, 1, 16, 1, ACT, VEC, T>(p, stream);
        return few_launch<4, 1, 1, 16, 1, ACT, VEC, T>(p, stream);
    }
    // Rows off 16 bytes are read element by element, with up to 488 bytes of spills: 8 tokens of 1001 x 2731 take 14.4 us, of
    // 2047 x 8191 48 (32 tokens: 32 and 58).
    // 2048 x 8192, 8 tokens: 1024 CTAs, 6.7 for each processor, all of them resident at once: 12.3 us (5.5 TB/s).  More tokens, with
    // 16 rows to a CTA in place of 8: 16 of them 13.9 us (17.2), 32 17.5 (23.7).
    if (p.tokens <= 8) return few_launch<1, 1, 4, 4, 7, ACT, VEC, T>(p, stream);
    if (p.tokens <= 16) return few_launch<2, 2, 2, 4, 4, ACT, VEC, T>(p, stream);
    return few_launch<4, 2, 1, 4, 4, ACT, VEC, T>(p, stream);
}

// ---------------------------------------------------------------- element-wise part of the backward pass
constexpr int ROW_THREADS = 256;

__device__ __forceinline__ void clear_status(uint8_t *status) {
    static_assert(GDR_FFN_STATUS_BYTES <= ROW_THREADS);
    if (blockIdx.x == 0 && threadIdx.x < GDR_FFN_STATUS_BYTES) status[threadIdx.x] = 0;
}

// dg and du are rounded to the operands' type, since the tensor cores take nothing else beside x and the weights: up to half a step
// of each more in the gradients (bf16 0.0023 off in place of 0.0017); in fp16 what passes 65504 becomes infinite and what is
// below 2^-25 is lost, as for any gradient of that type.
// Rows that are multiples of 16 bytes: 8 elements for each thread.  Others: 256 for each warp, its lanes side by side.
template <int ACT, bool VEC, typename T> __global__ void __launch_bounds__(ROW_THREADS) k15_act(const FfnAct p, const FastDiv blocks) {
    clear_status(p.status);
    const T *dh = static_cast<const T *>(p.dh);
    T *dg = static_cast<T *>(p.dg), *du = static_cast<T *>(p.du);
    if constexpr (VEC) {
        const uint32_t i = blockIdx.x * ROW_THREADS + threadIdx.x, row = blocks.div(i);
        if (row >= p.tokens) return;
        const int64_t col = (int64_t)(i - row * blocks.d) * 8, at = row * p.inner + col, to = row * p.pitch + col;
        float d[8], g[8], u[8];
        load8(dh + row * p.dh_ts + col, d), load8(p.gate + at, g), load8(p.up + at, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a, da;
            activate_slope<ACT>(g[j], a, da);
            g[j] = d[j] * u[j] * da, u[j] = d[j] * a;
        }
        store_pack<T, 8>(dg + to, g);
        store_pack<T, 8>(du + to, u);
    } else {
        const uint32_t i = blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32, row = blocks.div(i);
        if (row >= p.tokens) return;
        const int64_t col = (int64_t)(i - row * blocks.d) * 256 + threadIdx.x % 32, at = row * p.inner + col, to = row * p.pitch + col;
        float d[8], g[8], u[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const bool on = col + 32 * j < p.inner;
            d[j] = on ? to_f32(dh[row * p.dh_ts + col + 32 * j]) : 0.f;
            g[j] = on ? p.gate[at + 32 * j] : 0.f, u[j] = on ? p.up[at + 32 * j] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float a, da;
            activate_slope<ACT>(g[j], a, da);
            if (col + 32 * j < p.inner) dg[to + 32 * j] = to_out_t<T>(d[j] * u[j] * da), du[to + 32 * j] = to_out_t<T>(d[j] * a);
        }
    }
}

template <int ACT, typename T> cudaError_t act_of(const FfnAct &p, cudaStream_t stream) {
    const int64_t per_row = p.vec ? p.inner / 8 : (p.inner + 255) / 256, threads = p.tokens * per_row * (p.vec ? 1 : 32);
    const FastDiv blocks = FastDiv::of((uint32_t)per_row);
    const unsigned grid = (unsigned)((threads + ROW_THREADS - 1) / ROW_THREADS);
    if (p.vec) k15_act<ACT, true, T><<<grid, ROW_THREADS, 0, stream>>>(p, blocks);
    else k15_act<ACT, false, T><<<grid, ROW_THREADS, 0, stream>>>(p, blocks);
    return cudaGetLastError();
}
template <typename T> cudaError_t act_t(const FfnAct &p, cudaStream_t stream) {
    return p.act == FFN_SILU ? act_of<FFN_SILU, T>(p, stream) : p.act == FFN_SIGMOID ? act_of<FFN_SIGMOID, T>(p, stream)
                                                                                    : act_of<FFN_GELU_TANH, T>(p, stream);
}

// ---------------------------------------------------------------- rows to 16-byte boundaries
// 256 elements of a row for each warp, its lanes side by side.
__global__ void __launch_bounds__(ROW_THREADS) k15_pad(const FfnPad p) {
    clear_status(p.status);
    uint32_t i = blockIdx.x * (ROW_THREADS / 32) + threadIdx.x / 32;
    int m = 0;
    while (m < p.count && i >= p.warps[m]) i -= p.warps[m++];
    if (m == p.count) return;
    const uint32_t row = p.per_row.div(i);
    const int col = (int)(i - row * p.per_row.d) * 256 + (int)(threadIdx.x % 32);
    const uint16_t *from = static_cast<const uint16_t *>(p.from[m]) + row * p.stride[m];
    uint16_t *to = static_cast<uint16_t *>(p.to[m]) + row * p.pitch;
    uint16_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col + 32 * j < p.cols ? from[col + 32 * j] : 0;
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (col + 32 * j < p.pitch) to[col + 32 * j] = v[j];
}

}  // namespace

cudaError_t launch_ffn_few(const FfnFew &p, cudaStream_t stream) {
#define BY_ACT(VEC, T)                                                      \
    (p.act == FFN_SILU      ? few_t<FFN_SILU, VEC, T>(p, stream)            \
     : p.act == FFN_SIGMOID ? few_t<FFN_SIGMOID, VEC, T>(p, stream)         \
                            : few_t<FFN_GELU_TANH, VEC, T>(p, stream))
    if (p.dtype == BF16) return p.vec ? BY_ACT(true, __nv_bfloat16) : BY_ACT(false, __nv_bfloat16);
    return p.vec ? BY_ACT(true, __half) : BY_ACT(false, __half);
#undef BY_ACT
}

cudaError_t launch_ffn_act(const FfnAct &p, cudaStream_t stream) {
    return p.dtype == BF16 ? act_t<__nv_bfloat16>(p, stream) : act_t<__half>(p, stream);
}

cudaError_t launch_ffn_pad(FfnPad p, cudaStream_t stream) {
    p.pitch = (p.cols + 7) / 8 * 8;
    p.per_row = FastDiv::of((uint32_t)((p.pitch + 255) / 256));
    int64_t warps = 0;
    for (int m = 0; m < p.count; ++m) warps += p.warps[m] = (uint32_t)(p.rows[m] * p.per_row.d);
    k15_pad<<<(unsigned)((warps + ROW_THREADS / 32 - 1) / (ROW_THREADS / 32)), ROW_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdr
