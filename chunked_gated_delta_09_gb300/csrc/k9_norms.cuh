// k9_norms.cuh -- the norms on both sides of a block, forward and backward (included once per activation type):
//
//   after, over each head of D channels      y = w x rs act(z)            rs = (mean(x^2) + eps)^-1/2
//     t = dy act(z) w ;  dx = rs t - x rs^3 mean(t x) ;  dz = dy x rs w act'(z) ;  dw = sum over rows of dy act(z) x rs
//   before, over the residual stream         r = res + s x ;  y = w r rs  rs = (mean(r^2) + eps)^-1/2
//     t = dy w ;  dr = rs t - r rs^3 mean(t r) + dres ;  dx = s dr ;  dw = sum of dy r rs ;  ds = sum of dr x
//
// Both row sums of a backward (of squares and of t x) come from one pass over values that stay in registers, so
// every input is read once and every output written once: the kernels are bound by HBM, which a plain copy moves at
// 6.8 TB/s.  After a block, 32768 x 16 x 128 bf16: forward 0.064 ms (6.3 TB/s), backward 0.126 ms with its column sums (5.3
// TB/s; instructions are issued in 79 % of the cycles, the activation and its derivative for every element).  Before one:
// forward 48763 x 4096 bf16 0.252 ms (6.3), backward 0.309 (6.5); 32768 x 2048 bf16 on an fp32 stream 0.134 (6.0), backward
// with the gradient of the scale 0.198 (6.1).  Few rows take the time of a launch.  A row belongs to 8, 16 or 32 lanes, to
// a whole CTA of up to 1024 threads, a piece of VEC elements for each, or to a cluster of CTAs of up to 512 (4000 x 16384 bf16
// on an fp32 stream forward 0.159 ms, backward 0.242; one CTA with two pieces to a thread 0.177, 0.368; clusters of CTAs of
// 1024, one to an SM, 0.179, 0.257; for 8000 x 8192 one CTA is faster, 0.129, 0.216 against 0.151, 0.225).  Lanes sum by
// shuffles, CTAs and clusters through shared memory.  The grid is persistent: the weights are read once per thread, and the
// column sums of a backward (dw, ds) stay in registers until the CTA writes its partial row, which k9_colsum adds in a fixed
// order.
// The rows ahead come in one of three ways (see Ahead), whichever measured fastest for the kernel.
#pragma once

#include "block_common.cuh"

namespace gdr {
namespace {

constexpr int NORM_THREADS = 256;  // of a CTA whose groups are warps or parts of one

template <typename T> __device__ __forceinline__ float sigmoid_t(float z) {
    if constexpr (sizeof(T) == 2) {
        // 16-bit results: the approximate exponential and reciprocal are 3e-7 off near 0; the exponent's own rounding grows with
        // it, to 3e-6 at z = -80: fewer bits than fp32 has, far below the result's 4e-3 or 5e-4
        float e;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(z * -1.44269504f));
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(1.f + e));
        return e;
    }
    return 1.f / (1.f + expf(-z));
}
constexpr int ACT_NONE = 2;  // besides the C interface's silu and sigmoid

// A row's threads: G lanes, a whole CTA, or the CTAs of a cluster.
constexpr int WHOLE = 0, SPREAD = -1, MAX_SPREAD = 8;

__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ int cluster_ctas() {
    int n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_meet() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sums of two values over the row's threads, in the same order whatever the row.
template <int G> struct GroupSum {
    static constexpr int PLACES = G > 0 ? 1 : 2 * 32 * (G == SPREAD ? MAX_SPREAD : 1);
    float2 *red;  // [2][CTAs][32 warps] in shared memory
    int buf = 0;
    __device__ __forceinline__ explicit GroupSum(float2 *r) : red(r) {
        if (G == SPREAD) cluster_meet();  // every CTA runs: its shared memory may be written
    }
    // TWO: b is wanted too
    template <bool TWO = true> __device__ __forceinline__ float2 operator()(float a, float b) {
#pragma unroll
        for (int o = (G > 0 ? G : 32) / 2; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            if (TWO) b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if constexpr (G <= 0) {
            // two buffers in turn: a warp can only be back at this one after the next row's barrier
            const int nw = blockDim.x / 32, lane = threadIdx.x & 31, w = threadIdx.x >> 5;
            float2 x = make_float2(0.f, 0.f);
            if constexpr (G == SPREAD) {
                const int ctas = cluster_ctas();
                float2 *at = red + buf * MAX_SPREAD * 32;
                if (lane < ctas) {  // a lane for each CTA, its own among them
                    uint32_t to;
                    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(smem_u32(at + cluster_rank() * 32 + w)), "r"(lane));
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(a), "f"(b) : "memory");
                }
                cluster_meet();
                for (int q = 0; q < ctas; ++q)
                    if (lane < nw) x.x += at[q * 32 + lane].x, x.y += at[q * 32 + lane].y;
            } else {
                if (lane == 0) red[buf * 32 + w] = make_float2(a, b);
                __syncthreads();
                if (lane < nw) x = red[buf * 32 + lane];
            }
            a = x.x, b = x.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                a += __shfl_xor_sync(0xffffffffu, a, o);
                if (TWO) b += __shfl_xor_sync(0xffffffffu, b, o);
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

// The thread's columns: piece i starts at column (t + i threads) VEC; threads: of a row.
template <int VEC, int G, int NV> struct Cols {
    int t, step, dim;
    bool on[NV];
    __device__ __forceinline__ explicit Cols(int dim_)
        : t(G > 0 ? threadIdx.x % (G > 0 ? G : 1) : threadIdx.x + (G == SPREAD ? cluster_rank() * blockDim.x : 0)),
          step(G > 0 ? G : blockDim.x), dim(dim_) {
#pragma unroll
        for (int i = 0; i < NV; ++i) on[i] = (t + i * step) * VEC < dim;
    }
    __device__ __forceinline__ int at(int i) const { return (t + i * step) * VEC; }
};
// Rows that a CTA works on at a time, and the thread's among them.
template <int G> __device__ __forceinline__ int cta_rows() { return G > 0 ? NORM_THREADS / (G > 0 ? G : 1) : 1; }
template <int G> __device__ __forceinline__ int cta_row() { return G > 0 ? threadIdx.x / (G > 0 ? G : 1) : 0; }
// What shares out the rows, CTAs or clusters, and which of them this is.
template <int G> __device__ __forceinline__ uint32_t walkers() { return G == SPREAD ? gridDim.x / cluster_ctas() : gridDim.x; }
template <int G> __device__ __forceinline__ uint32_t walker() { return G == SPREAD ? blockIdx.x / cluster_ctas() : blockIdx.x; }

// How the rows ahead come.
//   RING   by asynchronous copies to places in shared memory, several rows ahead, which takes no registers: the backward
//          kernels (32768 x 16 x 128 bf16 after a block 0.126 ms; PAIR 0.143; 48763 x 4096 bf16 before one 0.309; PAIR 0.484),
//          and the forward before a block on a 16-bit stream (48763 x 4096 0.252 ms; PAIR 0.271)
//   PAIR   the next row's pieces in registers while a row is worked on: the forward after a block (32768 x 16 x 128 bf16
//          0.064 ms; RING 0.072), before one on an fp32 stream (32768 x 2048 0.134; RING 0.141), and before one by single
//          elements, up to 4 to a thread (20000 x 1001 fp32 stream, backward 0.088 ms; NONE 0.135)
//   NONE   a row's pieces when it is its turn, other CTAs covering the wait: more than 4 single elements to a thread, for
//          which there are no registers, and after a block any number (20000 x 1001 forward 0.049 ms, backward 0.089; PAIR
//          0.063, 0.094)
enum class Ahead { NONE, PAIR, RING };

// How a thread gets its pieces of a row of one tensor; zeros where there is nothing.  In a RING a piece of two 16-byte places
// (fp32 beside 16-bit types) is copied by the lanes of the row's part in the order of memory, so that each instruction
// covers whole sectors.
template <typename T, int VEC, int G, int NV, Ahead A> struct Feed {
    static constexpr bool LATE = A == Ahead::NONE && NV * VEC > 8;  // read where it is used: registers would not hold it
    static constexpr int N = A == Ahead::RING ? VEC * (int)sizeof(T) / 16 : 0;  // 16-byte places of a thread
    static constexpr int L = G > 0 ? G : 32;                                    // lanes that copy for each other
    Pack<T, VEC> v[A == Ahead::RING || LATE ? 1 : NV];
    const T *row;
    const Cols<VEC, G, NV> *cols;
    bool live_;
    static __device__ __forceinline__ int place_of(int chunk) {  // (lanes that read two each hit different banks)
        return 16 * (N == 2 ? chunk ^ ((chunk >> 3) & 1) : chunk);
    }
    __device__ __forceinline__ void issue(char *place, const void *p, int64_t at, const Cols<VEC, G, NV> &c, bool live) {
        if constexpr (A == Ahead::RING) {
            const int lane = threadIdx.x % L, first = threadIdx.x - lane, t0 = c.t - lane;  // of the lanes
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int chunk = lane + k * L, col = t0 * VEC + chunk * (16 / (int)sizeof(T));
                const bool on = live && col < c.dim;
                copy16(place + place_of(first * N + chunk), reinterpret_cast<const T *>(p) + (on ? at + col : 0), on);
            }
        } else if constexpr (LATE) {
            row = reinterpret_cast<const T *>(p) + at, cols = &c, live_ = live;
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                v[i] = {};
                if (live && c.on[i]) v[i] = load_pack<T, VEC>(reinterpret_cast<const T *>(p) + at + c.at(i));
            }
        }
    }
    __device__ __forceinline__ void get(const char *place, int i, float (&o)[VEC]) const {
        if constexpr (A == Ahead::RING) {
            Pack<T, VEC> a;
#pragma unroll
            for (int k = 0; k < N; ++k)
                reinterpret_cast<uint4 *>(&a)[k] = *reinterpret_cast<const uint4 *>(place + place_of(threadIdx.x * N + k));
            unpack<T, VEC>(a, o);
        } else if constexpr (LATE) {
            Pack<T, VEC> a = {};
            if (live_ && cols->on[i]) a = load_pack<T, VEC>(row + cols->at(i));
            unpack<T, VEC>(a, o);
        } else {
            unpack<T, VEC>(v[i], o);
        }
    }
};
// (single elements always come in several pieces)
template <int NV> constexpr Ahead ahead_or_none(Ahead a) { return NV > 1 ? Ahead::NONE : a; }
template <int VEC, int NV> constexpr Ahead before_block(Ahead a) {
    return VEC == 1 && NV <= 4 ? Ahead::PAIR : ahead_or_none<NV>(a);
}

// Rows ahead for `places` 16-byte places of a thread and row, of `budget` places (12: 1024 threads of an SM can have them).
constexpr int norm_ahead(int places, int budget = 12) {
    return places == 0 ? 1 : budget / places < 2 ? 2 : budget / places > 6 ? 6 : budget / places;
}

// The weights of a thread's columns, in registers unless it has several pieces, and its column sums, which then lie in
// places of its own in shared memory.
template <int VEC, int G, int NV> struct Weights {
    static constexpr bool KEPT = NV * VEC <= 8;
    const void *p;
    int dt;
    float fill, v[KEPT ? NV : 1][KEPT ? VEC : 1];
    __device__ __forceinline__ Weights(const void *p_, int dt_, const Cols<VEC, G, NV> &c, float fill_) : p(p_), dt(dt_), fill(fill_) {
        if constexpr (KEPT)
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int j = 0; j < VEC; ++j) v[i][j] = p && c.on[i] ? load_scalar(p, c.at(i) + j, dt) : fill;
    }
    __device__ __forceinline__ void get(const Cols<VEC, G, NV> &c, int i, float (&o)[VEC]) const {
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            if constexpr (KEPT) o[j] = v[i][j];
            else o[j] = p && c.on[i] ? load_scalar(p, c.at(i) + j, dt) : fill;
        }
    }
};
template <int VEC, int G, int NV> struct Sums {
    static constexpr bool KEPT = NV * VEC <= 8;
    static constexpr int SHARED = KEPT ? 0 : NV * VEC;  // floats of a thread
    float v[KEPT ? NV : 1][KEPT ? VEC : 1];
    float *s;
    __device__ __forceinline__ explicit Sums(float *shared) : s(shared) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) at(i, j) = 0.f;
    }
    __device__ __forceinline__ float &at(int i, int j) {
        if constexpr (KEPT) return v[i][j];
        return s[(i * VEC + j) * blockDim.x + threadIdx.x];
    }
};

template <typename T, int VEC, int G, int NV>
__device__ __forceinline__ void store_piece(void *p, int64_t at, const Cols<VEC, G, NV> &c, int i, bool live,
                                            const float (&x)[VEC]) {
    if (live && c.on[i]) store_pack<T, VEC>(reinterpret_cast<T *>(p) + at + c.at(i), x);
}

// Where a CTA's column sums go: its (or its cluster's) partial row, or the result itself where it is the only one.
template <int G> struct ColumnSums {
    float *part;
    void *out;
    int dtype;
    __device__ __forceinline__ ColumnSums(float *p, void *o, int dt, int which, int dim)
        : part(p + ((size_t)which * walkers<G>() + walker<G>()) * dim), out(o), dtype(dt) {}
    __device__ __forceinline__ void put(int col, float x) const {
        if (walkers<G>() == 1) store_scalar(out, col, x, dtype);
        else part[col] = x;
    }
};
// The rows' threads are added in order, in `smem` that nothing else uses by then.
template <int VEC, int G, int NV>
__device__ __forceinline__ void write_sums(const ColumnSums<G> &to, float *smem, const Cols<VEC, G, NV> &c, int dim,
                                           Sums<VEC, G, NV> &acc) {
    if constexpr (G <= 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (c.on[i])
#pragma unroll
                for (int j = 0; j < VEC; ++j) to.put(c.at(i) + j, acc.at(i, j));
    } else {
        constexpr int W = G * NV * VEC, RPC = NORM_THREADS / G;  // columns held by a row's threads
        const int gi = threadIdx.x / G;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < VEC; ++j) smem[gi * W + c.at(i) + j] = acc.at(i, j);
        __syncthreads();
        for (int col = threadIdx.x; col < dim; col += NORM_THREADS) {
            float s = 0.f;
            for (int r = 0; r < RPC; ++r) s += smem[r * W + col];
            to.put(col, s);
        }
    }
}

// The rows of a persistent CTA.  In: a row's feeds; issue(in, place, row, live), work(in, place, row, live).
template <class In, Ahead A, int G, int S, int PLACES, class Issue, class Work>
__device__ __forceinline__ void walk_rows(uint32_t rows, char *ring, Issue issue, Work work) {
    const uint32_t step = walkers<G>() * cta_rows<G>();
    // (whole warps stay together: a row's lanes may lie beyond the last row)
    uint32_t base = walker<G>() * cta_rows<G>(), row = base + cta_row<G>();
    if constexpr (A == Ahead::RING) {
        In in;
        const uint32_t bytes = PLACES * 16 * blockDim.x;
#pragma unroll
        for (int k = 0; k < S - 1; ++k) {
            issue(in, ring + k * bytes, row + k * step, row + k * step < rows);
            copies_issued();
        }
        uint32_t slot = 0, ahead = S - 1;
        for (; base < rows; base += step, row += step) {
            __syncwarp();  // every lane has read the row before, whose place is filled now
            issue(in, ring + ahead * bytes, row + (S - 1) * step, row + (S - 1) * step < rows);
            copies_issued();
            copies_wait<S - 1>();
            __syncwarp();
            work(in, ring + slot * bytes, row, row < rows);
            slot = slot + 1 == S ? 0 : slot + 1;
            ahead = ahead + 1 == S ? 0 : ahead + 1;
        }
        copies_wait<0>();
    } else if constexpr (A == Ahead::PAIR) {
        In a, b;  // (two copies of the work, so that no register waits to be moved)
        issue(a, ring, row, row < rows);
        for (; base < rows; base += step, row += step) {
            issue(b, ring, row + step, row + step < rows);
            work(a, ring, row, row < rows);
            if ((base += step) >= rows) break;
            row += step;
            issue(a, ring, row + step, row + step < rows);
            work(b, ring, row, row < rows);
        }
    } else {
        for (; base < rows; base += step, row += step) {
            In in;
            issue(in, ring, row, row < rows);
            work(in, ring, row, row < rows);
        }
    }
}

// What a kernel has of shared memory: the rows ahead (PLACES 16-byte places for each thread and row), in which the column
// sums are added at the end, or the sums themselves.
template <typename T, int VEC, int G, int NV> struct GateFwd {
    static constexpr Ahead A = ahead_or_none<NV>(Ahead::PAIR);
    static constexpr int PLACES = 2 * Feed<T, VEC, G, NV, A>::N, S = norm_ahead(PLACES);
    static constexpr int bytes(int threads) { return S * PLACES * 16 * threads; }
};
template <int VEC, int G, int NV> constexpr int sums_bytes(int sums, int threads) {
    return sums * Sums<VEC, G, NV>::SHARED * 4 * threads + (G > 0 ? 4 * threads * NV * VEC : 0);
}
template <typename T, int VEC, int G, int NV> struct GateBwd {
    static constexpr Ahead A = ahead_or_none<NV>(Ahead::RING);
    static constexpr int PLACES = 3 * Feed<T, VEC, G, NV, A>::N, S = norm_ahead(PLACES);
    static constexpr int bytes(int threads) {
        const int a = S * PLACES * 16 * threads, b = sums_bytes<VEC, G, NV>(1, threads);
        return a > b ? a : b;
    }
};

// ---------------------------------------------------------------- after a block
template <int ACT, typename T, int VEC, int G, int NV, class L>
__device__ __forceinline__ void gated_fwd(const GatedNormParams &p, char *ring) {
    struct In {
        Feed<T, VEC, G, NV, L::A> x, z;
    };
    __shared__ float2 red[GroupSum<G>::PLACES];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(p.dim);
    const Weights<VEC, G, NV> weight(p.weight, p.weight_dtype, c, 1.f);
    const float inv_dim = 1.f / (float)p.dim;
    const int zo = L::PLACES / 2 * 16 * blockDim.x;
    walk_rows<In, L::A, G, L::S, L::PLACES>(
        p.rows, ring,
        [&](In &in, char *at, uint32_t row, bool live) {
            in.x.issue(at, p.x, live ? p.xm.at(row, p.heads) : 0, c, live);
            if (ACT != ACT_NONE) in.z.issue(at + zo, p.z, live ? p.zm.at(row, p.heads) : 0, c, live);
        },
        [&](const In &in, const char *at, uint32_t row, bool live) {
            float x[NV][VEC], s1 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                in.x.get(at, i, x[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) s1 = fmaf(x[i][j], x[i][j], s1);
            }
            const float rs = rsqrtf(sum.template operator()<false>(s1, 0.f).x * inv_dim + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float y[VEC], z[VEC], w[VEC];
                weight.get(c, i, w);
                if (ACT != ACT_NONE) in.z.get(at + zo, i, z);
                if constexpr (VEC > 1) {  // two values to an instruction
#pragma unroll
                    for (int j = 0; j < VEC; j += 2) {
                        F2 v = mul2(mul2(F2(x[i][j], x[i][j + 1]), F2(rs)), F2(w[j], w[j + 1]));
                        if (ACT != ACT_NONE) v = mul2(v, F2(sigmoid_t<T>(z[j]), sigmoid_t<T>(z[j + 1])));
                        if (ACT == 0) v = mul2(v, F2(z[j], z[j + 1]));
                        v.get(y[j], y[j + 1]);
                    }
                } else {
                    y[0] = x[i][0] * rs * w[0];
                    if (ACT != ACT_NONE) y[0] *= sigmoid_t<T>(z[0]);
                    if (ACT == 0) y[0] *= z[0];
                }
                store_piece<T>(p.y, (int64_t)row * p.dim, c, i, live, y);
            }
        });
}

template <int ACT, typename T, int VEC, int G, int NV, class L>
__device__ __forceinline__ void gated_bwd(const GatedNormParams &p, char *ring, float *shared) {
    struct In {
        Feed<T, VEC, G, NV, L::A> x, dy, z;
    };
    __shared__ float2 red[GroupSum<G>::PLACES];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(p.dim);
    const Weights<VEC, G, NV> weight(p.weight, p.weight_dtype, c, 1.f);
    Sums<VEC, G, NV> dw(shared);
    const float inv_dim = 1.f / (float)p.dim;
    const int one = L::PLACES / 3 * 16 * blockDim.x;
    walk_rows<In, L::A, G, L::S, L::PLACES>(
        p.rows, ring,
        [&](In &in, char *at, uint32_t row, bool live) {
            in.x.issue(at, p.x, live ? p.xm.at(row, p.heads) : 0, c, live);
            in.dy.issue(at + one, p.dy, live ? p.dym.at(row, p.heads) : 0, c, live);
            if (ACT != ACT_NONE) in.z.issue(at + 2 * one, p.z, live ? p.zm.at(row, p.heads) : 0, c, live);
        },
        [&](const In &in, const char *at, uint32_t row, bool live) {
            float x[NV][VEC], up[NV][VEC], dz[NV][VEC], s1 = 0.f, s2 = 0.f;  // up = dy act(z), dz = dy act'(z)
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float w[VEC];
                weight.get(c, i, w);
                in.x.get(at, i, x[i]);
                in.dy.get(at + one, i, up[i]);
                if (ACT != ACT_NONE) in.z.get(at + 2 * one, i, dz[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    if (ACT != ACT_NONE) {
                        const float z = dz[i][j], d = up[i][j], sg = sigmoid_t<T>(z), rest = fmaf(-sg, sg, sg);
                        up[i][j] = d * (ACT == 0 ? z * sg : sg);
                        dz[i][j] = d * (ACT == 0 ? fmaf(z, rest, sg) : rest);
                    }
                    s1 = fmaf(x[i][j], x[i][j], s1);
                    s2 = fmaf(up[i][j] * w[j], x[i][j], s2);
                }
            }
            const float2 s = sum(s1, s2);
            // A row past the end is zeros and adds nothing to the column sums, also where eps is 0.  (1 there rather than rs set
            // to 0, which is a branch around the root: 403795 x 34 on an fp32 stream 0.188 ms, so 0.162.)
            const float rs = rsqrtf(s.x * inv_dim + (G <= 0 || live ? p.eps : 1.f));
            const NormGrad q(rs, s.y * inv_dim, p.dim, p.eps);
            const int64_t o = (int64_t)row * p.dim;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float dx[VEC], w[VEC];
                weight.get(c, i, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    const float xr = x[i][j] * rs;
                    dx[j] = q(up[i][j] * w[j], x[i][j]);
                    if (ACT != ACT_NONE) dz[i][j] *= xr * w[j];
                    dw.at(i, j) = fmaf(up[i][j], xr, dw.at(i, j));
                }
                store_piece<T>(p.dx, o, c, i, live, dx);
                if (ACT != ACT_NONE) store_piece<T>(p.dz, o, c, i, live, dz[i]);
            }
        });
    if (p.dweight) write_sums<VEC, G, NV>({p.part, p.dweight, p.weight_dtype, 0, p.dim}, shared, c, p.dim, dw);
}

template <typename T, int VEC, int G, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k9_gated_fwd(const __grid_constant__ GatedNormParams p) {
    extern __shared__ __align__(16) char norm_smem[];
    using L = GateFwd<T, VEC, G, NV>;
    if (!p.z) gated_fwd<ACT_NONE, T, VEC, G, NV, L>(p, norm_smem);
    else if (p.act == 0) gated_fwd<0, T, VEC, G, NV, L>(p, norm_smem);
    else gated_fwd<1, T, VEC, G, NV, L>(p, norm_smem);
}
template <typename T, int VEC, int G, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k9_gated_bwd(const __grid_constant__ GatedNormParams p) {
    extern __shared__ __align__(16) char norm_smem[];
    using L = GateBwd<T, VEC, G, NV>;
    float *shared = reinterpret_cast<float *>(norm_smem);
    if (!p.z) gated_bwd<ACT_NONE, T, VEC, G, NV, L>(p, norm_smem, shared);
    else if (p.act == 0) gated_bwd<0, T, VEC, G, NV, L>(p, norm_smem, shared);
    else gated_bwd<1, T, VEC, G, NV, L>(p, norm_smem, shared);
}

// ---------------------------------------------------------------- before a block
template <typename T, typename R, int VEC, int G, int NV> struct AddFwd {
    static constexpr Ahead A = before_block<VEC, NV>(sizeof(R) == 4 ? Ahead::PAIR : Ahead::RING);
    static constexpr int PLACES = 1 * Feed<T, VEC, G, NV, A>::N + 1 * Feed<R, VEC, G, NV, A>::N, S = norm_ahead(PLACES, 6);
    static constexpr int bytes(int threads) { return S * PLACES * 16 * threads; }
};
template <typename T, typename R, int VEC, int G, int NV> struct AddBwd {
    static constexpr Ahead A = before_block<VEC, NV>(Ahead::RING);
    static constexpr int PLACES = 2 * Feed<T, VEC, G, NV, A>::N + 2 * Feed<R, VEC, G, NV, A>::N, S = norm_ahead(PLACES);
    static constexpr int bytes(int threads) {
        const int a = S * PLACES * 16 * threads, b = sums_bytes<VEC, G, NV>(2, threads);
        return a > b ? a : b;
    }
};

template <typename T, typename R, int VEC, int G, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k9_add_fwd(const __grid_constant__ AddNormParams p) {
    using L = AddFwd<T, R, VEC, G, NV>;
    using X = Feed<T, VEC, G, NV, L::A>;
    struct In {
        X x;
        Feed<R, VEC, G, NV, L::A> r;
    };
    extern __shared__ __align__(16) char norm_smem[];
    __shared__ float2 red[GroupSum<G>::PLACES];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(p.dim);
    const Weights<VEC, G, NV> weight(p.weight, p.weight_dtype, c, 1.f), scale(p.scale_vec, p.scale_dtype, c, p.scale);
    const float inv_dim = 1.f / (float)p.dim;
    const int ro = X::N * 16 * blockDim.x;
    walk_rows<In, L::A, G, L::S, L::PLACES>(
        p.rows, norm_smem,
        [&](In &in, char *at, uint32_t row, bool live) {
            in.x.issue(at, p.x, (int64_t)row * p.x_ts, c, live);
            in.r.issue(at + ro, p.residual, (int64_t)row * p.r_ts, c, live && p.residual);
        },
        [&](const In &in, const char *at, uint32_t row, bool live) {
            float r[NV][VEC], s1 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[VEC], sc[VEC];
                scale.get(c, i, sc);
                in.x.get(at, i, x);
                in.r.get(at + ro, i, r[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    r[i][j] = fmaf(sc[j], x[j], r[i][j]);
                    s1 = fmaf(r[i][j], r[i][j], s1);
                }
            }
            if (p.residual_out)
#pragma unroll
                for (int i = 0; i < NV; ++i) store_piece<R>(p.residual_out, (int64_t)row * p.ro_ts, c, i, live, r[i]);
            const float rs = rsqrtf(sum.template operator()<false>(s1, 0.f).x * inv_dim + p.eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float y[VEC], w[VEC];
                weight.get(c, i, w);
#pragma unroll
                for (int j = 0; j < VEC; ++j) y[j] = r[i][j] * rs * w[j];
                store_piece<T>(p.y, (int64_t)row * p.dim, c, i, live, y);
            }
        });
}

template <typename T, typename R, int VEC, int G, int NV, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) k9_add_bwd(const __grid_constant__ AddNormParams p) {
    using L = AddBwd<T, R, VEC, G, NV>;
    using X = Feed<T, VEC, G, NV, L::A>;
    using Res = Feed<R, VEC, G, NV, L::A>;
    struct In {
        X dy, x;
        Res r, dres;
    };
    extern __shared__ __align__(16) char norm_smem[];
    float *shared = reinterpret_cast<float *>(norm_smem);
    __shared__ float2 red[GroupSum<G>::PLACES];
    GroupSum<G> sum(red);
    const Cols<VEC, G, NV> c(p.dim);
    const Weights<VEC, G, NV> weight(p.weight, p.weight_dtype, c, 1.f), scale(p.scale_vec, p.scale_dtype, c, p.scale);
    Sums<VEC, G, NV> dw(shared), ds(shared + Sums<VEC, G, NV>::SHARED * blockDim.x);
    const float inv_dim = 1.f / (float)p.dim;
    const int xo = X::N * 16 * blockDim.x, ro = 2 * xo, so = ro + Res::N * 16 * blockDim.x;
    walk_rows<In, L::A, G, L::S, L::PLACES>(
        p.rows, norm_smem,
        [&](In &in, char *at, uint32_t row, bool live) {
            in.dy.issue(at, p.dy, (int64_t)row * p.dy_ts, c, live);
            in.r.issue(at + ro, p.residual_out, (int64_t)row * p.ro_ts, c, live);
            in.dres.issue(at + so, p.dres, (int64_t)row * p.dres_ts, c, live && p.dres);
            in.x.issue(at + xo, p.x, (int64_t)row * p.x_ts, c, live && p.dscale);
        },
        [&](const In &in, const char *at, uint32_t row, bool live) {
            float r[NV][VEC], up[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float w[VEC];
                weight.get(c, i, w);
                in.dy.get(at, i, up[i]);
                in.r.get(at + ro, i, r[i]);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    s1 = fmaf(r[i][j], r[i][j], s1);
                    s2 = fmaf(up[i][j] * w[j], r[i][j], s2);
                }
            }
            const float2 s = sum(s1, s2);
            const float rs = rsqrtf(s.x * inv_dim + (G <= 0 || live ? p.eps : 1.f));  // (as after a block)
            const NormGrad q(rs, s.y * inv_dim, p.dim, p.eps);
            const int64_t o = (int64_t)row * p.dim;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float d[VEC], x[VEC], w[VEC], sc[VEC];
                weight.get(c, i, w);
                scale.get(c, i, sc);
                in.dres.get(at + so, i, d);
                in.x.get(at + xo, i, x);
#pragma unroll
                for (int j = 0; j < VEC; ++j) {
                    d[j] += q(up[i][j] * w[j], r[i][j]);
                    dw.at(i, j) = fmaf(up[i][j], r[i][j] * rs, dw.at(i, j));
                    ds.at(i, j) = fmaf(d[j], x[j], ds.at(i, j));
                }
                if (p.dresidual) store_piece<R>(p.dresidual, o, c, i, live, d);
                if (p.dx) {
#pragma unroll
                    for (int j = 0; j < VEC; ++j) x[j] = sc[j] * d[j];
                    store_piece<T>(p.dx, o, c, i, live, x);
                }
            }
        });
    if (p.dweight) write_sums<VEC, G, NV>({p.part, p.dweight, p.weight_dtype, 0, p.dim}, shared, c, p.dim, dw);
    if (p.dscale) write_sums<VEC, G, NV>({p.part, p.dscale, p.scale_dtype, p.dweight ? 1 : 0, p.dim}, shared, c, p.dim, ds);
}

// ---------------------------------------------------------------- choice of the row's threads
// CALL(VEC, G, NV, most threads, threads) with `ctas` CTAs to a row: one piece to a thread up to 8 x 512 threads, in whole
// warps; single elements, several to a thread.
#define NORM_DISPATCH(T, vec, dim, CALL)                                                      \
    do {                                                                                      \
        int ctas = 1;                                                                         \
        if (vec) {                                                                            \
            constexpr int VE = 16 / (int)sizeof(T);                                           \
            const int n = (dim) / VE, up = (n + 31) / 32 * 32;                                \
            if (n <= 8) { CALL(VE, 8, 1, NORM_THREADS, NORM_THREADS); }                       \
            else if (n <= 16) { CALL(VE, 16, 1, NORM_THREADS, NORM_THREADS); }                \
            else if (n <= 32) { CALL(VE, 32, 1, NORM_THREADS, NORM_THREADS); }                \
            else if (n <= 256) { CALL(VE, WHOLE, 1, 256, up); }                               \
            else if (n <= 512) { CALL(VE, WHOLE, 1, 512, up); }                               \
            else if (n <= 1024) { CALL(VE, WHOLE, 1, 1024, up); }                             \
            else {                                                                            \
                ctas = (n + 511) / 512;                                                       \
                const int per = ((n + ctas - 1) / ctas + 31) / 32 * 32;                       \
                CALL(VE, SPREAD, 1, 512, per);                                                \
            }                                                                                 \
        } else {                                                                              \
            const int up = ((dim) + 63) / 64 * 32;                                            \
            if ((dim) <= 128) { CALL(1, 32, 4, NORM_THREADS, NORM_THREADS); }                 \
            else if ((dim) <= 512) { CALL(1, WHOLE, 2, 256, up); }                                \
            else if ((dim) <= 1024) { CALL(1, WHOLE, 2, 512, up); }                               \
            else if ((dim) <= 2048) { CALL(1, WHOLE, 2, 1024, up); }                              \
            else if ((dim) <= 4096) { CALL(1, WHOLE, 4, 1024, 1024); }                            \
            else { CALL(1, WHOLE, 16, 1024, 1024); }                                              \
        }                                                                                     \
    } while (0)

// CTAs of a backward that sums columns, at most.  Few rows take one, which writes the sums itself: a row in turn costs it about
// 1 us, a second launch 2 us on the device and 8 us on the host where the device waits for it.
inline int sum_ctas(int64_t rows, int rows_per_cta, int dim) { return rows <= 4 * rows_per_cta ? 1 : norm_parts(rows, dim); }

// Launches the persistent grid of a kernel; L says what shared memory it takes; grid: its number of CTAs (of clusters where
// several CTAs share a row), at most `most`.
template <class L, class P>
cudaError_t norm_launch(void (*kernel)(P), const P &p, int threads, int max_threads, int ctas, int rows_per_cta, int most,
                        int &grid, cudaStream_t stream) {
    const int smem = L::bytes(threads);
    cudaError_t e =
        norm_grid((const void *)kernel, threads, ctas, smem, L::bytes(max_threads), p.rows, rows_per_cta, most, grid);
    if (e != cudaSuccess) return e;
    if (ctas == 1) {
        kernel<<<grid, threads, smem, stream>>>(p);
        return cudaGetLastError();
    }
    ClusterLaunch l(grid * ctas, threads, smem, ctas, stream);
    return cudaLaunchKernelEx(&l.cfg, kernel, p);
}

}  // namespace

cudaError_t launch_colsum(const float *part, int parts, int dim, int sums, void *out0, int dtype0, void *out1, int dtype1,
                          cudaStream_t stream);

// CTAs of an SM that a kernel is compiled for, of `threads` threads at most: 1024 threads in all; 2048 for the forward before a
// block, which needs few registers (48763 x 4096 bf16 0.276 -> 0.258 ms); 512 for the backward before a block with longer
// rows in one CTA, whose column sums take them.
constexpr int add_fwd_ctas(int residual_size, int vec, int threads) {
    return (residual_size == 4 || vec == 1 ? 1024 : 2048) / threads;
}
constexpr int add_bwd_ctas(int vec, int g, int threads) {
    return threads <= 256 || vec == 1 || g == SPREAD ? 1024 / threads : 1;
}
#define NORM_ROWS(G) ((G) > 0 ? NORM_THREADS / ((G) > 0 ? (G) : 1) : 1)
template <typename T> cudaError_t gated_norm_fwd_t(const GatedNormParams &p, cudaStream_t stream) {
    int grid = 0;
#define CALL(V, G, NV, MAXT, threads)                                                                                  \
    return norm_launch<GateFwd<T, V, G, NV>>(k9_gated_fwd<T, V, G, NV, MAXT, 1024 / MAXT>, p, threads, MAXT, ctas, NORM_ROWS(G), \
                    1 << 30, grid, stream)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
}

template <typename T> cudaError_t gated_norm_bwd_t(const GatedNormParams &p, cudaStream_t stream) {
    int grid = 0;
    cudaError_t e = cudaSuccess;
#define CALL(V, G, NV, MAXT, threads)                                                                                  \
    e = norm_launch<GateBwd<T, V, G, NV>>(k9_gated_bwd<T, V, G, NV, MAXT, 1024 / MAXT>, p, threads, MAXT, ctas, NORM_ROWS(G), \
                    sum_ctas(p.rows, NORM_ROWS(G), p.dim), grid, stream)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
    if (e != cudaSuccess || !p.dweight || grid == 1) return e;
    return launch_colsum(p.part, grid, p.dim, 1, p.dweight, p.weight_dtype, nullptr, 0, stream);
}

template <typename T, typename R> cudaError_t add_norm_fwd_t(const AddNormParams &p, cudaStream_t stream) {
    int grid = 0;
#define CALL(V, G, NV, MAXT, threads)                                                                                  \
    return norm_launch<AddFwd<T, R, V, G, NV>>(k9_add_fwd<T, R, V, G, NV, MAXT, add_fwd_ctas(sizeof(R), V, MAXT)>, p, threads, MAXT, ctas, NORM_ROWS(G), \
                    1 << 30, grid, stream)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
}

template <typename T, typename R> cudaError_t add_norm_bwd_t(const AddNormParams &p, cudaStream_t stream) {
    int grid = 0;
    cudaError_t e = cudaSuccess;
#define CALL(V, G, NV, MAXT, threads)                                                                                  \
    e = norm_launch<AddBwd<T, R, V, G, NV>>(k9_add_bwd<T, R, V, G, NV, MAXT, add_bwd_ctas(V, G, MAXT)>, p, threads, MAXT, ctas, NORM_ROWS(G), \
                    sum_ctas(p.rows, NORM_ROWS(G), p.dim), grid, stream)
    NORM_DISPATCH(T, p.vec, p.dim, CALL);
#undef CALL
    const int sums = (p.dweight ? 1 : 0) + (p.dscale ? 1 : 0);
    if (e != cudaSuccess || !sums || grid == 1) return e;
    if (!p.dweight) return launch_colsum(p.part, grid, p.dim, 1, p.dscale, p.scale_dtype, nullptr, 0, stream);
    return launch_colsum(p.part, grid, p.dim, sums, p.dweight, p.weight_dtype, p.dscale, p.scale_dtype, stream);
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
