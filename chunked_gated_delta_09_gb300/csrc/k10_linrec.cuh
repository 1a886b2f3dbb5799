// k10_linrec.cuh -- the gated linear recurrence, forward and backward (included once per activation type):
//
//   h_t = a_t h_{t-1} + b_t ,  a = exp(g) ,  b = x or (1 - a) x          per channel, packed or dense sequences
//   m_t = a_t (dh_t + m_{t+1}) ;  dx_t = dh_t + m_{t+1} (times 1 - a_t) ;  dg_t = m_t (h_{t-1} - x_t or 0)
//
// Both directions are scans of maps s -> A s + B, which compose as (A2 A1, A2 B1 + B2).  The rows are cut into tiles,
// whatever the sequences: where a sequence starts (or, backwards, ends) inside a tile, the row's map forgets what
// came before it (a flag rather than A = 0, so that a nan does not pass from one sequence to the next).
//
// A cluster of CTAs owns a block of 32 channels and goes through all rows, a tile for each CTA at a time.  A warp
// composes 16 rows of its CTA's tile (two groups of 8, 16 lanes with two channels each) and keeps a and b in registers;
// the warps' maps are composed in shared memory, and the CTA's map is sent to every CTA of the cluster, which then
// knows the state that enters its own tile and finishes its rows.  So every value is read once and written once, nothing
// is exchanged through memory, and the order of all sums is fixed: results are bit-identical from run to run.  The next
// tiles arrive by tensor-map loads meanwhile.  The forward saves the state that enters each LR_TILE rows, from which the
// backward recomputes h instead of reading it back rounded.
#pragma once

#include "block_common.cuh"
#include "tc_util.cuh"

namespace gdr {
namespace {

using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;

constexpr int LR_WROWS = 16;      // rows of a warp: two groups of 8
constexpr int LR_FWD_WARPS = 16;  // 256 rows
constexpr int LR_BWD_WARPS = LR_TILE / LR_WROWS;
constexpr int LR_FWD_STAGES = 2, LR_BWD_STAGES = 3;

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
__device__ __forceinline__ F2 shfl2(F2 a, int lane) {
    float x, y;
    a.get(x, y);
    return F2(__shfl_sync(0xffffffffu, x, lane), __shfl_sync(0xffffffffu, y, lane));
}

// exp(g) and 1 - exp(g), both to about one unit in the last place and without a lean to one side, which a channel that
// remembers hundreds of tokens would add up (decays near 1 that come out a quarter of a unit too low put h off by
// 1e-5).  Cody and Waite's reduction g = n ln 2 + r, then exp(r) - 1 = r + r^2 q(r) with q a Chebyshev fit of degree 4
// (1e-8 off), so that 1 - a is exact to rounding near a = 1.  Below -87.7 a is 0; above 88.3 it is taken at 88.3.
__device__ __forceinline__ void decay2(float g0, float g1, F2 &a, F2 &rest) {
    const float lo = -88.f, hi = 88.3f;
    asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+f"(g0) : "f"(hi), "f"(lo));
    asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+f"(g1) : "f"(hi), "f"(lo));
    const F2 g(g0, g1), shift(12582912.f), one(1.f);  // 1.5 x 2^23: the sum's low bits are the rounded integer
    const F2 t = fma2(g, F2(1.44269504f), shift), n = add2(t, F2(-12582912.f));
    const F2 r = fma2(n, F2(-0.693147181f), g);  // (ln 2 is 1.9e-9 off: n times that, below a rounding of a until a < 1e-9)
    F2 q = fma2(r, F2(0.0013933823f), F2(0.0083632953f));
    q = fma2(q, r, F2(0.041666463f));
    q = fma2(q, r, F2(0.16666576f));
    q = fma2(q, r, F2(0.5f));
    const F2 p = fma2(mul2(r, r), q, r);
    float t0, t1;
    t.get(t0, t1);
    const F2 s(__int_as_float((__float_as_int(t0) << 23) + 0x3f800000),
               __int_as_float((__float_as_int(t1) << 23) + 0x3f800000));  // 2^n
    a = fma2(p, s, s);
    const F2 ns = mul2(s, F2(-1.f));
    rest = fma2(p, ns, add2(one, ns));
}

// ---------------------------------------------------------------- maps
// The map s -> a s + b, or b where what came before is cut off.
struct Map {
    float a = 1.f, b = 0.f;
    bool cut = false;
    __device__ __forceinline__ void then(float a2, float b2, bool cut2) {
        b = cut2 ? b2 : fmaf(a2, b, b2);
        a *= a2;
        cut |= cut2;
    }
    __device__ __forceinline__ float of(float s) const { return cut ? b : fmaf(a, s, b); }
};

__device__ __forceinline__ int cluster_rank() {
    int r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The address in the CTA `rank` of a variable of this one.
__device__ __forceinline__ uint32_t in_cta(const void *p, int rank) {
    uint32_t a;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}

// Waits for a phase; one that takes longer than the limit is reported, and awaited further all the same, so that nothing
// arrives after the CTA has moved on.
__device__ __forceinline__ void wait_phase(uint64_t *bar, uint32_t parity, const LinrecParams &p) {
    if (!mbar_wait(bar, parity, p.spin)) {
        atomicOr(p.status, ST_TIMEOUT);
        mbar_wait(bar, parity, DRAIN_LIMIT);
    }
}

// The same for a phase that other CTAs of the cluster complete: what they wrote is visible afterwards.
__device__ __forceinline__ void wait_peers(uint64_t *bar, uint32_t parity, const LinrecParams &p) {
    uint32_t done = 0;
    for (uint64_t polls = 0; polls < (uint64_t)p.spin + DRAIN_LIMIT; ++polls) {
        asm volatile(
            "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(smem_u32(bar)), "r"(parity)
            : "memory");
        if (done) break;
        if (polls == p.spin) atomicOr(p.status, ST_TIMEOUT);
    }
}

// What the CTAs of a cluster tell each other: the maps of their tiles, by stores that count themselves on the receiver's
// barrier.  Two buffers in turn: a CTA sends its map of the tile after next only after it has that of the next from
// everybody, and nobody sends that before having done with this one.
struct Peers {
    float2 map[2][LR_MAX_CLUSTER][LR_CH];
    int cut[2][LR_MAX_CLUSTER];
    uint64_t bar[2];
    // one warp, a lane for each channel
    __device__ __forceinline__ void tell(int buf, int rank, int size, const Map &m) {
        const int lane = threadIdx.x & 31;
        if (lane == 0) mbar_expect_tx(&bar[buf], (uint32_t)size * (LR_CH * 8 + 4));
        uint64_t v;
        asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(m.a), "f"(m.b));
        for (int q = 0; q < size; ++q) {
            const uint32_t b = in_cta(&bar[buf], q);
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                             in_cta(&map[buf][rank][lane], q)),
                         "l"(v), "r"(b)
                         : "memory");
            if (lane == 0)
                asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                                 in_cta(&cut[buf][rank], q)),
                             "r"((int)m.cut), "r"(b)
                             : "memory");
        }
    }
    // the state s taken through all tiles of the cluster, for a lane's channel
    __device__ __forceinline__ float through(int buf, int size, float s) const {
        for (int q = 0; q < size; ++q) {
            const float2 v = map[buf][q][threadIdx.x & 31];
            s = cut[buf][q] ? v.y : fmaf(v.x, s, v.y);
        }
        return s;
    }
    // the states s taken through the tiles before that of CTA `rank`, for two channels
    __device__ __forceinline__ F2 entry(int buf, int rank, int ch, F2 s) const {
        for (int q = 0; q < rank; ++q) {
            const float4 v = *reinterpret_cast<const float4 *>(&map[buf][q][ch]);
            s = cut[buf][q] ? F2(v.y, v.w) : fma2(F2(v.x, v.z), s, F2(v.y, v.w));
        }
        return s;
    }
};

// ---------------------------------------------------------------- a tile's rows
// First and last rows of sequences among a tile's ROWS rows, and the rows' sequences.
template <int ROWS> struct Sequences {
    uint32_t head[ROWS / 32], tail[ROWS / 32];
    int seq[ROWS];
    // the last sequence that starts at or before the row
    static __device__ __forceinline__ int of_row(const LinrecParams &p, int row) {
        if (!p.cu) return p.per_seq.div(row);
        int lo = 0, hi = p.N;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (p.cu[mid] <= row) lo = mid;
            else hi = mid;
        }
        return lo;
    }
    // by one warp
    __device__ __forceinline__ void find(const LinrecParams &p, int tile) {
        const int lane = threadIdx.x & 31, row0 = tile * ROWS, end = min(row0 + ROWS, p.rows);
        bool none = row0 >= p.rows;
        if (!none) {
            const int s = of_row(p, row0), a = p.cu ? p.cu[s] : s * p.tokens, b = p.cu ? p.cu[s + 1] : a + p.tokens;
            none = a < row0 && b > end;  // the tile lies within one sequence
        }
        for (int k = 0; k < ROWS / 32; ++k) {
            bool h = false, e = false;
            if (!none) {
                const int row = row0 + 32 * k + lane;
                if (row < p.rows) {
                    const int s = of_row(p, row), a = p.cu ? p.cu[s] : s * p.tokens, b = p.cu ? p.cu[s + 1] : a + p.tokens;
                    h = a == row;
                    e = b == row + 1;
                    seq[32 * k + lane] = s;
                }
            }
            const uint32_t hb = __ballot_sync(0xffffffffu, h), eb = __ballot_sync(0xffffffffu, e);
            if (lane == 0) head[k] = hb, tail[k] = eb;
        }
    }
    // of a warp's 16 rows
    __device__ __forceinline__ uint32_t heads(int w) const { return head[w >> 1] >> (16 * (w & 1)) & 0xffff; }
    __device__ __forceinline__ uint32_t tails(int w) const { return tail[w >> 1] >> (16 * (w & 1)) & 0xffff; }
};

// A tile of one tensor in shared memory: ROWS rows of 32 channels.
template <typename T, int ROWS> struct Tile {
    T v[ROWS][LR_CH];
    __device__ __forceinline__ void get(int r, int ch, float &x, float &y) const {
        const Pack<T, 2> q = *reinterpret_cast<const Pack<T, 2> *>(&v[r][ch]);
        x = to_f32(q.v[0]);
        y = to_f32(q.v[1]);
    }
    __device__ __forceinline__ F2 get(int r, int ch) const {
        float x, y;
        get(r, ch, x, y);
        return F2(x, y);
    }
    // where the rows cannot be moved by a tensor map: a warp brings its own 16 rows, w of them
    __device__ __forceinline__ void bring(const void *src, int64_t ts, int tile, int w, int cb, const LinrecParams &p) {
        const int lane = threadIdx.x & 31, c = cb * LR_CH + lane;
#pragma unroll 4
        for (int r = w * LR_WROWS; r < (w + 1) * LR_WROWS; ++r) {
            const int row = tile * ROWS + r;
            T x = to_out_t<T>(0.f);
            if (row < p.rows && c < p.dim) x = reinterpret_cast<const T *>(src)[(int64_t)row * ts + c];
            v[r][lane] = x;
        }
    }
};
__device__ __forceinline__ void load_tile(void *dst, const CUtensorMap *map, int c, int row, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c), "r"(row), "r"(smem_u32(bar))
        : "memory");
}

template <bool V> struct Const {
    static constexpr bool value = V;
};

// Two neighbouring values of a row; VEC: they lie in one aligned piece.
template <bool VEC, typename T>
__device__ __forceinline__ void put2(T *p, int64_t at, F2 v, int c, int dim) {
    float x, y;
    v.get(x, y);
    if (VEC) {
        const float o[2] = {x, y};
        if (c < dim) store_pack<T, 2>(p + at, o);
    } else {
        if (c < dim) p[at] = to_out_t<T>(x);
        if (c + 1 < dim) p[at + 1] = to_out_t<T>(y);
    }
}
__device__ __forceinline__ F2 get2(const float *p, int64_t at, int c, int dim) {
    return F2(p && c < dim ? p[at] : 0.f, p && c + 1 < dim ? p[at + 1] : 0.f);
}

// Sequences without a token have no row: their last state is their first (forward), their gradients pass through
// (backward).  The tiles share them out; by one warp.
__device__ __forceinline__ void empty_sequences(const LinrecParams &p, int64_t tile, int cb, const float *from, float *to) {
    if ((!p.cu && p.tokens > 0) || !to || tile >= p.tiles) return;
    const int64_t lo = p.N * tile / p.tiles, hi = p.N * (tile + 1) / p.tiles;
    const int c = cb * LR_CH + (threadIdx.x & 31);
    for (int64_t s = lo; s < hi; ++s)
        if (c < p.dim && (!p.cu || p.cu[s] == p.cu[s + 1])) to[s * p.dim + c] = from ? from[s * p.dim + c] : 0.f;
}

// cu_seqlens that do not rise from 0 to the number of rows are reported; the grid shares the check.
__device__ __forceinline__ void check_sequences(const LinrecParams &p) {
    const int t = blockIdx.x * blockDim.x + threadIdx.x;
    if (p.clear && t == 0) *p.status = 0;
    if (!p.cu) return;
    bool bad = t == 0 && (p.cu[0] != 0 || p.cu[p.N] != p.rows);
    for (int s = t; s < p.N; s += gridDim.x * blockDim.x) bad |= p.cu[s + 1] < p.cu[s];
    if (bad) atomicOr(p.status, ST_BAD_SEQLENS);
}

// a group's map (channels ch, ch + 1) as the scan's records lie in shared memory
__device__ __forceinline__ void put_maps(float2 *at, F2 a, F2 b) {
    float x, y, u, v;
    a.get(x, y);
    b.get(u, v);
    *reinterpret_cast<float4 *>(at) = make_float4(x, u, y, v);
}

// ---------------------------------------------------------------- forward
template <typename T, typename G> struct FwdStage {
    static constexpr int ROWS = LR_FWD_WARPS * LR_WROWS;
    Tile<G, ROWS> g;
    Tile<T, ROWS> x;
};

template <typename T, typename G, bool COMP, bool VEC>
__global__ void __launch_bounds__(32 * LR_FWD_WARPS, 2)
    k10_fwd(const __grid_constant__ LinrecParams p, const __grid_constant__ LinrecMaps maps) {
    using Stage = FwdStage<T, G>;
    constexpr int W = LR_FWD_WARPS, ROWS = Stage::ROWS, S = LR_FWD_STAGES;
    extern __shared__ __align__(128) char dynamic[];
    Stage *stages = reinterpret_cast<Stage *>(dynamic);
    __shared__ Sequences<ROWS> seqs[2];
    __shared__ __align__(16) float2 agg[W][LR_CH];  // a warp's map, then that of the tile's rows before it
    __shared__ __align__(16) Peers peers;
    __shared__ __align__(8) uint64_t full[S];
    __shared__ uint32_t pcut;  // bit per warp: there is a cut in the tile's rows before it
    __shared__ float carry[LR_CH];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = lane >> 4, ch = 2 * (lane & 15);
    const int rank = cluster_rank(), cb = blockIdx.x / p.cluster, c = cb * LR_CH + ch;

    auto fetch = [&](int k) {  // VEC: one thread; else every warp
        Stage &st = stages[k % S];
        const int tile = k * p.cluster + rank;
        if (VEC) {
            mbar_expect_tx(&full[k % S], sizeof(Stage));
            load_tile(&st.g, &maps.g, cb * LR_CH, tile * ROWS, &full[k % S]);
            load_tile(&st.x, &maps.x, cb * LR_CH, tile * ROWS, &full[k % S]);
        } else {
            st.g.bring(p.g, p.g_ts, tile, wid, cb, p);
            st.x.bring(p.x, p.x_ts, tile, wid, cb, p);
            __syncwarp();
        }
    };
    if (threadIdx.x == 0) {
        for (int q = 0; q < S; ++q) mbar_init(&full[q], 1);
        mbar_init(&peers.bar[0], 1);
        mbar_init(&peers.bar[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    check_sequences(p);
    if (wid == 2) seqs[0].find(p, rank);
    cluster_sync();  // the barriers are there, everywhere
    for (int k = 0; k < S && k < p.supers; ++k)
        if (!VEC || threadIdx.x == 0) fetch(k);
    float walked = 0.f;  // (warp 1) the state that enters the cluster's rows
    for (int k = 0; k < p.supers; ++k) {
        const int buf = k & 1, tile = k * p.cluster + rank, first = wid * LR_WROWS + 8 * group, row0 = tile * ROWS + first;
        const Sequences<ROWS> &sq = seqs[buf];
        const Stage &st = stages[k % S];
        const uint32_t wheads = sq.heads(wid), heads = wheads >> (8 * group) & 0xff;
        const uint32_t wtails = sq.tails(wid), tails = wtails >> (8 * group) & 0xff;
        // most warps: every row and channel is there, and no sequence starts or ends among the rows
        const bool plain = VEC && !(wheads | wtails) && tile * ROWS + (wid + 1) * LR_WROWS <= p.rows &&
                           (cb + 1) * LR_CH <= p.dim;
        if (VEC) wait_phase(&full[k % S], (k / S) & 1, p);
        F2 a[8], b[8], A, B;
        auto compose = [&](auto any) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float g0, g1;
                st.g.get(first + r, ch, g0, g1);
                F2 rest;
                decay2(g0, g1, a[r], rest);
                b[r] = st.x.get(first + r, ch);
                if (COMP) b[r] = mul2(b[r], rest);
                if (any.value && (heads >> r) & 1) {
                    b[r] = fma2(a[r], get2(p.h0, (int64_t)sq.seq[first + r] * p.dim + c, c, p.dim), b[r]);
                    B = b[r];
                } else {
                    B = r == 0 ? b[r] : fma2(a[r], B, b[r]);
                }
                A = r == 0 ? a[r] : mul2(A, a[r]);
            }
        };
        if (plain) compose(Const<false>());
        else compose(Const<true>());
        // the first group's map for the lanes of the second, and the warp's map
        const F2 A0 = shfl2(A, lane & 15), B0 = shfl2(B, lane & 15);
        if (group) put_maps(&agg[wid][ch], mul2(A, A0), heads ? B : fma2(A, B0, B));
        __syncthreads();
        // the tile's rows are in registers: their place takes the tile after next
        if (k + S < p.supers && (!VEC || threadIdx.x == 96)) fetch(k + S);
        if (wid == 0) {
            Map m;
            uint32_t pc = 0;
#pragma unroll 4
            for (int w = 0; w < W; ++w) {
                const float2 v = agg[w][lane];
                agg[w][lane] = make_float2(m.a, m.b);
                pc |= (uint32_t)m.cut << w;
                m.then(v.x, v.y, sq.heads(w) != 0);
            }
            if (lane == 0) pcut = pc;
            peers.tell(buf, rank, p.cluster, m);
        } else if (wid == 1) {
            carry[lane] = walked;
        } else if (wid == 2) {
            if (k + 1 < p.supers) seqs[buf ^ 1].find(p, tile + p.cluster);
            empty_sequences(p, tile, cb, p.h0, p.ht);
        }
        __syncthreads();
        wait_peers(&peers.bar[buf], (k >> 1) & 1, p);
        if (wid == 1) walked = peers.through(buf, p.cluster, walked);
        F2 h = peers.entry(buf, rank, ch, F2(carry[ch], carry[ch + 1]));
        {
            const float4 m = *reinterpret_cast<const float4 *>(&agg[wid][ch]);
            h = (pcut >> wid) & 1 ? F2(m.y, m.w) : fma2(F2(m.x, m.z), h, F2(m.y, m.w));
        }
        if (p.states && wid % LR_BWD_WARPS == 0 && group == 0 && row0 < p.rows)
            put2<VEC>(p.states, (int64_t)(row0 / LR_TILE) * p.dim + c, h, c, p.dim);
        if (group) h = wheads & 0xff ? B0 : fma2(A0, h, B0);
        T *to = reinterpret_cast<T *>(p.h) + (int64_t)row0 * p.dim + c;
        if (plain && p.h) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                h = fma2(a[r], h, b[r]);
                put2<true>(to, 0, h, 0, 1);
                to += p.dim;
            }
        } else {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                h = (heads >> r) & 1 ? b[r] : fma2(a[r], h, b[r]);
                if (row0 + r < p.rows) {
                    if (p.h) put2<VEC>(to, (int64_t)r * p.dim, h, c, p.dim);
                    if (p.ht && (tails >> r) & 1) put2<VEC>(p.ht, (int64_t)sq.seq[first + r] * p.dim + c, h, c, p.dim);
                }
            }
        }
    }
    cluster_sync();  // no CTA ends while another may still write to it
}

// ---------------------------------------------------------------- backward
template <typename T, typename G> struct BwdStage {
    static constexpr int ROWS = LR_TILE;
    Tile<G, ROWS> g;
    Tile<T, ROWS> x, dh;
};

template <typename T, typename G, bool COMP, bool VEC>
__global__ void __launch_bounds__(32 * LR_BWD_WARPS, 2)
    k10_bwd(const __grid_constant__ LinrecParams p, const __grid_constant__ LinrecMaps maps) {
    using Stage = BwdStage<T, G>;
    constexpr int W = LR_BWD_WARPS, ROWS = Stage::ROWS, S = LR_BWD_STAGES;
    extern __shared__ __align__(128) char dynamic[];
    Stage *stages = reinterpret_cast<Stage *>(dynamic);
    __shared__ Sequences<ROWS> seqs[2];
    __shared__ __align__(16) float2 agg[W][LR_CH], fwd[W][LR_CH];  // a warp's maps, backward and forward
    __shared__ __align__(16) Peers peers;
    __shared__ __align__(8) uint64_t full[S];
    __shared__ __align__(8) float entry[W][LR_CH];  // the h that enters a warp's rows
    __shared__ uint32_t scut;                       // bit per warp: there is a cut in the tile's rows behind it
    __shared__ __align__(8) float carry[LR_CH];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = lane >> 4, ch = 2 * (lane & 15);
    const int rank = cluster_rank(), cb = blockIdx.x / p.cluster, c = cb * LR_CH + ch;

    // the scan goes from the last rows to the first, in the cluster too
    auto tile_of = [&](int k) { return (p.supers - k) * p.cluster - 1 - rank; };
    auto fetch = [&](int k) {
        Stage &st = stages[k % S];
        const int tile = tile_of(k);
        if (VEC) {
            mbar_expect_tx(&full[k % S], sizeof(Stage));
            load_tile(&st.g, &maps.g, cb * LR_CH, tile * ROWS, &full[k % S]);
            load_tile(&st.x, &maps.x, cb * LR_CH, tile * ROWS, &full[k % S]);
            load_tile(&st.dh, &maps.dh, cb * LR_CH, tile * ROWS, &full[k % S]);
        } else {
            st.g.bring(p.g, p.g_ts, tile, wid, cb, p);
            st.x.bring(p.x, p.x_ts, tile, wid, cb, p);
            st.dh.bring(p.dh, p.dh_ts, tile, wid, cb, p);
            __syncwarp();
        }
    };
    if (threadIdx.x == 0) {
        for (int q = 0; q < S; ++q) mbar_init(&full[q], 1);
        mbar_init(&peers.bar[0], 1);
        mbar_init(&peers.bar[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    check_sequences(p);
    if (wid == 2) seqs[0].find(p, tile_of(0));
    cluster_sync();
    for (int k = 0; k < S - 1 && k < p.supers; ++k)
        if (!VEC || threadIdx.x == 0) fetch(k);
    float walked = 0.f;
    for (int k = 0; k < p.supers; ++k) {
        const int buf = k & 1, tile = tile_of(k), first = wid * LR_WROWS + 8 * group, row0 = tile * ROWS + first;
        const Sequences<ROWS> &sq = seqs[buf];
        const Stage &st = stages[k % S];
        const uint32_t wheads = sq.heads(wid), heads = wheads >> (8 * group) & 0xff;
        const uint32_t wtails = sq.tails(wid), tails = wtails >> (8 * group) & 0xff;
        const bool plain = VEC && !(wheads | wtails) && tile * ROWS + (wid + 1) * LR_WROWS <= p.rows &&
                           (cb + 1) * LR_CH <= p.dim;
        auto dh_at = [&](int r, auto any) {  // with the gradient of the last state on a sequence's last row
            F2 d = st.dh.get(first + r, ch);
            if (any.value && (tails >> r) & 1)
                d = add2(d, get2(p.dht, (int64_t)sq.seq[first + r] * p.dim + c, c, p.dim));
            return d;
        };
        if (VEC) wait_phase(&full[k % S], (k / S) & 1, p);
        F2 a[8], rest[COMP ? 8 : 1], A, B, R;  // B, R: of the forward and the backward map
        auto compose = [&](auto any) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                float g0, g1;
                st.g.get(first + r, ch, g0, g1);
                F2 u;
                decay2(g0, g1, a[r], u);
                F2 b = st.x.get(first + r, ch);
                if (COMP) rest[r] = u, b = mul2(b, u);
                if (any.value && (heads >> r) & 1)
                    B = fma2(a[r], get2(p.h0, (int64_t)sq.seq[first + r] * p.dim + c, c, p.dim), b);
                else B = r == 0 ? b : fma2(a[r], B, b);
                A = r == 0 ? a[r] : mul2(A, a[r]);
            }
#pragma unroll
            for (int r = 7; r >= 0; --r) {
                const F2 d = dh_at(r, any);
                R = mul2(a[r], r == 7 || (any.value && (tails >> r) & 1) ? d : add2(d, R));
            }
        };
        if (plain) compose(Const<false>());
        else compose(Const<true>());
        // forward: the first group's map for the lanes of the second; backward: the second's for those of the first
        const F2 A0 = shfl2(A, lane & 15), B0 = shfl2(B, lane & 15), A1 = shfl2(A, lane | 16), R1 = shfl2(R, lane | 16);
        if (group) put_maps(&fwd[wid][ch], mul2(A, A0), heads ? B : fma2(A, B0, B));
        else put_maps(&agg[wid][ch], mul2(A, A1), tails ? R : fma2(A, R1, R));
        __syncthreads();
        // everybody is done with the tile before: its place takes the one S - 1 further on
        if (k + S - 1 < p.supers && (!VEC || threadIdx.x == 96)) fetch(k + S - 1);
        if (wid == 0) {
            Map m;
            uint32_t sc = 0;
#pragma unroll 4
            for (int w = W - 1; w >= 0; --w) {
                const float2 v = agg[w][lane];
                agg[w][lane] = make_float2(m.a, m.b);
                sc |= (uint32_t)m.cut << w;
                m.then(v.x, v.y, sq.tails(w) != 0);
            }
            if (lane == 0) scut = sc;
            peers.tell(buf, rank, p.cluster, m);
        } else if (wid == 1) {
            carry[lane] = walked;
            const int col = cb * LR_CH + lane;
            float h = !(sq.head[0] & 1) && tile > 0 && tile < p.tiles && col < p.dim ? p.states[(size_t)tile * p.dim + col] : 0.f;
#pragma unroll 4
            for (int w = 0; w < W; ++w) {
                entry[w][lane] = h;
                const float2 v = fwd[w][lane];
                h = sq.heads(w) ? v.y : fmaf(v.x, h, v.y);
            }
        } else if (wid == 2) {
            if (k + 1 < p.supers) seqs[buf ^ 1].find(p, tile - p.cluster);
            empty_sequences(p, tile, cb, p.dht, p.dh0);
        }
        __syncthreads();
        // the part that does not need what enters backwards: h_{t-1} of every row, less x_t with COMP
        F2 h(entry[wid][ch], entry[wid][ch + 1]), before[8];
        if (group) h = wheads & 0xff ? B0 : fma2(A0, h, B0);
        auto recompute = [&](auto any) {
#pragma unroll
            for (int r = 0; r < 8; ++r) {
                if (any.value && (heads >> r) & 1) h = get2(p.h0, (int64_t)sq.seq[first + r] * p.dim + c, c, p.dim);
                const F2 x = st.x.get(first + r, ch);
                before[r] = COMP ? fma2(x, F2(-1.f), h) : h;
                h = fma2(a[r], h, COMP ? mul2(x, rest[r]) : x);
            }
        };
        if (plain) recompute(Const<false>());
        else recompute(Const<true>());
        wait_peers(&peers.bar[buf], (k >> 1) & 1, p);
        if (wid == 1) walked = peers.through(buf, p.cluster, walked);
        F2 m = peers.entry(buf, rank, ch, F2(carry[ch], carry[ch + 1]));
        {
            const float4 q = *reinterpret_cast<const float4 *>(&agg[wid][ch]);
            m = (scut >> wid) & 1 ? F2(q.y, q.w) : fma2(F2(q.x, q.z), m, F2(q.y, q.w));
        }
        if (!group) m = wtails >> 8 ? R1 : fma2(A1, m, R1);
        auto finish = [&](auto any) {
            const int64_t end = (int64_t)(row0 + 7) * p.dim + c;
            T *dx = reinterpret_cast<T *>(p.dx) + end;
            G *dg = reinterpret_cast<G *>(p.dg) + end;
#pragma unroll
            for (int r = 7; r >= 0; --r) {
                const F2 d = dh_at(r, any), lam = any.value && (tails >> r) & 1 ? d : add2(d, m);
                m = mul2(a[r], lam);
                if (!any.value) {
                    put2<true>(dx, 0, COMP ? mul2(rest[r], lam) : lam, 0, 1);
                    put2<true>(dg, 0, mul2(m, before[r]), 0, 1);
                } else if (row0 + r < p.rows) {
                    put2<VEC>(dx, 0, COMP ? mul2(rest[r], lam) : lam, c, p.dim);
                    put2<VEC>(dg, 0, mul2(m, before[r]), c, p.dim);
                    if (p.dh0 && (heads >> r) & 1)
                        put2<VEC>(p.dh0, (int64_t)sq.seq[first + r] * p.dim + c, m, c, p.dim);
                }
                dx -= p.dim, dg -= p.dim;
            }
        };
        if (plain) finish(Const<false>());
        else finish(Const<true>());
    }
    cluster_sync();
}

// ---------------------------------------------------------------- single tokens
template <typename T, typename G, int V, bool COMP> __global__ void __launch_bounds__(128) k10_step(const StepParams p) {
    const int per = p.pieces.d;  // pieces of V channels in a row
    const int64_t e = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (e >= p.batch * per) return;
    const uint32_t i = p.pieces.div((uint32_t)e);
    const int c = ((uint32_t)e - i * per) * V;
    const int64_t slot = p.slots ? p.slots[i] : i;
    const Pack<G, V> gp = load_pack<G, V>(reinterpret_cast<const G *>(p.g) + (int64_t)i * p.g_ts + c);
    const Pack<T, V> xp = load_pack<T, V>(reinterpret_cast<const T *>(p.x) + (int64_t)i * p.x_ts + c);
    float y[V] = {}, g[V], x[V], h[V];
    unpack<G, V>(gp, g);
    unpack<T, V>(xp, x);
    if (slot >= 0 && slot < p.num_slots) {
        float *at = p.state + slot * p.dim + c;
        unpack<float, V>(load_pack<float, V>(at), h);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            F2 a, rest;
            decay2(g[j], g[j], a, rest);
            float a0, a1, r0, r1;
            a.get(a0, a1);
            rest.get(r0, r1);
            y[j] = fmaf(a0, h[j], COMP ? r0 * x[j] : x[j]);
        }
        store_pack<float, V>(at, y);
    }
    store_pack<T, V>(reinterpret_cast<T *>(p.y) + (int64_t)i * p.dim + c, y);
}

}  // namespace

#define RUN(KERNEL, STAGE, STAGES, THREADS)                                                         \
    do {                                                                                            \
        constexpr int smem = (int)sizeof(STAGE) * STAGES;                                           \
        LinrecLaunch l((const void *)KERNEL, THREADS, smem);                                        \
        cudaError_t e = linrec_plan(p, l, STAGE::ROWS, stream);                                     \
        LinrecMaps maps;                                                                            \
        if (e == cudaSuccess && p.vec) e = linrec_maps(p, maps, STAGE::ROWS);                       \
        if (e != cudaSuccess) return e;                                                             \
        return cudaLaunchKernelEx(&l.cfg, KERNEL, static_cast<const LinrecParams>(p), static_cast<const LinrecMaps>(maps)); \
    } while (0)
#define RUN_ALL(KERNEL, STAGE, STAGES, THREADS)                                                     \
    do {                                                                                            \
        using Stage = STAGE;                                                                        \
        if (p.vec && p.complement) RUN((KERNEL<T, G, true, true>), Stage, STAGES, THREADS);         \
        if (p.vec) RUN((KERNEL<T, G, false, true>), Stage, STAGES, THREADS);                        \
        if (p.complement) RUN((KERNEL<T, G, true, false>), Stage, STAGES, THREADS);                 \
        RUN((KERNEL<T, G, false, false>), Stage, STAGES, THREADS);                                  \
    } while (0)

template <typename T, typename G> cudaError_t linrec_fwd_t(LinrecParams &p, cudaStream_t stream) {
    using FS = FwdStage<T, G>;
    RUN_ALL(k10_fwd, FS, LR_FWD_STAGES, 32 * LR_FWD_WARPS);
}
template <typename T, typename G> cudaError_t linrec_bwd_t(LinrecParams &p, cudaStream_t stream) {
    using BS = BwdStage<T, G>;
    RUN_ALL(k10_bwd, BS, LR_BWD_STAGES, 32 * LR_BWD_WARPS);
}
#undef RUN
#undef RUN_ALL

template <typename T, typename G> cudaError_t linrec_step_t(StepParams &p, cudaStream_t stream) {
#define RUN(V, COMP)                                                                                        \
    do {                                                                                                    \
        p.pieces = FastDiv::of((uint32_t)(p.dim / V));                                                      \
        k10_step<T, G, V, COMP><<<(unsigned)((p.batch * (p.dim / V) + 127) / 128), 128, 0, stream>>>(p);    \
    } while (0)
    if (p.vec) {
        if (p.complement) RUN(4, true);
        else RUN(4, false);
    } else {
        if (p.complement) RUN(1, true);
        else RUN(1, false);
    }
#undef RUN
    return cudaGetLastError();
}

// what a translation unit instantiates for its activation and gate types
#define LINREC_INSTANTIATE(T, G)                                                   \
    template cudaError_t linrec_fwd_t<T, G>(LinrecParams &, cudaStream_t);         \
    template cudaError_t linrec_bwd_t<T, G>(LinrecParams &, cudaStream_t);         \
    template cudaError_t linrec_step_t<T, G>(StepParams &, cudaStream_t);

}  // namespace gdr
