// k10_linrec.cuh -- the gated linear recurrence, forward and backward (included once per activation type):
//
//   h_t = a_t h_{t-1} + b_t ,  a = exp(g) ,  b = x or (1 - a) x          per channel, packed or dense sequences
//   m_t = a_t (dh_t + m_{t+1}) ;  dx_t = dh_t + m_{t+1} (times 1 - a_t) ;  dg_t = m_t (h_{t-1} - x_t or 0)
//
// Both directions are scans of maps s -> A s + B, which compose as (A2 A1, A2 B1 + B2).  The rows are cut into tiles,
// whatever the sequences: where a sequence starts (or, backwards, ends) inside a tile, the row's map forgets what
// came before it (a flag rather than A = 0, so that a nan does not pass from one sequence to the next).
//
// A cluster of CTAs owns a block of 32 channels and goes through all rows, a tile for each CTA at a time.  Eight lanes
// with four channels each (backwards 16 with two) compose a group of 8 rows and keep a and b in registers; the groups' maps
// are composed over shared memory, four to a lane, and the tile's map is sent to every CTA of the cluster, which then knows
// the state that enters its own tile and finishes its rows.  So every value is read once and written once, nothing is
// exchanged through memory, and the order of all sums is fixed: results are bit-identical from run to run.  The next
// tile arrives by tensor-map loads meanwhile.  The forward saves the state that enters each LR_SAVE rows (a warp's rows of
// the backward), from which the backward recomputes h instead of reading it back rounded.
//
// Measured: 32768 x 2048 bf16 with fp32 gates forward 0.096 ms (5.6 TB/s of the 6.8 of a plain copy), backward 0.164 ms
// (5.8); 48763 x 4096 bf16 with 1 - a, packed, forward 0.280 ms (4.3), backward 0.486 ms (4.2); 30000 x 16384 forward
// 0.533 ms (5.5).  Bytes do not bind it yet but, SM by SM, the instructions (24 to an element, backwards 43, half of them the
// exponential) between the two barriers of a tile and the cluster's exchange.  Widths of 2048 or 4096 make 64 or 128 blocks
// of channels, whose clusters fill 93 or 84 % of the SMs' places.  CTAs of 4 warps, of which an SM holds five (backwards five or six),
// hide the exchange best: 8 warps took 0.310 ms where 4 took 0.289 and 2 took 0.302 (48763 x 4096, forward, an earlier state).
#pragma once

#include "block_common.cuh"
#include "tc_util.cuh"

namespace gdr {
namespace {

using tc::mbar_expect_tx;
using tc::mbar_init;
using tc::mbar_wait;

constexpr int LR_R = 8;                       // rows of a group
constexpr int LR_FWD_PER = 4, LR_BWD_PER = 2;  // groups of a warp
static_assert(LR_SAVE == LR_BWD_PER * LR_R, "a saved state enters each warp's rows of the backward");

// exp(g) and 1 - exp(g).  Near a = 1 both are right to rounding and without a lean to one side, which a channel that
// remembers hundreds of tokens would add up (decays near 1 that come out a quarter of a unit too low put h off by 1e-5).
// Cody and Waite's reduction g = n ln 2 + r, then exp(r) - 1 = r + r^2 q(r) with q a Chebyshev fit of degree 4 (1e-8 off).
// ln 2 is one constant, 1.9e-9 off, which n times leans further out, where a state is soon forgotten.  a is off, in units of
// 2^-24, at most and on average: gates in [-1, 0] 1.3, 0.0; [-10, -1] 1.6, 0.3; [-40, -10] 3.1, 1.2; [-87, -40] 5.2, 2.9; [0, 1]
// 1.3, 0.0; [1, 10] 1.6, -0.3; [10, 88] 5.2, -2.3.  Below -87.7 a is 0; above 88.3 it is taken at 88.3.
__device__ __forceinline__ void decay2(F2 g, F2 &a, F2 &rest) {
    const F2 shift(12582912.f), one(1.f);  // 1.5 x 2^23: the sum's low bits are the rounded integer
    const F2 t = fma2(g, F2(1.44269504f), shift), n = add2(t, F2(-12582912.f));
    const F2 r = fma2(n, F2(-0.693147181f), g);  // (ln 2 is 1.9e-9 off: n times that, a rounding of a at a = 1e-9)
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

// Two gates as they lie in memory, taken to [-88, 88] (16-bit types: both by one instruction) or [-88, 88.3]; a nan stays one.
__device__ __forceinline__ F2 gates(Pack<float, 2> g) {
    const float lo = -88.f, hi = 88.3f;
    asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+f"(g.v[0]) : "f"(hi), "f"(lo));
    asm("min.NaN.f32 %0, %0, %1;\n\tmax.NaN.f32 %0, %0, %2;" : "+f"(g.v[1]) : "f"(hi), "f"(lo));
    return F2(g.v[0], g.v[1]);
}
__device__ __forceinline__ F2 gates(Pack<__nv_bfloat16, 2> g) {
    uint32_t v = *reinterpret_cast<uint32_t *>(&g);
    asm("min.NaN.bf16x2 %0, %0, %1;\n\tmax.NaN.bf16x2 %0, %0, %2;" : "+r"(v) : "r"(0x42b042b0u), "r"(0xc2b0c2b0u));
    return F2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ F2 gates(Pack<__half, 2> g) {
    uint32_t v = *reinterpret_cast<uint32_t *>(&g);
    asm("min.NaN.f16x2 %0, %0, %1;\n\tmax.NaN.f16x2 %0, %0, %2;" : "+r"(v) : "r"(0x55805580u), "r"(0xd580d580u));
    const __half2 h = *reinterpret_cast<__half2 *>(&v);
    return F2(__low2float(h), __high2float(h));
}

// Four neighbouring channels of a row.
struct F4 {
    F2 lo, hi;
};
__device__ __forceinline__ F4 fma4(F4 a, F4 b, F4 c) { return {fma2(a.lo, b.lo, c.lo), fma2(a.hi, b.hi, c.hi)}; }
__device__ __forceinline__ F4 mul4(F4 a, F4 b) { return {mul2(a.lo, b.lo), mul2(a.hi, b.hi)}; }
__device__ __forceinline__ F4 make4(float x, float y, float z, float w) { return {F2(x, y), F2(z, w)}; }

// ---------------------------------------------------------------- maps
// The maps of W groups (or warps).  Rows of 34 put the lanes of a scan on different banks and each pair of maps on 16 bytes.
template <int W> using Maps = float2[W][LR_CH + 2];

__device__ __forceinline__ void put_pair(float2 *at, F2 a, F2 b) {
    float x, y, u, v;
    a.get(x, y), b.get(u, v);
    *reinterpret_cast<float4 *>(at) = make_float4(x, u, y, v);
}
__device__ __forceinline__ void get_pair(const float2 *at, F2 &a, F2 &b) {
    const float4 m = *reinterpret_cast<const float4 *>(at);
    a = F2(m.x, m.z), b = F2(m.y, m.w);
}

// Composes W maps along the scan (from the last to the first with BACK): in place each becomes the map of the rows before
// it, and `total` that of all of them.  A warp takes its share of the channels, its lanes share out the positions: each
// composes some in turn, the lanes' maps over distances 1, 2 and 4, and its own again from what comes before them; bit j
// of cuts: the map at position j cuts off what came before.
template <int WARPS, int W, bool BACK, bool CUTS>
__device__ __forceinline__ void scan_maps(Maps<W> &maps, uint32_t cuts, int wid, int lane, float2 *total) {
    constexpr int CH = LR_CH / WARPS, PARTS = 32 / CH, N = W / PARTS;  // channels of a warp, lanes of one, positions of a lane
    static_assert(W <= 32 && N >= 1 && N * PARTS == W, "");
    const int part = lane / CH, ch = CH * wid + lane % CH;
    auto at = [&](int i) -> float2 & { return maps[BACK ? W - 1 - part * N - i : part * N + i][ch]; };
    float2 m[N];
#pragma unroll
    for (int i = 0; i < N; ++i) m[i] = at(i);
    auto add = [&](float2 first, int i) {  // the map of position i after that of the rows before it
        const bool cut = CUTS && (cuts >> (part * N + i)) & 1;
        return make_float2(m[i].x * first.x, cut ? m[i].y : fmaf(m[i].x, first.y, m[i].y));
    };
    float2 own = m[0];
#pragma unroll
    for (int i = 1; i < N; ++i) own = add(own, i);
#pragma unroll
    for (int d = 1; d < PARTS; d *= 2) {
        const float a1 = __shfl_up_sync(0xffffffffu, own.x, CH * d), b1 = __shfl_up_sync(0xffffffffu, own.y, CH * d);
        if (part >= d) {
            const bool cut = CUTS && (cuts >> ((part - d + 1) * N)) & ((1u << (d * N)) - 1);
            if (!cut) own.y = fmaf(own.x, b1, own.y);
            own.x *= a1;
        }
    }
    if (part == PARTS - 1) total[ch] = own;
    float2 before = make_float2(__shfl_up_sync(0xffffffffu, own.x, CH), __shfl_up_sync(0xffffffffu, own.y, CH));
    if (part == 0) before = make_float2(1.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        at(i) = before;
        if (i + 1 < N) before = add(before, i);
    }
}
// Two channels' states taken through a map that scan_maps left; cut: that map cuts off.
__device__ __forceinline__ F2 through(const float2 *m, bool cut, const float *s) {
    F2 a, b;
    get_pair(m, a, b);
    return cut ? b : fma2(a, F2(s[0], s[1]), b);
}
__device__ __forceinline__ F2 shfl2(F2 v, int lane) {
    float x, y;
    v.get(x, y);
    return F2(__shfl_sync(0xffffffffu, x, lane), __shfl_sync(0xffffffffu, y, lane));
}

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
    // by every warp, which has its channels of `total`: this CTA's map to all
    template <int WARPS> __device__ __forceinline__ void tell(int buf, int rank, int size, const float2 *total, bool c) {
        constexpr int PER = LR_CH / WARPS;  // channels of a warp
        const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, ch = PER * wid + lane % PER;
        __syncwarp();
        if (threadIdx.x == 32) mbar_expect_tx(&bar[buf], (uint32_t)size * (LR_CH * 8 + 4));
        uint64_t v;
        asm("mov.b64 %0, {%1, %2};" : "=l"(v) : "f"(total[ch].x), "f"(total[ch].y));
        for (int q = lane / PER; q < size; q += 32 / PER)
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b64 [%0], %1, [%2];" ::"r"(
                             in_cta(&map[buf][rank][ch], q)),
                         "l"(v), "r"(in_cta(&bar[buf], q))
                         : "memory");
        if (wid == 0 && lane < size)
            asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(
                             in_cta(&cut[buf][rank], lane)),
                         "r"((int)c), "r"(in_cta(&bar[buf], lane))
                         : "memory");
    }
    // For a lane's channel, the state s that enters the cluster's rows taken through the tiles before that of CTA `rank`;
    // s itself is taken through all of them.
    __device__ __forceinline__ float entry(int buf, int rank, int size, float &s) const {
        float at = s;
        for (int q = 0; q < size; ++q) {
            const float2 v = map[buf][q][threadIdx.x & 31];
            if (q == rank) at = s;
            s = cut[buf][q] ? v.y : fmaf(v.x, s, v.y);
        }
        return at;
    }
};

// ---------------------------------------------------------------- a tile's rows
// Which rows of a tile are the first or the last of a sequence.
template <int ROWS> struct Ends {
    static constexpr int R = LR_R;
    uint32_t head[ROWS / 32], tail[ROWS / 32];  // a bit for each row; written where there is any
    bool any;
    // by one warp; [a, b): the sequence that the warp met last, with which it goes on
    __device__ __forceinline__ void find(const LinrecParams &p, int tile, int &a, int &b) {
        const int lane = threadIdx.x & 31, row0 = tile * ROWS, end = min(row0 + ROWS, p.rows);
        if (row0 < p.rows && !(a <= row0 && row0 < b)) sequence_of(p, row0, a, b);
        if (row0 >= p.rows || (a < row0 && b > end)) {  // the tile lies within one sequence, or has no rows
            if (lane == 0) any = false;
            return;
        }
        if (lane == 0) any = true;
        for (int k = 0; k < ROWS / 32; ++k) {
            const int row = row0 + 32 * k + lane;
            int from = -1, to = -1;
            if (row < p.rows) sequence_of(p, row, from, to);
            const uint32_t h = __ballot_sync(0xffffffffu, from == row), e = __ballot_sync(0xffffffffu, to == row + 1);
            if (lane == 0) head[k] = h, tail[k] = e;
        }
    }
    // the last sequence that starts at or before the row, and its rows
    static __device__ __forceinline__ int sequence_of(const LinrecParams &p, int row, int &a, int &b) {
        int s;
        if (p.cu) {
            int hi = p.N;
            s = 0;
            while (hi - s > 1) {
                const int mid = (s + hi) >> 1;
                if (p.cu[mid] <= row) s = mid;
                else hi = mid;
            }
            a = p.cu[s], b = p.cu[s + 1];
        } else {
            s = p.per_seq.div(row);
            a = s * p.tokens, b = a + p.tokens;
        }
        return s;
    }
    static __device__ __forceinline__ int sequence_of(const LinrecParams &p, int row) {
        int a, b;
        return sequence_of(p, row, a, b);
    }
    // of a group's rows
    __device__ __forceinline__ uint32_t heads(int g) const { return head[g * R / 32] >> (g * R % 32) & ((1u << R) - 1); }
    __device__ __forceinline__ uint32_t tails(int g) const { return tail[g * R / 32] >> (g * R % 32) & ((1u << R) - 1); }
    // bit per group: a sequence starts among its rows
    __device__ __forceinline__ uint32_t head_cuts() const {
        constexpr int N = ROWS / R;  // groups
        static_assert(N <= 32 && (N & (N - 1)) == 0, "a lane for each group");
        return __ballot_sync(0xffffffffu, heads(threadIdx.x & (N - 1))) & (0xffffffffu >> (32 - N));
    }
    // bit per warp, from the last one on: a sequence ends among its rows
    __device__ __forceinline__ uint32_t tail_cuts() const {
        constexpr int N = ROWS / LR_SAVE;  // warps
        const int w = N - 1 - (threadIdx.x & (N - 1));
        const uint32_t e = tail[w * LR_SAVE / 32] >> (w * LR_SAVE % 32) & ((1u << LR_SAVE) - 1);
        return __ballot_sync(0xffffffffu, e) & ((1u << N) - 1);
    }
};

// A tile of one tensor in shared memory: ROWS rows of 32 channels.
template <typename T, int ROWS> struct Tile {
    T v[ROWS][LR_CH];
    __device__ __forceinline__ void get(int r, int ch, float (&o)[4]) const {
        unpack<T, 4>(*reinterpret_cast<const Pack<T, 4> *>(&v[r][ch]), o);
    }
    __device__ __forceinline__ F4 get4(int r, int ch) const {
        float o[4];
        get(r, ch, o);
        return make4(o[0], o[1], o[2], o[3]);
    }
    __device__ __forceinline__ F2 get2(int r, int ch) const {
        const Pack<T, 2> q = *reinterpret_cast<const Pack<T, 2> *>(&v[r][ch]);
        return F2(to_f32(q.v[0]), to_f32(q.v[1]));
    }
    // Where the rows cannot be moved by a tensor map a warp brings its own N: by asynchronous copies of pieces, or 16 single
    // elements at a time where those have 16 bits and nothing larger is aligned (32768 x 2052 bf16 with fp32 gates forward
    // 0.189 ms, 2050 0.197, 2049 0.267; by registers, 16 loads at a time, 0.265, 0.297 and 0.323).
    template <int N>
    __device__ __forceinline__ void bring(const void *src, int64_t ts, int piece, int tile, int wid, int cb, const LinrecParams &p) {
        const T *from = reinterpret_cast<const T *>(src);
        if (piece == 4) pieces<N, 4>(from, ts, tile, wid, cb, p);
        else if (piece == 2) pieces<N, 2>(from, ts, tile, wid, cb, p);
        else if constexpr (sizeof(T) == 4) pieces<N, 1>(from, ts, tile, wid, cb, p);
        else singles<N>(from, ts, tile, wid, cb, p);
    }
    template <int N, int E>
    __device__ __forceinline__ void pieces(const T *src, int64_t ts, int tile, int wid, int cb, const LinrecParams &p) {
        constexpr int LANES = LR_CH / E, STEP = 32 / LANES, BYTES = E * (int)sizeof(T);
        const int lane = threadIdx.x & 31, r0 = wid * N + lane / LANES, row0 = tile * ROWS + r0, ch = lane % LANES * E;
        const int c = cb * LR_CH + ch;
        const T *from = src + (int64_t)row0 * ts + c;
        if ((tile + 1) * ROWS <= p.rows && (cb + 1) * LR_CH <= p.dim) {
#pragma unroll
            for (int r = 0; r < N; r += STEP, from += STEP * ts) copy_piece<BYTES>(&v[r0 + r][ch], from);
        } else {
            for (int r = 0; r < N; r += STEP, from += STEP * ts) {
                if (row0 + r < p.rows && c < p.dim) {
                    copy_piece<BYTES>(&v[r0 + r][ch], from);
                } else {
#pragma unroll
                    for (int j = 0; j < E; ++j) v[r0 + r][ch + j] = to_out_t<T>(0.f);
                }
            }
        }
    }
    template <int N>
    __device__ __forceinline__ void singles(const T *src, int64_t ts, int tile, int wid, int cb, const LinrecParams &p) {
        const int lane = threadIdx.x & 31, c = cb * LR_CH + lane;
        for (int r0 = wid * N; r0 < (wid + 1) * N; r0 += 16) {
            T x[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) {
                const int row = tile * ROWS + r0 + r;
                x[r] = to_out_t<T>(0.f);
                if (row < p.rows && c < p.dim) x[r] = src[(int64_t)row * ts + c];
            }
#pragma unroll
            for (int r = 0; r < 16; ++r) v[r0 + r][lane] = x[r];
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

// Two or four neighbouring values of a row, of which `piece` at a time are aligned and lie inside together; VEC: all.
template <bool VEC, typename T> __device__ __forceinline__ void put2(T *p, F2 v, int c, int dim, int piece) {
    float o[2];
    v.get(o[0], o[1]);
    if (VEC || piece >= 2) {
        if (c < dim) store_pack<T, 2>(p, o);
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j)
            if (c + j < dim) p[j] = to_out_t<T>(o[j]);
    }
}
template <bool VEC, typename T> __device__ __forceinline__ void put4(T *p, F4 v, int c, int dim, int piece) {
    if (VEC || piece == 4) {
        float o[4];
        v.lo.get(o[0], o[1]), v.hi.get(o[2], o[3]);
        if (c < dim) store_pack<T, 4>(p, o);
    } else {
        put2<false>(p, v.lo, c, dim, piece);
        put2<false>(p + 2, v.hi, c + 2, dim, piece);
    }
}
__device__ __forceinline__ F2 row2(const float *p, int64_t row, int c, int dim) {
    return F2(p && c < dim ? p[row * dim + c] : 0.f, p && c + 1 < dim ? p[row * dim + c + 1] : 0.f);
}
// Four channels of an fp32 row that may be absent (zero).
__device__ __forceinline__ F4 row4(const float *p, int64_t row, int c, int dim) {
    float o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = p && c + j < dim ? p[row * dim + c + j] : 0.f;
    return make4(o[0], o[1], o[2], o[3]);
}

// Sequences without a token have no row: their last state is their first (forward), their gradients pass through
// (backward).  The cluster's warps share out the sequences of its block of channels.
__device__ __forceinline__ void empty_sequences(const LinrecParams &p, int rank, int cb, const float *from, float *to) {
    if ((!p.cu && p.tokens > 0) || !to) return;
    const int lane = threadIdx.x & 31, c = cb * LR_CH + lane;
    const int warps = blockDim.x >> 5;
    for (int base = 32 * (rank * warps + (int)(threadIdx.x >> 5)); base < p.N; base += 32 * warps * p.cluster) {
        const int s = base + lane;
        uint32_t empty = __ballot_sync(0xffffffffu, s < p.N && (!p.cu || p.cu[s] == p.cu[s + 1]));
        for (; empty; empty &= empty - 1) {
            const int64_t at = (int64_t)(base + __ffs(empty) - 1) * p.dim + c;
            if (c < p.dim) to[at] = from ? from[at] : 0.f;
        }
    }
}

// cu_seqlens that do not rise from 0 to the number of rows are reported.  The first CTA checks short lists and sets the word;
// the grid shares long ones, for which it was cleared before.
__device__ __noinline__ void check_sequences(const LinrecParams &p) {
    if (p.clear && blockIdx.x) return;
    bool bad = false;
    if (p.cu) {
        const int t = blockIdx.x * blockDim.x + threadIdx.x, n = p.clear ? blockDim.x : gridDim.x * blockDim.x;
        bad = t == 0 && (p.cu[0] != 0 || p.cu[p.N] != p.rows);
#pragma unroll 4
        for (int s = t; s < p.N; s += n) bad |= p.cu[s + 1] < p.cu[s];
    }
    if (p.clear) {
        const bool any = __syncthreads_or(bad);
        if (threadIdx.x == 0) *p.status = any ? ST_BAD_SEQLENS : 0;
    } else if (bad) {
        atomicOr(p.status, ST_BAD_SEQLENS);
    }
}

// What the two kernels have in common: a CTA's shared memory besides the stages.
template <int ROWS, int S, int W> struct LinrecSmem {
    alignas(16) Maps<W> maps;
    Peers peers;
    float2 total[LR_CH];          // the tile's map
    float carry[LR_CH];           // what enters the tile
    uint64_t full[S];             // a stage's rows are there
    Ends<ROWS> ends[2];
    uint32_t again;               // the channels that go token by token
};

// A warp's copies of its own rows have arrived, but for the LEFT groups of them issued last.
template <int LEFT> __device__ __forceinline__ void own_rows_there() {
    copies_wait<LEFT>();
    __syncwarp();
}

__device__ __forceinline__ void init_barriers(uint64_t *full, int stages, Peers &peers, uint32_t &again) {
    if (threadIdx.x == 0) {
        again = 0;
        for (int q = 0; q < stages; ++q) mbar_init(&full[q], 1);
        mbar_init(&peers.bar[0], 1);
        mbar_init(&peers.bar[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
}

// ---------------------------------------------------------------- growth
// The walk's maps need factors of at most 1, which decays have.  Gates above 0 grow: the factor of some rows then passes fp32,
// and makes a nan of a state of 0 and of growth that later decays take back; a factor that underflowed has lost what
// growth would bring back; and an infinite state times such a factor is a nan.  So the walk looks for groups that grow and for
// tiles that are entered by an infinity or a nan, and marks their channels, without a value kept for it.  Where there are
// marks, the cluster goes through its rows once more when the walk has ended, as the recurrence is written: a lane for
// each channel, a warp for each range of rows, first for the range's map, its factor with the exponent apart, then for
// the rows themselves.  Channels that do have a decay above 1 or an infinity keep what this gives.  Gates of at most 0 and
// finite states mark nothing; the walk takes 0 to 3 % longer for looking.  32768 x 2048 bf16 with fp32 gates on both
// sides of 0: forward 0.76 ms, backward 1.28 (one lane a channel from the first row to the last: 11 and 18 ms).
struct Watch {
    uint32_t *again;  // in shared memory, a bit for each channel
    uint32_t channels;
    __device__ __forceinline__ Watch(uint32_t &a, uint32_t c) : again(&a), channels(c) {}
    __device__ __forceinline__ void factors(F2 a, F2 b) const {  // (a nan counts: infinity times 0)
        float x, y, z, w;
        a.get(x, y), b.get(z, w);
        if (__builtin_expect(!(x <= 1.f) | !(y <= 1.f) | !(z <= 1.f) | !(w <= 1.f), 0)) atomicOr(again, channels);
    }
    __device__ __forceinline__ void entered(float s) const {  // by a lane for each channel
        if (__builtin_expect(!(fabsf(s) < INFINITY), 0)) atomicOr(again, 1u << (threadIdx.x & 31));
    }
    // Before the cluster's last barrier: this CTA's marks to all.
    __device__ __forceinline__ void tell(int size) const {
        __syncthreads();
        const uint32_t c = *again;
        if (c && (int)threadIdx.x < size)
            asm volatile("red.relaxed.cluster.shared::cluster.or.b32 [%0], %1;" ::"r"(in_cta(again, threadIdx.x)), "r"(c) : "memory");
    }
};

// A map of one channel whose factor is m 2^e, m in [1, 2) or 0 or a nan.
struct WideMap {
    float m, b;
    int e, how;  // CUTS: it forgets what came before; MET: growth or an infinity among its rows
    static constexpr int CUTS = 1, MET = 2;
    __device__ __forceinline__ void factor(float a) {
        const bool up = a > 1.f;  // (neither product leaves fp32: a is below 2^128, and may be as small as 2^-127)
        m *= up ? 0.25f * a : a, e += up ? 2 : 0;
        if (m < 1.17549435e-38f) m *= 0x1p64f, e -= 64;
        if (m > 0.f && m < INFINITY) {
            const int x = (__float_as_int(m) >> 23) - 127;
            m = __int_as_float(__float_as_int(m) - (x << 23));
            e = max(min(e + x, 1 << 28), -(1 << 28));  // (far beyond what any state comes back from)
        }
    }
    __device__ __forceinline__ float operator()(float s) const {
        if (how & CUTS) return b;
        float v = 0.5f * m * s;  // (at most s)
        for (int left = max(min(e + 1, 400), -400); left;) {  // (towards the result from one side: no step passes it)
            const int x = max(min(left, 100), -100);
            v *= __int_as_float((x + 127) << 23), left -= x;
        }
        return v + b;
    }
};

// The cluster's rows in ranges of whole blocks of LR_SAVE, one for each warp.
struct Range {
    int from, to, index, ranges;
    __device__ __forceinline__ Range(const LinrecParams &p, int rank) {
        const int warps = blockDim.x >> 5;
        index = rank * warps + (int)(threadIdx.x >> 5), ranges = p.cluster * warps;
        const int64_t blocks = (p.rows + LR_SAVE - 1) / LR_SAVE, n = (blocks + ranges - 1) / ranges * LR_SAVE;
        from = (int)min((int64_t)p.rows, n * index), to = (int)min((int64_t)p.rows, n * (index + 1));
    }
};
// Which rows of a block are the first or the last of a sequence: a bit for each.  By a whole warp.
struct BlockEnds {
    uint32_t heads, tails;
    __device__ __forceinline__ BlockEnds(const LinrecParams &p, int first) {
        const int row = first + (threadIdx.x & 31);
        int a = -1, b = -1;
        if (row < min(first + LR_SAVE, p.rows)) Ends<32>::sequence_of(p, row, a, b);
        heads = __ballot_sync(0xffffffffu, a == row), tails = __ballot_sync(0xffffffffu, b == row + 1);
        heads &= (1u << LR_SAVE) - 1, tails &= (1u << LR_SAVE) - 1;
    }
};
// A channel's values in a block of rows; zeros (and decays of 1) past the last row, and for a channel that is none.
template <typename T, typename G, bool COMP> struct Block {
    float a[LR_SAVE], b[LR_SAVE], rest[COMP ? LR_SAVE : 1], x[COMP ? LR_SAVE : 1];
    __device__ __forceinline__ void read(const LinrecParams &p, int first, int c, bool on) {
        const T *xp = reinterpret_cast<const T *>(p.x) + c;
        const G *gp = reinterpret_cast<const G *>(p.g) + c;
#pragma unroll
        for (int r = 0; r < LR_SAVE; r += 2) {
            Pack<G, 2> g;
            float v[2] = {};
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int64_t row = first + r + j;
                g.v[j] = to_out_t<G>(0.f);
                if (on && row < p.rows) g.v[j] = gp[row * p.g_ts], v[j] = to_f32(xp[row * p.x_ts]);
            }
            F2 a2, r2;
            decay2(gates(g), a2, r2);
            float q[2];
            a2.get(a[r], a[r + 1]), r2.get(q[0], q[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                b[r + j] = COMP ? v[j] * q[j] : v[j];
                if (COMP) rest[r + j] = q[j], x[r + j] = v[j];
            }
        }
    }
};
// What enters a warp's range, from the maps of those before it (BACK: after it), and whether any of all has met something.
template <bool BACK> __device__ __forceinline__ float enter_range(WideMap own, const Range &range, WideMap *maps, bool &met) {
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    maps[threadIdx.x] = own;
    cluster_sync();
    float s = 0.f, at = 0.f;
    met = false;
    for (int i = 0; i < range.ranges; ++i) {
        const int q = BACK ? range.ranges - 1 - i : i;
        if (q == range.index) at = s;
        uint32_t m, b, e, how;
        asm volatile("ld.shared::cluster.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(m), "=r"(b), "=r"(e), "=r"(how)
                     : "r"(in_cta(&maps[q % warps * 32 + lane], q / warps))
                     : "memory");
        const WideMap map = {__uint_as_float(m), __uint_as_float(b), (int)e, (int)how};
        s = map(s);
        met |= (how & WideMap::MET) || fabsf(s) == INFINITY;
    }
    cluster_sync();  // no CTA ends while another reads its maps
    return at;
}
static_assert(sizeof(WideMap) == 16, "");

// By all threads of the cluster.  maps: one for each thread, in shared memory.
template <typename T, typename G, bool COMP>
__device__ __noinline__ void forward_again(const LinrecParams &p, int rank, int c, bool on, WideMap *maps) {
    const Range range(p, rank);
    Block<T, G, COMP> v;
    auto first_state = [&](int row) { return p.h0 && on ? p.h0[(int64_t)Ends<32>::sequence_of(p, row) * p.dim + c] : 0.f; };
    WideMap map = {1.f, 0.f, 0, 0};
    for (int first = range.from; first < range.to; first += LR_SAVE) {
        const BlockEnds ends(p, first);
        v.read(p, first, c, on);
#pragma unroll
        for (int r = 0; r < LR_SAVE; ++r) {
            if (ends.heads >> r & 1) map.b = first_state(first + r), map.how |= WideMap::CUTS;
            map.b = fmaf(v.a[r], map.b, v.b[r]);
            map.factor(v.a[r]);
            if (v.a[r] > 1.f || fabsf(map.b) == INFINITY) map.how |= WideMap::MET;
        }
    }
    bool met;
    float h = enter_range<false>(map, range, maps, met);
    const bool write = on && met;
    for (int first = range.from; first < range.to; first += LR_SAVE) {
        const BlockEnds ends(p, first);
        v.read(p, first, c, on);
        if (write && p.states) p.states[(int64_t)(first / LR_SAVE) * p.dim + c] = h;
#pragma unroll
        for (int r = 0; r < LR_SAVE; ++r) {
            if (ends.heads >> r & 1) h = first_state(first + r);
            h = fmaf(v.a[r], h, v.b[r]);
            if (!write || first + r >= p.rows) continue;
            if (p.h) reinterpret_cast<T *>(p.h)[(int64_t)(first + r) * p.dim + c] = to_out_t<T>(h);
            if (p.ht && (ends.tails >> r & 1)) p.ht[(int64_t)Ends<32>::sequence_of(p, first + r) * p.dim + c] = h;
        }
    }
}

template <typename T, typename G, bool COMP>
__device__ __noinline__ void backward_again(const LinrecParams &p, int rank, int c, bool on, WideMap *maps) {
    const Range range(p, rank);
    Block<T, G, COMP> v;
    auto of_sequence = [&](const float *q, int row) { return q && on ? q[(int64_t)Ends<32>::sequence_of(p, row) * p.dim + c] : 0.f; };
    // lambda before the rows after are added, with the gradient of the last state on a sequence's last row
    auto dh_at = [&](int row, bool tail) {
        float d = on && row < p.rows ? to_f32(reinterpret_cast<const T *>(p.dh)[(int64_t)row * p.dh_ts + c]) : 0.f;
        if (tail) d += of_sequence(p.dht, row);
        return d;
    };
    auto entering = [&](int first) { return on ? p.states[(int64_t)(first / LR_SAVE) * p.dim + c] : 0.f; };
    const int last = range.from + (range.to - range.from - 1) / LR_SAVE * LR_SAVE;  // block
    WideMap map = {1.f, 0.f, 0, 0};
    for (int first = last; first >= range.from && range.from < range.to; first -= LR_SAVE) {
        const BlockEnds ends(p, first);
        v.read(p, first, c, on);
        if (!(ends.heads & 1) && fabsf(entering(first)) == INFINITY) map.how |= WideMap::MET;
#pragma unroll
        for (int r = LR_SAVE - 1; r >= 0; --r) {
            const bool tail = ends.tails >> r & 1;
            const float d = dh_at(first + r, tail), lam = tail ? d : d + map.b;
            if (tail) map.how |= WideMap::CUTS;
            map.b = v.a[r] * lam;
            map.factor(v.a[r]);
            if (v.a[r] > 1.f || fabsf(lam) == INFINITY) map.how |= WideMap::MET;
        }
    }
    bool met;
    float m = enter_range<true>(map, range, maps, met);
    const bool write = on && met;
    for (int first = last; first >= range.from && range.from < range.to; first -= LR_SAVE) {
        const BlockEnds ends(p, first);
        v.read(p, first, c, on);
        float before[LR_SAVE], h = entering(first);
#pragma unroll
        for (int r = 0; r < LR_SAVE; ++r) {
            if (ends.heads >> r & 1) h = of_sequence(p.h0, first + r);
            before[r] = COMP ? h - v.x[COMP ? r : 0] : h;
            h = fmaf(v.a[r], h, v.b[r]);
        }
#pragma unroll
        for (int r = LR_SAVE - 1; r >= 0; --r) {
            const bool tail = ends.tails >> r & 1;
            const float d = dh_at(first + r, tail), lam = tail ? d : d + m;
            m = v.a[r] * lam;
            if (!write || first + r >= p.rows) continue;
            const int64_t at = (int64_t)(first + r) * p.dim + c;
            reinterpret_cast<T *>(p.dx)[at] = to_out_t<T>(COMP ? v.rest[COMP ? r : 0] * lam : lam);
            reinterpret_cast<G *>(p.dg)[at] = to_out_t<G>(m * before[r]);
            if (p.dh0 && (ends.heads >> r & 1)) p.dh0[(int64_t)Ends<32>::sequence_of(p, first + r) * p.dim + c] = m;
        }
    }
}

// ---------------------------------------------------------------- forward
template <typename T, typename G, int WARPS> struct FwdStages {
    static constexpr int GROUPS = LR_FWD_PER * WARPS, ROWS = LR_R * GROUPS, S = 1;
    static constexpr uint32_t BYTES = sizeof(Tile<G, ROWS>) + sizeof(Tile<T, ROWS>);
    Tile<G, ROWS> g[S];
    Tile<T, ROWS> x[S];
};

template <typename T, typename G, int WARPS, bool COMP, bool VEC>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 4 ? 5 : 2)
    k10_fwd(const __grid_constant__ LinrecParams p, const __grid_constant__ LinrecMaps maps) {
    using Stages = FwdStages<T, G, WARPS>;
    constexpr int R = LR_R, ROWS = Stages::ROWS, S = Stages::S, GROUPS = Stages::GROUPS;
    extern __shared__ __align__(128) char dynamic[];
    Stages &st = *reinterpret_cast<Stages *>(dynamic);
    __shared__ __align__(16) LinrecSmem<ROWS, S, GROUPS> sm;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = threadIdx.x >> 3, ch = 4 * (lane & 7);
    const int rank = cluster_rank(), cb = blockIdx.x / p.cluster, c = cb * LR_CH + ch;
    const bool channels = (cb + 1) * LR_CH <= p.dim;

    auto fetch = [&](int k) {  // VEC: one thread; else every warp
        const int tile = k * p.cluster + rank;
        if (VEC) {
            mbar_expect_tx(&sm.full[k % S], Stages::BYTES);
            load_tile(&st.g[k % S], &maps.g, cb * LR_CH, tile * ROWS, &sm.full[k % S]);
            load_tile(&st.x[k % S], &maps.x, cb * LR_CH, tile * ROWS, &sm.full[k % S]);
        } else {
            st.g[k % S].template bring<LR_FWD_PER * R>(p.g, p.g_ts, p.g_piece, tile, wid, cb, p);
            st.x[k % S].template bring<LR_FWD_PER * R>(p.x, p.x_ts, p.x_piece, tile, wid, cb, p);
            copies_issued();
        }
    };
    init_barriers(sm.full, S, sm.peers, sm.again);
    check_sequences(p);
    int sa = 0, sb = 0;  // (warp 2) the sequence met last
    if (wid == 2) sm.ends[0].find(p, rank, sa, sb);
    cluster_sync();  // the barriers are there, everywhere
    for (int k = 0; k < S && k < p.supers; ++k)
        if (!VEC || threadIdx.x == 0) fetch(k);
    __syncwarp();
    empty_sequences(p, rank, cb, p.h0, p.ht);
    float walked = 0.f;  // (warp 1) the state that enters the cluster's rows
    const Watch watch(sm.again, 0xfu << ch);
    for (int k = 0; k < p.supers; ++k) {
        const int buf = k & 1, tile = k * p.cluster + rank, first = group * R, row0 = tile * ROWS + first;
        const Ends<ROWS> &ends = sm.ends[buf];
        const auto &gt = st.g[k % S];
        const auto &xt = st.x[k % S];
        // as a rule every row and channel is there, and no sequence starts or ends among the warp's rows
        bool plain = channels && (tile + 1) * ROWS <= p.rows;
        uint32_t cuts = 0, heads = 0, tails = 0;
        if (ends.any) {
            cuts = ends.head_cuts(), heads = ends.heads(group), tails = ends.tails(group);
            plain = plain && !__any_sync(0xffffffffu, heads | tails);
        }
        if (VEC) wait_phase(&sm.full[k % S], (k / S) & 1, p);
        else own_rows_there<0>();
        F4 a[R], b[R], A, B;
        auto compose = [&](auto any) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const Pack<G, 4> g = *reinterpret_cast<const Pack<G, 4> *>(&gt.v[first + r][ch]);
                F4 rest;
                decay2(gates(*reinterpret_cast<const Pack<G, 2> *>(&g.v[0])), a[r].lo, rest.lo);
                decay2(gates(*reinterpret_cast<const Pack<G, 2> *>(&g.v[2])), a[r].hi, rest.hi);
                b[r] = xt.get4(first + r, ch);
                if (COMP) b[r] = mul4(b[r], rest);
                if (any.value && (heads >> r) & 1) {
                    b[r] = fma4(a[r], row4(p.h0, ends.sequence_of(p, row0 + r), c, p.dim), b[r]);
                    B = b[r];
                } else {
                    B = r == 0 ? b[r] : fma4(a[r], B, b[r]);
                }
                A = r == 0 ? a[r] : mul4(A, a[r]);
            }
        };
        if (plain) compose(Const<false>());
        else compose(Const<true>());
        put_pair(&sm.maps[group][ch], A.lo, B.lo);
        put_pair(&sm.maps[group][ch + 2], A.hi, B.hi);
        watch.factors(A.lo, A.hi);
        __syncthreads();
        // the tile's rows are in registers: their place takes the tile S further on
        if (k + S < p.supers && (!VEC || threadIdx.x == 96)) fetch(k + S);
        if (cuts) scan_maps<WARPS, GROUPS, false, true>(sm.maps, cuts, wid, lane, sm.total);
        else scan_maps<WARPS, GROUPS, false, false>(sm.maps, cuts, wid, lane, sm.total);
        sm.peers.template tell<WARPS>(buf, rank, p.cluster, sm.total, cuts != 0);
        if (wid == 1) {
            wait_peers(&sm.peers.bar[buf], (k >> 1) & 1, p);
            sm.carry[lane] = sm.peers.entry(buf, rank, p.cluster, walked);
            watch.entered(sm.carry[lane]);
        } else if (wid == 2) {
            if (k + 1 < p.supers) sm.ends[buf ^ 1].find(p, tile + p.cluster, sa, sb);
        }
        __syncthreads();
        const bool cut = cuts & ((1u << group) - 1);
        F4 h = {through(&sm.maps[group][ch], cut, &sm.carry[ch]), through(&sm.maps[group][ch + 2], cut, &sm.carry[ch + 2])};
        if (p.states && first % LR_SAVE == 0 && row0 < p.rows)
            put4<VEC>(p.states + (int64_t)(row0 / LR_SAVE) * p.dim + c, h, c, p.dim, 1);
        T *to = reinterpret_cast<T *>(p.h) + (int64_t)row0 * p.dim + c;
        if (plain && p.h) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = fma4(a[r], h, b[r]);
                put4<VEC>(to, h, VEC ? 0 : c, VEC ? 1 : p.dim, p.x_piece);
                to += p.dim;
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = (heads >> r) & 1 ? b[r] : fma4(a[r], h, b[r]);
                if (row0 + r < p.rows) {
                    if (p.h) put4<VEC>(to + (int64_t)r * p.dim, h, c, p.dim, p.x_piece);
                    if (p.ht && (tails >> r) & 1)
                        put4<VEC>(p.ht + (int64_t)ends.sequence_of(p, row0 + r) * p.dim + c, h, c, p.dim, 1);
                }
            }
        }
    }
    watch.tell(p.cluster);
    cluster_sync();  // no CTA ends while another may still write to it
    if (const uint32_t again = sm.again)
        forward_again<T, G, COMP>(p, rank, cb * LR_CH + lane, (again >> lane & 1) && cb * LR_CH + lane < p.dim,
                                  reinterpret_cast<WideMap *>(dynamic));
}

// ---------------------------------------------------------------- backward
// g is done with when the groups' maps are formed and its place then takes the tile after next; x and dh are read again to
// finish a tile, and theirs takes the next but one when the next tile's maps are formed.
template <typename T, typename G, int WARPS> struct BwdStages {
    static constexpr int ROWS = LR_R * LR_BWD_PER * WARPS;
    Tile<G, ROWS> g[2];
    Tile<T, ROWS> x[2], dh[2];
};

template <typename T, typename G, int WARPS, bool COMP, bool VEC>
__global__ void __launch_bounds__(32 * WARPS, WARPS == 4 ? 6 : 3)
    k10_bwd(const __grid_constant__ LinrecParams p, const __grid_constant__ LinrecMaps maps) {
    using Stages = BwdStages<T, G, WARPS>;
    constexpr int R = LR_R, ROWS = Stages::ROWS;
    extern __shared__ __align__(128) char dynamic[];
    Stages &st = *reinterpret_cast<Stages *>(dynamic);
    __shared__ __align__(16) LinrecSmem<ROWS, 4, WARPS> sm;  // full: of g's two places, of those of x and dh
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, group = threadIdx.x >> 4, ch = 2 * (lane & 15);
    const int rank = cluster_rank(), cb = blockIdx.x / p.cluster, c = cb * LR_CH + ch;
    const bool channels = (cb + 1) * LR_CH <= p.dim;

    // the scan goes from the last rows to the first, in the cluster too
    auto tile_of = [&](int k) { return (p.supers - k) * p.cluster - 1 - rank; };
    auto fetch_g = [&](int k) {
        const int buf = k & 1, tile = tile_of(k);
        if (VEC) {
            mbar_expect_tx(&sm.full[buf], sizeof(st.g[0]));
            load_tile(&st.g[buf], &maps.g, cb * LR_CH, tile * ROWS, &sm.full[buf]);
        } else {
            st.g[buf].template bring<LR_BWD_PER * R>(p.g, p.g_ts, p.g_piece, tile, wid, cb, p);
            copies_issued();
        }
    };
    auto fetch_x = [&](int k) {
        const int buf = k & 1, tile = tile_of(k);
        if (VEC) {
            mbar_expect_tx(&sm.full[2 + buf], 2 * sizeof(st.x[0]));
            load_tile(&st.x[buf], &maps.x, cb * LR_CH, tile * ROWS, &sm.full[2 + buf]);
            load_tile(&st.dh[buf], &maps.dh, cb * LR_CH, tile * ROWS, &sm.full[2 + buf]);
        } else {
            st.x[buf].template bring<LR_BWD_PER * R>(p.x, p.x_ts, p.x_piece, tile, wid, cb, p);
            st.dh[buf].template bring<LR_BWD_PER * R>(p.dh, p.dh_ts, p.x_piece, tile, wid, cb, p);
            copies_issued();
        }
    };
    init_barriers(sm.full, 4, sm.peers, sm.again);
    check_sequences(p);
    int sa = 0, sb = 0;
    if (wid == 2) sm.ends[0].find(p, tile_of(0), sa, sb);
    cluster_sync();
    if (!VEC || threadIdx.x == 0) {
        fetch_g(0);
        fetch_x(0);
        if (p.supers > 1) fetch_g(1);
        else if (!VEC) copies_issued();
    }
    __syncwarp();
    empty_sequences(p, rank, cb, p.dht, p.dh0);
    float walked = 0.f;
    const Watch watch(sm.again, 3u << ch);
    for (int k = 0; k < p.supers; ++k) {
        const int buf = k & 1, tile = tile_of(k), first = group * R, row0 = tile * ROWS + first;
        const Ends<ROWS> &ends = sm.ends[buf];
        const auto &gt = st.g[buf];
        const auto &xt = st.x[buf], &dt = st.dh[buf];
        bool plain = channels && (tile + 1) * ROWS <= p.rows;
        uint32_t tcuts = 0, heads = 0, tails = 0;
        if (ends.any) {
            tcuts = ends.tail_cuts(), heads = ends.heads(group), tails = ends.tails(group);
            plain = plain && !__any_sync(0xffffffffu, heads | tails);
        }
        const int warp0 = tile * ROWS + wid * LR_SAVE;  // the warp's first row
        // the h that enters it
        F2 h = VEC && plain ? *reinterpret_cast<const F2 *>(p.states + (int64_t)(warp0 / LR_SAVE) * p.dim + c)
                     : row2(warp0 < p.rows ? p.states : nullptr, warp0 / LR_SAVE, c, p.dim);
        if (VEC) {
            wait_phase(&sm.full[buf], (k >> 1) & 1, p);
            wait_phase(&sm.full[2 + buf], (k >> 1) & 1, p);
        } else {
            own_rows_there<1>();  // (the next tile's g may be under way)
        }
        auto dh_at = [&](int r, auto any) {  // with the gradient of the last state on a sequence's last row
            F2 d = dt.get2(first + r, ch);
            if (any.value && (tails >> r) & 1) d = add2(d, row2(p.dht, ends.sequence_of(p, row0 + r), c, p.dim));
            return d;
        };
        F2 a[R], rest[COMP ? R : 1], A, B, Q;  // B, Q: of the group's forward and backward map
        auto compose = [&](auto any) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const Pack<G, 2> g = *reinterpret_cast<const Pack<G, 2> *>(&gt.v[first + r][ch]);
                F2 u;
                decay2(gates(g), a[r], u);
                F2 b = xt.get2(first + r, ch);
                if (COMP) rest[r] = u, b = mul2(b, u);
                if (any.value && (heads >> r) & 1) B = fma2(a[r], row2(p.h0, ends.sequence_of(p, row0 + r), c, p.dim), b);
                else B = r == 0 ? b : fma2(a[r], B, b);
                A = r == 0 ? a[r] : mul2(A, a[r]);
            }
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                const F2 d = dh_at(r, any);
                Q = mul2(a[r], r == R - 1 || (any.value && (tails >> r) & 1) ? d : add2(d, Q));
            }
        };
        if (plain) compose(Const<false>());
        else compose(Const<true>());
        // backward: the second group's map for the lanes of the first, which leave the warp's
        const uint32_t ended = __ballot_sync(0xffffffffu, tails);
        const F2 A1 = shfl2(A, lane | 16), Q1 = shfl2(Q, lane | 16);
        if (lane < 16) put_pair(&sm.maps[wid][ch], mul2(A, A1), tails ? Q : fma2(A, Q1, Q));
        // forward: what leaves the first group enters the second
        const F2 out = shfl2(heads ? B : fma2(A, h, B), lane & 15);
        if (lane >= 16) h = out;
        __syncthreads();
        if (tcuts) scan_maps<WARPS, WARPS, true, true>(sm.maps, tcuts, wid, lane, sm.total);
        else scan_maps<WARPS, WARPS, true, false>(sm.maps, tcuts, wid, lane, sm.total);
        sm.peers.template tell<WARPS>(buf, rank, p.cluster, sm.total, tcuts != 0);
        watch.factors(A, A);
        // everybody is done with this tile's g and with x and dh of the tile before
        if (!VEC || threadIdx.x == 96) {
            if (k + 1 < p.supers) fetch_x(k + 1);
            if (k + 2 < p.supers) fetch_g(k + 2);
            else if (!VEC) copies_issued();  // (none: what is waited for is all but the last)
        }
        if (wid == 1) {
            wait_peers(&sm.peers.bar[buf], (k >> 1) & 1, p);
            sm.carry[lane] = sm.peers.entry(buf, rank, p.cluster, walked);
            watch.entered(sm.carry[lane]);
        } else if (wid == 2) {
            if (k + 1 < p.supers) sm.ends[buf ^ 1].find(p, tile - p.cluster, sa, sb);
        }
        __syncthreads();
        F2 m = through(&sm.maps[wid][ch], tcuts & ((1u << (WARPS - 1 - wid)) - 1), &sm.carry[ch]);
        if (lane < 16) m = ended >> 16 ? Q1 : fma2(A1, m, Q1);
        auto finish = [&](auto any) {
            F2 before[R];  // h_{t-1}, less x_t with COMP
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (any.value && (heads >> r) & 1) h = row2(p.h0, ends.sequence_of(p, row0 + r), c, p.dim);
                const F2 x = xt.get2(first + r, ch);
                before[r] = COMP ? fma2(x, F2(-1.f), h) : h;
                h = fma2(a[r], h, COMP ? mul2(x, rest[r]) : x);
            }
            const int64_t end = (int64_t)(row0 + R - 1) * p.dim + c;
            T *dx = reinterpret_cast<T *>(p.dx) + end;
            G *dg = reinterpret_cast<G *>(p.dg) + end;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {
                const F2 d = dh_at(r, any), lam = any.value && (tails >> r) & 1 ? d : add2(d, m);
                m = mul2(a[r], lam);
                if (!any.value) {
                    put2<VEC>(dx, COMP ? mul2(rest[r], lam) : lam, VEC ? 0 : c, VEC ? 1 : p.dim, p.x_piece);
                    put2<VEC>(dg, mul2(m, before[r]), VEC ? 0 : c, VEC ? 1 : p.dim, p.g_piece);
                } else if (row0 + r < p.rows) {
                    put2<VEC>(dx, COMP ? mul2(rest[r], lam) : lam, c, p.dim, p.x_piece);
                    put2<VEC>(dg, mul2(m, before[r]), c, p.dim, p.g_piece);
                    if (p.dh0 && (heads >> r) & 1)
                        put2<VEC>(p.dh0 + (int64_t)ends.sequence_of(p, row0 + r) * p.dim + c, m, c, p.dim, 1);
                }
                dx -= p.dim, dg -= p.dim;
            }
        };
        if (plain) finish(Const<false>());
        else finish(Const<true>());
    }
    watch.tell(p.cluster);
    cluster_sync();
    if (const uint32_t again = sm.again)
        backward_again<T, G, COMP>(p, rank, cb * LR_CH + lane, (again >> lane & 1) && cb * LR_CH + lane < p.dim,
                                   reinterpret_cast<WideMap *>(dynamic));
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
            decay2(gates(Pack<float, 2>{g[j], g[j]}), a, rest);
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

// Few blocks of channels leave the SMs with one or two CTAs each, which then wait for each tile: CTAs of 8 warps take twice
// the rows to a tile (65536 x 512 bf16 forward 0.072 ms, backward 0.132; 4 warps 0.085, 0.155).
#define RUN(KERNEL, STAGES, WARPS, COMP, VEC)                                                       \
    do {                                                                                            \
        auto kernel = KERNEL<T, G, WARPS, COMP, VEC>;                                               \
        using Stages = STAGES<T, G, WARPS>;                                                         \
        LinrecLaunch l((const void *)kernel, 32 * WARPS, (int)sizeof(Stages));                      \
        bool narrow = false;                                                                        \
        cudaError_t e = linrec_plan(p, l, Stages::ROWS, WARPS == 4 ? &narrow : nullptr, stream);    \
        if (narrow) break;                                                                          \
        LinrecMaps maps;                                                                            \
        if (e == cudaSuccess && p.vec) e = linrec_maps(p, maps, Stages::ROWS);                      \
        if (e != cudaSuccess) return e;                                                             \
        return cudaLaunchKernelEx(&l.cfg, kernel, static_cast<const LinrecParams>(p), static_cast<const LinrecMaps>(maps)); \
    } while (0)
#define RUN_ALL(KERNEL, STAGES, WARPS)                                                              \
    do {                                                                                            \
        if (p.vec && p.complement) RUN(KERNEL, STAGES, WARPS, true, true);                          \
        else if (p.vec) RUN(KERNEL, STAGES, WARPS, false, true);                                    \
        else if (p.complement) RUN(KERNEL, STAGES, WARPS, true, false);                             \
        else RUN(KERNEL, STAGES, WARPS, false, false);                                              \
    } while (0)

template <typename T, typename G> cudaError_t linrec_fwd_t(LinrecParams &p, cudaStream_t stream) {
    RUN_ALL(k10_fwd, FwdStages, 4);
    RUN_ALL(k10_fwd, FwdStages, 8);
    return cudaErrorUnknown;
}
template <typename T, typename G> cudaError_t linrec_bwd_t(LinrecParams &p, cudaStream_t stream) {
    RUN_ALL(k10_bwd, BwdStages, 4);
    RUN_ALL(k10_bwd, BwdStages, 8);
    return cudaErrorUnknown;
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
