// k10_linrec.cuh -- the gated linear recurrence, forward and backward (included once per activation type):
//
//   h_t = a_t h_{t-1} + b_t ,  a = exp(g) ,  b = x or (1 - a) x          per channel, packed or dense sequences
//   m_t = a_t (dh_t + m_{t+1}) ;  dx_t = dh_t + m_{t+1} (times 1 - a_t) ;  dg_t = m_t (h_{t-1} - x_t or 0)
//
// Both directions are scans of maps s -> A s + B, which compose as (A2 A1, A2 B1 + B2).  The rows are cut into tiles
// of LR_TILE, whatever the sequences: where a sequence starts (or, backwards, ends) inside a tile, the row's map
// forgets what came before it (a flag rather than A = 0, so that a nan does not pass from one sequence to the next).
// A CTA takes one tile of 32 V channels: each of its 8 warps composes 8 rows, the warps' maps meet in shared memory,
// and the tile's map is left for the tiles behind it.  The state that enters the tile is then composed from the maps
// of the tiles before it, in a fixed tree: 8 tiles make a group, 8 groups a block, 8 blocks a span; the last tile of a
// group, block or span leaves the map of the whole (the state itself, for a span).  So every value is read once and
// written once, the state needs one hop through memory per span of 512 tiles rather than per tile, and the order of
// all sums is fixed: results are bit-identical from run to run.
//
// CTAs take their tiles by a ticket, in the order of the scan, so the tiles that one waits for belong to CTAs that
// already run; the waits are bounded all the same.  The forward saves the state that enters each tile, from which the
// backward recomputes h inside the tile instead of reading it back rounded.
#pragma once

#include "block_common.cuh"

namespace gdr {
namespace {

constexpr int LR_WARPS = 8, LR_ROWS = LR_TILE / LR_WARPS, LR_THREADS = 32 * LR_WARPS;

// exp(g) and 1 - exp(g), both to about one unit in the last place and without a lean to one side, which a channel that
// remembers hundreds of tokens would add up (a function that returns decays near 1 a quarter of a unit too low puts
// h off by 1e-5).  Cody and Waite's reduction g = n ln 2 + r, then exp(r) - 1 = r + r^2 q(r) with q a Chebyshev fit
// of degree 4 (1e-8 off), so that 1 - a is exact to rounding near a = 1.  Below -87.7 a is 0; above 88.3 it is
// taken at 88.3.
__device__ __forceinline__ void decay(float g, float &a, float &rest) {
    asm("min.NaN.f32 %0, %0, 0f42B09A1D;\n\tmax.NaN.f32 %0, %0, 0fC2B00000;" : "+f"(g));  // [-88, 88.301]
    const float shift = 12582912.f;  // 1.5 x 2^23: the sum's low bits are the rounded integer
    const float t = fmaf(g, 1.44269504f, shift), n = t - shift;
    float r = fmaf(n, -0.693359375f, g);
    r = fmaf(n, 2.12194440e-4f, r);
    float q = fmaf(r, 0.0013933823f, 0.0083632953f);
    q = fmaf(q, r, 0.041666463f);
    q = fmaf(q, r, 0.16666576f);
    q = fmaf(q, r, 0.5f);
    const float p = fmaf(r * r, q, r);
    const float s = __int_as_float((__float_as_int(t) << 23) + 0x3f800000);  // 2^n
    a = fmaf(p, s, s);
    rest = fmaf(-p, s, 1.f - s);
}

// ---------------------------------------------------------------- the tree of maps in the workspace
__device__ __forceinline__ void publish(int *flag, int value) {
    asm volatile("st.release.gpu.global.b32 [%0], %1;" ::"l"(flag), "r"(value) : "memory");
}
__device__ __forceinline__ int peek(const int *flag) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(flag) : "memory");
    return v;
}

// One warp waits until each lane's flag (null: none) is set; returns the lane's flag (0 when the wait gave up).
__device__ __forceinline__ int wait_flag(const int *flag, const LinrecParams &p) {
    int v = flag ? peek(flag) : 1;
    for (uint32_t polls = 0; __any_sync(0xffffffffu, v == 0); ++polls) {
        if (polls >= p.spin || ((polls & 255) == 255 && (*(volatile int *)p.status & ST_TIMEOUT))) {
            if (v == 0) atomicOr(p.status, ST_TIMEOUT);
            break;
        }
        __nanosleep(32);
        if (flag && v == 0) v = peek(flag);
    }
    return v;
}

// The map s -> a s + b, or b where what came before is cut off.
struct Map {
    float a = 1.f, b = 0.f;
    bool cut = false;
    __device__ __forceinline__ void then(float a2, float b2, bool cut2) {
        b = cut2 ? b2 : fmaf(a2, b, b2);
        a *= a2;
        cut |= cut2;
    }
    __device__ __forceinline__ void then(const Map &m) { then(m.a, m.b, m.cut); }
    __device__ __forceinline__ float of(float s) const { return cut ? b : fmaf(a, s, b); }
};

template <int CB> struct ScanSmem {
    uint32_t head[2], tail[2];  // bit per row of the tile: first / last of its sequence
    int seq[LR_TILE];           // the row's sequence
    int ticket;
    uint32_t cuts;  // of the records waited for: tiles at bit 0, groups at 8, blocks at 16
    float carry[CB];
    float2 agg[LR_WARPS][CB];
};

// A tile's place in the tree, i counted along the scan, and the state that enters it.
template <int CB> struct Tree {
    const LinrecParams &p;
    ScanSmem<CB> &sm;
    const int i, cb, col;  // col: the thread's channel, for the first CB threads
    const bool owner;
    __device__ __forceinline__ Tree(const LinrecParams &p_, ScanSmem<CB> &s, int i_, int cb_)
        : p(p_), sm(s), i(i_), cb(cb_), col(cb_ * CB + (int)threadIdx.x), owner(threadIdx.x < CB && col < p_.dim) {}

    __device__ __forceinline__ int *flag(int level, int k) const { return p.flags[level] + (size_t)k * p.nblk + cb; }
    __device__ __forceinline__ float2 *rec(int level, int k) const { return p.recs[level] + (size_t)k * p.dim; }

    // Leaves a map for the tiles behind; called by the owners' warps.
    __device__ __forceinline__ void leave(int level, int k, const Map &m) const {
        if (owner) __stcg(rec(level, k) + col, make_float2(m.a, m.b));
        asm volatile("bar.sync 1, %0;" ::"n"(CB) : "memory");
        if (threadIdx.x == 0) publish(flag(level, k), 1 | (m.cut ? 2 : 0));
    }

    // The last warp waits for the records before this tile at the levels of `which`; everybody meets afterwards.
    __device__ __forceinline__ void wait(int which) const {
        if (threadIdx.x / 32 == LR_WARPS - 1) {
            const int lane = threadIdx.x & 31, level = lane >> 3, j = lane & 7;
            const int *f = nullptr;
            if ((which >> level) & 1) {
                const int at = i >> (3 * level);
                if (level < 3 && j < (at & 7)) f = flag(level, (at & ~7) + j);
                if (level == 3 && j == 0 && at > 0) f = flag(3, at - 1);
            }
            const int v = wait_flag(f, p);
            const uint32_t cuts = __ballot_sync(0xffffffffu, f && (v & 2));
            if (lane == 0) sm.cuts = cuts;
        }
        __syncthreads();
    }

    // The map of the records before this tile at one level.
    __device__ __forceinline__ Map before(int level) const {
        Map m;
        if (owner) {
            const int at = i >> (3 * level), n = at & 7;
            float2 v[7];
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < n) v[j] = __ldcg(rec(level, (at & ~7) + j) + col);
#pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < n) m.then(v[j].x, v[j].y, (sm.cuts >> (8 * level + j)) & 1);
        }
        return m;
    }

    // Every thread calls this, the owners with the tile's map of their channel.  cut: that map forgets what came before;
    // need: the state that enters the tile matters (it is left in sm.carry); last: no tile follows.  All three are the
    // same for the whole CTA.
    __device__ __forceinline__ void enter(const Map &mine, bool cut, bool need, bool last) const {
        const bool closes = !last && (i & 7) == 7;
        const int closed = (i & 511) == 511 ? 3 : (i & 63) == 63 ? 2 : 1;  // level of what this tile closes
        const bool warps = threadIdx.x < CB;
        if (!last && !closes && warps) leave(0, i, mine);
        if (closes && cut) {  // what came before does not matter to those behind
            if (warps) leave(closed, i >> (3 * closed), mine);
        } else if (closes) {
            Map whole[4];
            wait(1);
            if (warps) {
                whole[0] = before(0);
                whole[0].then(mine);
                if (closed == 1) leave(1, i >> 3, whole[0]);
            }
            if (closed >= 2) {
                __syncthreads();
                wait(2);
                if (warps) {
                    whole[1] = before(1);
                    whole[1].then(whole[0]);
                    if (closed == 2) leave(2, i >> 6, whole[1]);
                }
            }
            if (closed == 3) {
                __syncthreads();
                wait(4 | 8);
                if (warps) {
                    if (i >> 9 && owner) whole[3].then(0.f, __ldcg(rec(3, (i >> 9) - 1) + col).y, true);
                    whole[2] = before(2);
                    whole[2].then(whole[1]);
                    whole[3].then(whole[2]);
                    whole[3].cut = true;  // a state, not a map
                    leave(3, i >> 9, whole[3]);
                }
            }
            __syncthreads();
        }
        if (need) {
            wait(15);
            if (owner) {
                Map m;
                if (i >> 9) m.then(0.f, __ldcg(rec(3, (i >> 9) - 1) + col).y, true);
                m.then(before(2));
                m.then(before(1));
                m.then(before(0));
                sm.carry[threadIdx.x] = m.b;
            }
        }
        __syncthreads();
    }
};

// First and last rows of sequences in the tile that starts at row0, and the rows' sequences.
template <int CB> __device__ __forceinline__ void find_sequences(const LinrecParams &p, ScanSmem<CB> &sm, int row0) {
    const int t = threadIdx.x;
    if (t < LR_TILE) {
        const int row = row0 + t;
        int s = 0;
        bool head = false, tail = false;
        if (row < p.rows) {
            if (p.cu) {
                int lo = 0, hi = p.N;  // the last sequence that starts at or before the row
                while (hi - lo > 1) {
                    const int mid = (lo + hi) >> 1;
                    if (p.cu[mid] <= row) lo = mid;
                    else hi = mid;
                }
                s = lo;
                head = p.cu[s] == row;
                tail = p.cu[s + 1] == row + 1;
            } else {
                s = p.per_seq.div(row);
                const int at = row - s * p.tokens;
                head = at == 0;
                tail = at == p.tokens - 1;
            }
        }
        sm.seq[t] = s;
        const uint32_t hb = __ballot_sync(0xffffffffu, head), tb = __ballot_sync(0xffffffffu, tail);
        if ((t & 31) == 0) sm.head[t >> 5] = hb, sm.tail[t >> 5] = tb;
    }
}

// Sequences without a token have no row: their last state is their first (forward), their gradients pass through
// (backward).  The tiles share them out, and check cu_seqlens on the way; returns whether a fault was found.
template <int CB>
__device__ __forceinline__ bool empty_sequences(const LinrecParams &p, int64_t i, int64_t n, int cb, const float *from,
                                                float *to) {
    if (!p.cu && p.tokens > 0) return false;
    const int64_t lo = p.N * i / n, hi = p.N * (i + 1) / n;
    bool bad = p.cu && i == 0 && (p.cu[0] != 0 || p.cu[p.N] != p.rows);
    for (int64_t s = lo + threadIdx.x / CB; s < hi; s += LR_THREADS / CB) {
        if (p.cu) {
            const int a = p.cu[s], b = p.cu[s + 1];
            bad |= b < a;
            if (a != b) continue;
        }
        const int c = cb * CB + threadIdx.x % CB;
        if (to && c < p.dim) to[s * p.dim + c] = from ? from[s * p.dim + c] : 0.f;
    }
    return bad;
}

template <int CB> __device__ __forceinline__ void note_faults(const LinrecParams &p, int cb, bool bad) {
    if (p.walk) {  // one CTA writes the status word, which nothing else clears
        if (cb == 0) {
            bad = __syncthreads_or(bad);
            if (threadIdx.x == 0) *p.status = bad ? ST_BAD_SEQLENS : 0;
        }
    } else if (bad) {
        atomicOr(p.status, ST_BAD_SEQLENS);
    }
}

template <typename T, int V>
__device__ __forceinline__ void load_row(const void *base, int64_t at, bool on, float (&o)[V]) {
    Pack<T, V> v = {};
    if (on) v = load_pack<T, V>(reinterpret_cast<const T *>(base) + at);
    unpack<T, V>(v, o);
}
template <int V> __device__ __forceinline__ void load_f32(const float *base, int64_t at, bool on, float (&o)[V]) {
    load_row<float, V>(base, at, on && base, o);
}

template <int V> constexpr int block_channels() { return 32 * V; }

// ---------------------------------------------------------------- forward
template <typename T, typename G, int V, bool COMP>
__global__ void __launch_bounds__(LR_THREADS, 2) k10_fwd(const LinrecParams p) {
    constexpr int CB = block_channels<V>();
    __shared__ ScanSmem<CB> sm;
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, lc = lane * V;
    int i = 0, cb = blockIdx.x;
    if (!p.walk) {
        if (threadIdx.x == 0) sm.ticket = atomicAdd(p.ticket, 1);
        __syncthreads();
        i = p.blocks.div(sm.ticket);
        cb = sm.ticket - i * p.nblk;
    }
    const int c = cb * CB + lc;
    const bool on = c < p.dim;
    bool bad = false;
    do {
        const int row0 = i * LR_TILE + wid * LR_ROWS;
        float a[LR_ROWS][V], b[LR_ROWS][V];
#pragma unroll
        for (int r = 0; r < LR_ROWS; ++r) {
            const bool live = on && row0 + r < p.rows;
            load_row<G, V>(p.g, (int64_t)(row0 + r) * p.g_ts + c, live, a[r]);
            load_row<T, V>(p.x, (int64_t)(row0 + r) * p.x_ts + c, live, b[r]);
        }
        find_sequences<CB>(p, sm, i * LR_TILE);
        __syncthreads();
        const uint32_t heads = sm.head[wid >> 2] >> (8 * (wid & 3)) & 0xff;
        const uint32_t tails = sm.tail[wid >> 2] >> (8 * (wid & 3)) & 0xff;
        float A[V], B[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.f, B[j] = 0.f;
#pragma unroll
        for (int r = 0; r < LR_ROWS; ++r) {
            const bool head = (heads >> r) & 1;
            float first[V];
            if (head) load_f32<V>(p.h0, (int64_t)sm.seq[wid * LR_ROWS + r] * p.dim + c, on, first);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                float rest;
                decay(a[r][j], a[r][j], rest);
                if (COMP) b[r][j] *= rest;
                if (head) b[r][j] = B[j] = fmaf(a[r][j], first[j], b[r][j]);
                else B[j] = fmaf(a[r][j], B[j], b[r][j]);
                A[j] *= a[r][j];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sm.agg[wid][lc + j] = make_float2(A[j], B[j]);
        __syncthreads();
        const uint64_t cuts = sm.head[0] | (uint64_t)sm.head[1] << 32;
        const bool need = !(cuts & 1) && i > 0, last = i + 1 == p.tiles;
        Map mine;
        if (threadIdx.x < CB)
#pragma unroll
            for (int w = 0; w < LR_WARPS; ++w) {
                const float2 m = sm.agg[w][threadIdx.x];
                mine.then(m.x, m.y, (cuts >> (8 * w)) & 0xff);
            }
        if (!p.walk) Tree<CB>(p, sm, i, cb).enter(mine, cuts != 0, need, last);
        if (need && p.states && threadIdx.x < CB && cb * CB + threadIdx.x < p.dim)
            p.states[(size_t)i * p.dim + cb * CB + threadIdx.x] = sm.carry[threadIdx.x];
        float h[V];
#pragma unroll
        for (int j = 0; j < V; ++j) h[j] = need ? sm.carry[lc + j] : 0.f;
        for (int w = 0; w < wid; ++w)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 m = sm.agg[w][lc + j];
                h[j] = (cuts >> (8 * w)) & 0xff ? m.y : fmaf(m.x, h[j], m.y);
            }
#pragma unroll
        for (int r = 0; r < LR_ROWS; ++r) {
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = (heads >> r) & 1 ? b[r][j] : fmaf(a[r][j], h[j], b[r][j]);
            if (on && row0 + r < p.rows) {
                if (p.h) store_pack<T, V>(reinterpret_cast<T *>(p.h) + (int64_t)(row0 + r) * p.dim + c, h);
                if (p.ht && (tails >> r) & 1)
                    store_pack<float, V>(p.ht + (int64_t)sm.seq[wid * LR_ROWS + r] * p.dim + c, h);
            }
        }
        bad |= empty_sequences<CB>(p, i, p.tiles, cb, p.h0, p.ht);
        if (p.walk) {
            __syncthreads();  // everybody has read carry, agg and the rows' sequences
            if (threadIdx.x < CB) sm.carry[threadIdx.x] = mine.of(i > 0 ? sm.carry[threadIdx.x] : 0.f);
        }
        ++i;
    } while (p.walk && i < p.tiles);
    if (p.cu || p.walk) note_faults<CB>(p, cb, bad);
}

// ---------------------------------------------------------------- backward
template <typename T, typename G, int V, bool COMP>
__global__ void __launch_bounds__(LR_THREADS, 2) k10_bwd(const LinrecParams p) {
    constexpr int CB = block_channels<V>();
    __shared__ ScanSmem<CB> sm;
    __shared__ float2 fwd[LR_WARPS][CB];  // the warps' forward maps
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, lc = lane * V;
    int i = 0, cb = blockIdx.x;
    if (!p.walk) {
        if (threadIdx.x == 0) sm.ticket = atomicAdd(p.ticket, 1);
        __syncthreads();
        i = p.blocks.div(sm.ticket);
        cb = sm.ticket - i * p.nblk;
    }
    const int c = cb * CB + lc;
    const bool on = c < p.dim;
    bool bad = false;
    do {
        const int tile = p.tiles - 1 - i, row0 = tile * LR_TILE + wid * LR_ROWS;
        float a[LR_ROWS][V], rest[LR_ROWS][V], x[LR_ROWS][V], d[LR_ROWS][V];
#pragma unroll
        for (int r = 0; r < LR_ROWS; ++r) {
            const bool live = on && row0 + r < p.rows;
            load_row<G, V>(p.g, (int64_t)(row0 + r) * p.g_ts + c, live, a[r]);
            load_row<T, V>(p.x, (int64_t)(row0 + r) * p.x_ts + c, live, x[r]);
            load_row<T, V>(p.dh, (int64_t)(row0 + r) * p.dh_ts + c, live, d[r]);
        }
        find_sequences<CB>(p, sm, tile * LR_TILE);
        __syncthreads();
        const uint32_t heads = sm.head[wid >> 2] >> (8 * (wid & 3)) & 0xff;
        const uint32_t tails = sm.tail[wid >> 2] >> (8 * (wid & 3)) & 0xff;
        const uint64_t hcuts = sm.head[0] | (uint64_t)sm.head[1] << 32;
        const uint64_t tcuts = sm.tail[0] | (uint64_t)sm.tail[1] << 32;
        float A[V], B[V];
#pragma unroll
        for (int j = 0; j < V; ++j) A[j] = 1.f, B[j] = 0.f;
#pragma unroll
        for (int r = 0; r < LR_ROWS; ++r) {
            const bool head = (heads >> r) & 1;
            float first[V];
            if (head) load_f32<V>(p.h0, (int64_t)sm.seq[wid * LR_ROWS + r] * p.dim + c, on, first);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                decay(a[r][j], a[r][j], rest[r][j]);
                const float b = COMP ? rest[r][j] * x[r][j] : x[r][j];
                B[j] = fmaf(a[r][j], head ? first[j] : B[j], b);
                A[j] *= a[r][j];
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) fwd[wid][lc + j] = make_float2(A[j], B[j]), B[j] = 0.f;
#pragma unroll
        for (int r = LR_ROWS - 1; r >= 0; --r) {
            const bool tail = (tails >> r) & 1;
            float after[V];
            if (tail) load_f32<V>(p.dht, (int64_t)sm.seq[wid * LR_ROWS + r] * p.dim + c, on, after);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                if (tail) d[r][j] += after[j], B[j] = a[r][j] * d[r][j];
                else B[j] = a[r][j] * (d[r][j] + B[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) sm.agg[wid][lc + j] = make_float2(A[j], B[j]);
        float h[V];
        if (hcuts & 1)
#pragma unroll
            for (int j = 0; j < V; ++j) h[j] = 0.f;
        else load_f32<V>(p.states, (int64_t)tile * p.dim + c, on, h);
        __syncthreads();
        const bool need = tile + 1 < p.tiles && !(tcuts >> 63), last = tile == 0;
        Map mine;
        if (threadIdx.x < CB)
#pragma unroll
            for (int w = LR_WARPS - 1; w >= 0; --w) {
                const float2 m = sm.agg[w][threadIdx.x];
                mine.then(m.x, m.y, (tcuts >> (8 * w)) & 0xff);
            }
        if (!p.walk) Tree<CB>(p, sm, i, cb).enter(mine, tcuts != 0, need, last);
        for (int w = 0; w < wid; ++w)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 m = fwd[w][lc + j];
                h[j] = (hcuts >> (8 * w)) & 0xff ? m.y : fmaf(m.x, h[j], m.y);
            }
        float before[LR_ROWS][V];  // h_{t-1}, less x_t with COMP
#pragma unroll
        for (int r = 0; r < LR_ROWS; ++r) {
            if ((heads >> r) & 1) load_f32<V>(p.h0, (int64_t)sm.seq[wid * LR_ROWS + r] * p.dim + c, on, h);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                before[r][j] = COMP ? h[j] - x[r][j] : h[j];
                h[j] = fmaf(a[r][j], h[j], COMP ? rest[r][j] * x[r][j] : x[r][j]);
            }
        }
        float m[V];
#pragma unroll
        for (int j = 0; j < V; ++j) m[j] = need ? sm.carry[lc + j] : 0.f;
        for (int w = LR_WARPS - 1; w > wid; --w)
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float2 q = sm.agg[w][lc + j];
                m[j] = (tcuts >> (8 * w)) & 0xff ? q.y : fmaf(q.x, m[j], q.y);
            }
#pragma unroll
        for (int r = LR_ROWS - 1; r >= 0; --r) {
            float dx[V], dg[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float lam = (tails >> r) & 1 ? d[r][j] : d[r][j] + m[j];
                m[j] = a[r][j] * lam;
                dx[j] = COMP ? rest[r][j] * lam : lam;
                dg[j] = m[j] * before[r][j];
            }
            if (on && row0 + r < p.rows) {
                const int64_t o = (int64_t)(row0 + r) * p.dim + c;
                store_pack<T, V>(reinterpret_cast<T *>(p.dx) + o, dx);
                store_pack<G, V>(reinterpret_cast<G *>(p.dg) + o, dg);
                if (p.dh0 && (heads >> r) & 1)
                    store_pack<float, V>(p.dh0 + (int64_t)sm.seq[wid * LR_ROWS + r] * p.dim + c, m);
            }
        }
        bad |= empty_sequences<CB>(p, i, p.tiles, cb, p.dht, p.dh0);
        if (p.walk) {
            __syncthreads();
            if (threadIdx.x < CB) sm.carry[threadIdx.x] = mine.of(i > 0 ? sm.carry[threadIdx.x] : 0.f);
        }
        ++i;
    } while (p.walk && i < p.tiles);
    if (p.cu || p.walk) note_faults<CB>(p, cb, bad);
}

// ---------------------------------------------------------------- single tokens
template <typename T, typename G, int V, bool COMP> __global__ void __launch_bounds__(128) k10_step(const StepParams p) {
    const int per = p.pieces.d;  // pieces of V channels in a row
    const int64_t e = (int64_t)blockIdx.x * 128 + threadIdx.x;
    if (e >= p.batch * per) return;
    const uint32_t i = p.pieces.div((uint32_t)e);
    const int c = ((uint32_t)e - i * per) * V;
    const int64_t slot = p.slots ? p.slots[i] : i;
    float y[V] = {}, g[V], x[V], h[V];
    load_row<G, V>(p.g, (int64_t)i * p.g_ts + c, true, g);
    load_row<T, V>(p.x, (int64_t)i * p.x_ts + c, true, x);
    if (slot >= 0 && slot < p.num_slots) {
        float *at = p.state + slot * p.dim + c;
        load_row<float, V>(at, 0, true, h);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            float a, rest;
            decay(g[j], a, rest);
            y[j] = fmaf(a, h[j], COMP ? rest * x[j] : x[j]);
        }
        store_pack<float, V>(at, y);
    }
    store_pack<T, V>(reinterpret_cast<T *>(p.y) + (int64_t)i * p.dim + c, y);
}

}  // namespace

constexpr int LR_FWD_V = 4, LR_BWD_V = 2;  // channels per thread where rows can be moved in pieces

template <typename T, typename G> cudaError_t linrec_fwd_t(LinrecParams &p, cudaStream_t stream) {
#define RUN(V, COMP)                                                             \
    do {                                                                         \
        const cudaError_t e = linrec_blocks(p, block_channels<V>(), stream);     \
        if (e != cudaSuccess) return e;                                          \
        k10_fwd<T, G, V, COMP><<<p.grid, LR_THREADS, 0, stream>>>(p);            \
    } while (0)
    if (p.vec) {
        if (p.complement) RUN(LR_FWD_V, true);
        else RUN(LR_FWD_V, false);
    } else {
        if (p.complement) RUN(1, true);
        else RUN(1, false);
    }
#undef RUN
    return cudaGetLastError();
}

template <typename T, typename G> cudaError_t linrec_bwd_t(LinrecParams &p, cudaStream_t stream) {
#define RUN(V, COMP)                                                             \
    do {                                                                         \
        const cudaError_t e = linrec_blocks(p, block_channels<V>(), stream);     \
        if (e != cudaSuccess) return e;                                          \
        k10_bwd<T, G, V, COMP><<<p.grid, LR_THREADS, 0, stream>>>(p);            \
    } while (0)
    if (p.vec) {
        if (p.complement) RUN(LR_BWD_V, true);
        else RUN(LR_BWD_V, false);
    } else {
        if (p.complement) RUN(1, true);
        else RUN(1, false);
    }
#undef RUN
    return cudaGetLastError();
}

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
