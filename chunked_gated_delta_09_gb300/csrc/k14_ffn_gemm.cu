// k14_ffn_gemm.cu -- the matrix products of the gated feed-forward on the 5th-generation tensor cores.
//
//     FFN_FWD  [g u] = x [Wg; Wu]^T      both operands along their contiguous axis; h = act(g) u as the tile leaves
//     FFN_DX   dx    = dg Wg + du Wu     [dg du] along its contiguous axis, the weights across theirs
//     FFN_DW   dWg   = dg^T x , dWu = du^T x   both operands across their contiguous axis
//
// Two CTAs of a cluster (PAIR) work on 256 x 256 results, each with half of the rows and half of the columns' operand in
// its shared memory, and one of them issues the tcgen05 products of both; single CTAs work on 128 x 256.  One thread
// fetches 64 of the summed axis of both operands at a time by tensor maps (128-byte swizzle, several stages deep), products
// go to one half of tensor memory, and four warps take the other half's finished tile to its place.  In a forward tile 128
// columns are gates and 128 the values that they multiply.  The summed axis of products with few tiles is cut in parts whose
// fp32 results another kernel adds in order.
#include "ffn.h"
#include "ffn_act.cuh"
#include "tc_util.cuh"

#include <type_traits>
#include <utility>

namespace gdr {
namespace {

constexpr int GEMM_THREADS = 192, STORE_WARPS = 4;
// Bytes of a stage: 128 rows of one operand; 256 columns of the other, or half of them for each of a pair.
constexpr int A_BYTES = 128 * FFN_BK * 2;
constexpr int b_bytes(bool pair) { return (pair ? FFN_BN / 2 : FFN_BN) * FFN_BK * 2; }
constexpr int stages(bool pair) { return pair ? 6 : 4; }
constexpr int STAGE_ROW = 33;  // words of a row that waits to be stored element by element
constexpr int gemm_smem(bool pair) {
    return stages(pair) * (A_BYTES + b_bytes(pair)) + STORE_WARPS * 32 * STAGE_ROW * 4 + 1024;
}

// A fetch into this CTA's shared memory, counted at the barrier with shared::cluster address `bar` (a pair: the first CTA's).
template <bool PAIR> __device__ __forceinline__ void fetch(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    if constexpr (PAIR)
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
                smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];\n" ::"r"(
                smem_u32(dst)),
            "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];\n" ::"r"(smem_u32(bar)) : "memory");
}

// ---- pairs of CTAs
__device__ __forceinline__ uint32_t pair_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void pair_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;\n" ::: "memory");
}
// Where the first CTA has what this one has at p.
__device__ __forceinline__ uint32_t in_first(const void *p) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(smem_u32(p)));
    return a;
}
__device__ __forceinline__ void mbar_arrive_first(uint64_t *bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(in_first(bar)) : "memory");
}
// As tc::mbar_wait, for barriers at which the other CTA arrives.
__device__ __forceinline__ bool mbar_wait_pair(uint64_t *bar, uint32_t parity, uint32_t limit) {
    uint32_t done = 0;
    for (uint32_t it = 0; it < limit; ++it) {
        if (limit < (1u << 16))
            asm volatile(
                "{\n.reg .pred p;\nmbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(done)
                : "r"(smem_u32(bar)), "r"(parity)
                : "memory");
        else
            asm volatile(
                "{\n.reg .pred p;\nmbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\nselp.u32 %0, 1, 0, p;\n}\n"
                : "=r"(done)
                : "r"(smem_u32(bar)), "r"(parity)
                : "memory");
        if (done) return true;
    }
    return false;
}
template <bool PAIR> __device__ __forceinline__ void issue(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    if constexpr (PAIR)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.b32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(accumulate));
    else
        tc::mma(d, a, b, idesc, accumulate);
}
// Arrives at the barrier, of both CTAs of a pair, once all products issued so far are done.
template <bool PAIR> __device__ __forceinline__ void commit_all(uint64_t *bar) {
    if constexpr (PAIR)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(
                         smem_u32(bar)),
                     "h"((uint16_t)3)
                     : "memory");
    else
        tc::commit(bar);
}
template <bool PAIR> __device__ __forceinline__ void alloc_all(uint32_t *slot) {
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n");
    } else {
        tc::tmem_alloc(slot, 512);
    }
}
template <bool PAIR> __device__ __forceinline__ void free_all(uint32_t tmem) {
    if constexpr (PAIR)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem));
    else
        tc::tmem_dealloc(tmem, 512);
}

// Descriptors of operand tiles with the 128-byte swizzle.  Along the contiguous axis (K-major) a tile is rows of 128 bytes,
// 8 of them 1024 bytes; across it (MN-major) blocks of 64 operand rows x 64 of the summed axis, 8192 bytes each, in
// which 8 of the summed axis take 1024 bytes.  16 of the summed axis are 32 or 2048 bytes on.
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr, bool mn) {
    uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFF);
    d |= (uint64_t)((mn ? 8192 : 16) >> 4) << 16;
    d |= (uint64_t)(1024 >> 4) << 32;
    d |= (uint64_t)1 << 46;
    d |= (uint64_t)2 << 61;
    return d;
}

struct Unit {
    int job, m, n, kb0, kb1;  // tile, pieces of the summed axis
    int part;                 // which partial result it is, or -1: the whole of a tile
};
__device__ __forceinline__ void tile_of(const FfnPlan &p, int t, int &m, int &n) {
    const int per = p.group * p.nt, group = t / per;
    t -= group * per;
    const int first = group * p.group, size = min(p.mt - first, p.group);
    n = t / size;
    m = first + t - n * size;
}
// A CTA's (a pair's) units: those of the first job round after round; of the second, `extra` rounds for the CTAs that had a
// unit of the first job's last round, and the rest for the others.
struct Walk {
    const FfnGemm &p;
    int c, all, u1, u2, r;
    __device__ __forceinline__ Walk(const FfnGemm &p_, bool pair) : p(p_) {
        c = pair ? blockIdx.x / 2 : blockIdx.x, all = pair ? gridDim.x / 2 : gridDim.x;
        u1 = p.job[0].plan.units(), u2 = p.job[1].plan.units(), r = u1 % all;
    }
    __device__ __forceinline__ bool unit(int i, Unit &u) const {
        const int n1 = c < u1 ? (u1 - c + all - 1) / all : 0;
        int n = c + i * all;
        u.job = i >= n1;
        if (u.job) {
            i -= n1;
            if (c < r && i >= p.extra) return false;
            n = c < r ? c + r * i : r * p.extra + (c - r) + (all - r) * i;
            if (n >= u2) return false;
        }
        const FfnJob &job = p.job[u.job];
        const FfnPlan &plan = job.plan;
        u.kb0 = 0, u.kb1 = plan.kb, u.part = -1;
        if (n >= plan.whole) {
            const int cut = plan.mt * plan.nt - plan.whole, split = (n - plan.whole) / cut;
            u.part = job.first_part + n - plan.whole;
            n -= split * cut;
            u.kb0 = (int)((int64_t)plan.kb * split / plan.splits);
            u.kb1 = (int)((int64_t)plan.kb * (split + 1) / plan.splits);
        }
        tile_of(plan, n, u.m, u.n);
        return true;
    }
};

// 32 rows of 32 values, a row for each lane, to 32 rows `stride` apart, of which the first `rows` and the first n columns are
// inside the result.  `piece`: bytes that the rows can be stored in at a time; below 16 the rows go through `wait`, one
// of them at a time, so that what a store writes lies together.
template <typename T> __device__ __forceinline__ void store_block(T *to, int64_t stride, const float (&v)[32], int rows, int n, int piece, float *wait) {
    const int lane = threadIdx.x & 31;
    if (piece >= 16) {
        if (lane < rows) store_row32(to + lane * stride, v, n, piece);
        return;
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 32; ++i) wait[lane * STAGE_ROW + i] = v[i];
    __syncwarp();
    if (lane >= n) return;
    T *q = to + lane;
    if (rows == 32) {
#pragma unroll
        for (int r = 0; r < 32; ++r, q += stride) *q = to_out_t<T>(wait[r * STAGE_ROW + lane]);
    } else {
        for (int r = 0; r < rows; ++r, q += stride) *q = to_out_t<T>(wait[r * STAGE_ROW + lane]);
    }
}

template <bool FWD, int ACT, bool PAIR, typename T>
__device__ __forceinline__ void store_tile(const FfnGemm &p, const Unit &u, uint32_t rank, uint32_t tmem, float *wait) {
    const FfnJob &job = p.job[FWD ? 0 : u.job];
    const int quarter = (threadIdx.x >> 5) & 3;
    const int half_tiles = job.plan.mt / 2;  // FFN_DW: the rows of dWg, then those of dWu
    const int which = !FWD && job.what == FFN_DW && u.m >= half_tiles;
    const int64_t row = (int64_t)(u.m - which * half_tiles) * (PAIR ? 256 : 128) + rank * 128 + quarter * 32;  // the warp's first
    const int rows = (int)max((int64_t)0, min((int64_t)32, job.rows - row));
    // partial results: 256 columns of every row of a tile, one tile after the other
    float *part = p.part + (((int64_t)u.part * (PAIR ? 2 : 1) + rank) * 128 + quarter * 32 + (threadIdx.x & 31)) * FFN_BN;
    const uint32_t t0 = tmem + ((uint32_t)quarter * 32u << 16);
    if constexpr (FWD) {
        const int64_t col0 = (int64_t)u.n * (FFN_BN / 2);
        for (int c = 0; c < FFN_BN / 2; c += 32) {
            if (col0 + c >= job.cols) break;
            float g[32], v[32];
            tc::ld32(t0 + c, g);
            tc::ld32(t0 + FFN_BN / 2 + c, v);
            const int n = (int)min((int64_t)32, job.cols - col0 - c);
            if (u.part >= 0) {
                store_part32(part + c, g), store_part32(part + FFN_BN / 2 + c, v);
                continue;
            }
            const int64_t at = row * job.cols + col0 + c;
            if (p.gate) {
                store_block(p.gate + at, job.cols, g, rows, n, p.piece32, wait);
                store_block(p.up + at, job.cols, v, rows, n, p.piece32, wait);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= activate<ACT>(g[i]);
            if (job.out[0]) store_block(static_cast<T *>(job.out[0]) + at, job.cols, v, rows, n, job.piece, wait);
        }
    } else {
        const int64_t col0 = (int64_t)u.n * FFN_BN;
        T *out = static_cast<T *>(which ? job.out[1] : job.out[0]) + row * job.cols + col0;
        for (int c = 0; c < FFN_BN; c += 32) {
            if (col0 + c >= job.cols) break;
            float v[32];
            tc::ld32(t0 + c, v);
            if (u.part >= 0) store_part32(part + c, v);
            else store_block(out + c, job.cols, v, rows, (int)min((int64_t)32, job.cols - col0 - c), job.piece, wait);
        }
    }
}

// ---- a unit's fetches, and its products, by one thread each; false where a wait ran out.  The product is known to the compiler: both
// loops are on the way of every 64 of the summed axis (8192 x 2048 x 8192, dx: 317 us so, 348 with the choices inside).
template <int WHAT, bool PAIR>
__device__ __forceinline__ bool produce(const FfnPlan &plan, const Unit &u, const CUtensorMap *map_a, const CUtensorMap *map_b, uint32_t rank,
                                        unsigned char *tiles, uint64_t *full, uint64_t *empty, uint32_t &it, uint32_t spin) {
    constexpr int STAGES = stages(PAIR), B_BYTES = b_bytes(PAIR), STAGE_BYTES = A_BYTES + B_BYTES;
    const int k_half = WHAT == FFN_DX ? plan.kb / 2 : plan.kb, m_half = WHAT == FFN_DW ? plan.mt / 2 : plan.mt;
    const int which_m = WHAT == FFN_DW && u.m >= m_half;
    const int m = (u.m - which_m * m_half) * (PAIR ? 256 : 128) + (int)rank * 128;
    const int col = WHAT == FFN_FWD ? u.n * (FFN_BN / 2) : u.n * FFN_BN + (int)rank * 128;
    for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
        const uint32_t s = it % STAGES, round = it / STAGES;
        if (round > 0 && !tc::mbar_wait(&empty[s], (round - 1) & 1, spin)) return false;
        unsigned char *a = tiles + s * STAGE_BYTES, *b = a + A_BYTES;
        const uint32_t bar = PAIR ? in_first(&full[s]) : smem_u32(&full[s]);
        if (rank == 0) tc::mbar_expect_tx(&full[s], (PAIR ? 2 : 1) * STAGE_BYTES);
        const int which_k = WHAT == FFN_DX && kb >= k_half, k = (kb - which_k * k_half) * FFN_BK;
        if constexpr (WHAT == FFN_DW) {
            for (int j = 0; j < 2; ++j) fetch<PAIR>(a + j * 8192, map_a + which_m, m + j * 64, k, bar);
        } else {
            fetch<PAIR>(a, map_a + which_k, k, m, bar);
        }
        if constexpr (WHAT == FFN_FWD) {
            fetch<PAIR>(b, map_b + rank, k, col, bar);  // a pair: gates' rows here, values' rows there
            if (!PAIR) fetch<PAIR>(b + B_BYTES / 2, map_b + 1, k, col, bar);
        } else {
            for (int j = 0; j < B_BYTES / 8192; ++j) fetch<PAIR>(b + j * 8192, map_b + which_k, col + j * 64, k, bar);
        }
    }
    return true;
}
template <int WHAT, bool PAIR>
__device__ __forceinline__ bool multiply(const Unit &u, uint32_t d, unsigned char *tiles, uint64_t *full, uint64_t *empty, uint32_t &it, bool bf16,
                                         uint32_t spin) {
    constexpr int STAGES = stages(PAIR), STAGE_BYTES = A_BYTES + b_bytes(PAIR);
    constexpr bool a_mn = WHAT == FFN_DW, b_mn = WHAT != FFN_FWD;
    // (the types' field: 1 for bf16)
    const uint32_t id = tc::idesc_f16(PAIR ? 256 : 128, FFN_BN, a_mn, b_mn) | (bf16 ? (1u << 7) | (1u << 10) : 0u);
    for (int kb = u.kb0; kb < u.kb1; ++kb, ++it) {
        const uint32_t s = it % STAGES;
        if (!tc::mbar_wait(&full[s], (it / STAGES) & 1, spin)) return false;
        tc::fence_after();
        const uint32_t a = smem_u32(tiles + s * STAGE_BYTES);
        const uint64_t da = desc_sw128(a, a_mn), db = desc_sw128(a + A_BYTES, b_mn);
#pragma unroll
        for (int k = 0; k < FFN_BK / 16; ++k)
            issue<PAIR>(d, da + k * ((a_mn ? 2048 : 32) >> 4), db + k * ((b_mn ? 2048 : 32) >> 4), id, kb > u.kb0 || k > 0);
        commit_all<PAIR>(&empty[s]);
    }
    return true;
}

template <bool FWD, int ACT, bool PAIR, typename T>
__global__ void __launch_bounds__(GEMM_THREADS, 1) k14_gemm(const __grid_constant__ FfnMaps maps, const FfnGemm p) {
    constexpr int STAGES = stages(PAIR), B_BYTES = b_bytes(PAIR), STAGE_BYTES = A_BYTES + B_BYTES;
    extern __shared__ unsigned char raw[];
    unsigned char *tiles = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    // full: a stage's fetches have landed (a pair: those of both, at the first CTA's barrier); empty, done: products are done
    // with a stage, with a half of tensor memory; taken: that half has been read
    __shared__ uint64_t full[STAGES], empty[STAGES], done[2], taken[2], last;
    __shared__ uint32_t slot, fetched[2];  // stages that each CTA has fetched in all
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = PAIR ? pair_rank() : 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) tc::mbar_init(&full[s], 1), tc::mbar_init(&empty[s], 1);
        for (int b = 0; b < 2; ++b) tc::mbar_init(&done[b], 1), tc::mbar_init(&taken[b], STORE_WARPS * (PAIR ? 2 : 1));
        tc::mbar_init(&last, 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    }
    if (warp == 1) alloc_all<PAIR>(&slot);
    tc::fence_before();
    __syncthreads();
    if (PAIR) pair_sync();
    tc::fence_after();
    const uint32_t tmem = slot;
    const Walk walk(p, PAIR);
    Unit u;
    bool lost = false;

    if (warp == 0 && lane == 0) {
        uint32_t it = 0;
        for (int n = 0; walk.unit(n, u) && !lost; ++n) {
            const FfnJob &job = p.job[u.job];
            if constexpr (FWD)
                lost = !produce<FFN_FWD, PAIR>(job.plan, u, maps.a[0], maps.b[0], rank, tiles, full, empty, it, p.spin);
            else if (job.what == FFN_DX)
                lost = !produce<FFN_DX, PAIR>(job.plan, u, maps.a[u.job], maps.b[u.job], rank, tiles, full, empty, it, p.spin);
            else
                lost = !produce<FFN_DW, PAIR>(job.plan, u, maps.a[u.job], maps.b[u.job], rank, tiles, full, empty, it, p.spin);
        }
        // (both CTAs' counts where the first reads them)
        if (PAIR) asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(in_first(&fetched[rank])), "r"(it) : "memory");
        else fetched[0] = fetched[1] = it;
    } else if (warp == 1 && lane == 0 && rank == 0) {
        uint32_t it = 0, count = 0;
        for (; walk.unit((int)count, u) && !lost; ++count) {
            const uint32_t buf = count & 1, use = count >> 1;
            if (use > 0 && !mbar_wait_pair(&taken[buf], (use - 1) & 1, p.spin)) {
                lost = true;
                break;
            }
            tc::fence_after();
            const uint32_t d = tmem + buf * FFN_BN, bf16 = p.dtype == BF16;
            if constexpr (FWD) lost = !multiply<FFN_FWD, PAIR>(u, d, tiles, full, empty, it, bf16, p.spin);
            else if (p.job[u.job].what == FFN_DX) lost = !multiply<FFN_DX, PAIR>(u, d, tiles, full, empty, it, bf16, p.spin);
            else lost = !multiply<FFN_DW, PAIR>(u, d, tiles, full, empty, it, bf16, p.spin);
            if (!lost) commit_all<PAIR>(&done[buf]);
        }
        commit_all<PAIR>(&last);  // nothing may be read or written by a product after this
        tc::mbar_wait(&last, 0, DRAIN_LIMIT);
    } else if (warp == 1 && lane == 0) {
        tc::mbar_wait(&last, 0, DRAIN_LIMIT);
    } else if (warp >= 2) {
        float *wait = reinterpret_cast<float *>(tiles + STAGES * STAGE_BYTES) + (warp - 2) * 32 * STAGE_ROW;
        for (uint32_t count = 0; walk.unit((int)count, u); ++count) {
            const uint32_t buf = count & 1, use = count >> 1;
            // (the warp goes on together or not at all: it reads tensor memory as one)
            if (!__all_sync(0xffffffffu, tc::mbar_wait(&done[buf], use & 1, p.spin))) {
                lost = true;
                break;
            }
            tc::fence_after();
            store_tile<FWD, ACT, PAIR, T>(p, u, rank, tmem + buf * FFN_BN, wait);
            tc::fence_before();
            __syncwarp();
            if (lane == 0) {
                if (PAIR) mbar_arrive_first(&taken[buf]);
                else mbar_arrive(&taken[buf]);
            }
        }
    }
    __syncwarp();
    const int any = __syncthreads_or(lost);
    if (threadIdx.x == 0 && p.status) {
        p.status[blockIdx.x] = (uint8_t)(any || (!p.clear && p.status[blockIdx.x]));
        if (p.clear)  // (those of CTAs that an earlier call had more of)
            for (uint32_t i = blockIdx.x + gridDim.x; i < GDR_FFN_STATUS_BYTES; i += gridDim.x) p.status[i] = 0;
    }
    __syncwarp();
    if (PAIR) pair_sync();
    if (threadIdx.x == 0 && rank == 0) {
        // Nothing may land in shared memory after this.  Where waits ran out, one CTA of a pair may have fetched stages that the
        // other has not: those are made to expect what comes, and no more.
        const uint32_t mine = fetched[0], other = fetched[1], both = min(mine, other), most = max(mine, other);
        if (PAIR)
            for (uint32_t i = both; i < most; ++i) {
                if (i < mine)
                    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full[i % STAGES])), "r"(STAGE_BYTES) : "memory");
                else
                    tc::mbar_expect_tx(&full[i % STAGES], STAGE_BYTES);
            }
        for (uint32_t s = 0; s < STAGES && s < most; ++s)
            tc::mbar_wait(&full[s], ((most - s + STAGES - 1) / STAGES - 1) & 1, DRAIN_LIMIT);
    }
    if (PAIR) {
        __syncwarp();
        pair_sync();
    } else {
        __syncthreads();
    }
    if (warp == 1) free_all<PAIR>(tmem);
}

template <bool FWD, int ACT, bool PAIR, typename T> cudaError_t gemm_t(const FfnMaps &maps, const FfnGemm &p, cudaStream_t stream) {
    int sms = 0;
    cudaError_t e = device_sm_count(&sms);
    if (e == cudaSuccess) e = smem_opt_in((const void *)k14_gemm<FWD, ACT, PAIR, T>, gemm_smem(PAIR));
    if (e != cudaSuccess) return e;
    const int units = p.job[0].plan.units() + p.job[1].plan.units(), ctas = PAIR ? 2 : 1;
    const int most = min(sms, GDR_FFN_STATUS_BYTES) / ctas;  // (a byte of the status for each)
    ClusterLaunch l((units < most ? units : most) * ctas, GEMM_THREADS, gemm_smem(PAIR), ctas, stream);
    return cudaLaunchKernelEx(&l.cfg, k14_gemm<FWD, ACT, PAIR, T>, maps, p);
}

// ---------------------------------------------------------------- partial results added in order
constexpr int JOIN_THREADS = 256;

// A thread has 8 columns of a row of a tile that was cut (forward: 8 gates and the values beside them).
template <bool FWD, int ACT, typename T> __global__ void __launch_bounds__(JOIN_THREADS) k14_join(const FfnGemm p) {
    constexpr int HALVES = FWD ? 2 : 1, PER_ROW = FFN_BN / HALVES / 8;
    const int cut0 = p.job[0].plan.cut(), second = (int)blockIdx.y >= cut0, tile = blockIdx.y - second * cut0;
    const FfnJob &job = p.job[second];
    const int tile_rows = job.plan.pair ? 256 : 128, cut = job.plan.cut();
    const int in_tile = blockIdx.x * JOIN_THREADS + threadIdx.x, local = in_tile / PER_ROW, c = in_tile % PER_ROW * 8;
    int m, n;
    tile_of(job.plan, job.plan.whole + tile, m, n);
    const int half_tiles = job.plan.mt / 2;
    const bool which = !FWD && job.what == FFN_DW && m >= half_tiles;
    const int64_t row = (int64_t)(m - which * half_tiles) * tile_rows + local, col = (int64_t)n * (FFN_BN / HALVES) + c;
    if (row >= job.rows || col >= job.cols) return;
    float v[HALVES][8] = {};
    for (int s = 0; s < job.plan.splits; ++s)
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
            const float4 *q = reinterpret_cast<const float4 *>(
                p.part + ((job.first_part + (int64_t)s * cut + tile) * tile_rows + local) * FFN_BN + h * (FFN_BN / 2) + c);
            const float4 a = q[0], b = q[1];
            v[h][0] += a.x, v[h][1] += a.y, v[h][2] += a.z, v[h][3] += a.w;
            v[h][4] += b.x, v[h][5] += b.y, v[h][6] += b.z, v[h][7] += b.w;
        }
    const int count = (int)min((int64_t)8, job.cols - col);
    auto store = [&](auto *to, const float (&x)[8], int piece) {
        using To = std::remove_reference_t<decltype(*to)>;
        To *q = to + row * job.cols + col;
        if (piece >= 16 && count == 8) {
            store_pack<To, 8>(q, x);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j < count) q[j] = to_out_t<To>(x[j]);
        }
    };
    if constexpr (FWD) {
        if (p.gate) store(p.gate, v[0], p.piece32), store(p.up, v[1], p.piece32);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[1][j] *= activate<ACT>(v[0][j]);
        if (job.out[0]) store(static_cast<T *>(job.out[0]), v[1], job.piece);
    } else {
        store(static_cast<T *>(which ? job.out[1] : job.out[0]), v[0], job.piece);
    }
}

template <bool FWD, int ACT, typename T> cudaError_t product_t(const FfnMaps &maps, const FfnGemm &p, cudaStream_t stream) {
    const bool pair = p.job[0].plan.pair;
    const cudaError_t e = pair ? gemm_t<FWD, ACT, true, T>(maps, p, stream) : gemm_t<FWD, ACT, false, T>(maps, p, stream);
    const int cut = p.job[0].plan.cut() + p.job[1].plan.cut();
    if (e != cudaSuccess || cut == 0) return e;
    const unsigned threads = (pair ? 256u : 128u) * FFN_BN / (FWD ? 2 : 1) / 8;
    k14_join<FWD, ACT, T><<<dim3(threads / JOIN_THREADS, (unsigned)cut), JOIN_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}
template <typename T> cudaError_t product_of(const FfnMaps &maps, const FfnGemm &p, cudaStream_t stream) {
    if (p.job[0].what != FFN_FWD) return product_t<false, 0, T>(maps, p, stream);
    if (p.act == FFN_SILU) return product_t<true, FFN_SILU, T>(maps, p, stream);
    if (p.act == FFN_SIGMOID) return product_t<true, FFN_SIGMOID, T>(maps, p, stream);
    return product_t<true, FFN_GELU_TANH, T>(maps, p, stream);
}

// ---------------------------------------------------------------- plans
// Estimates in hundredths of a us: a unit's 64 of the summed axis 0.37 us (under load; single CTAs, whose operands take half as
// much shared-memory bandwidth again, 0.40: 8192 x 2048 x 8192 forward 345 against 330 us, dx 402 against 368) or its results'
// way out 2 us; 3 us to begin and end, pairs 3.5; parts are added by another kernel, 5 us and their bytes at 5 TB/s.
constexpr int64_t SHORTEST = 200;

int cut_in(int64_t n, int64_t by) { return (int)((n + by - 1) / by); }

FfnPlan plan_of(FfnProduct what, bool pair, int64_t tokens, int64_t dim, int64_t inner) {
    const int bm = pair ? 256 : 128;
    FfnPlan p = {};
    p.pair = pair, p.splits = 1, p.group = what == FFN_FWD ? 16 : 4;
    if (what == FFN_FWD) p.mt = cut_in(tokens, bm), p.nt = cut_in(inner, FFN_BN / 2), p.kb = cut_in(dim, FFN_BK);
    else if (what == FFN_DX) p.mt = cut_in(tokens, bm), p.nt = cut_in(dim, FFN_BN), p.kb = 2 * cut_in(inner, FFN_BK);
    else p.mt = 2 * cut_in(inner, bm), p.nt = cut_in(dim, FFN_BN), p.kb = cut_in(tokens, FFN_BK);
    p.whole = p.mt * p.nt;
    return p;
}
int64_t unit_time(const FfnPlan &p, int splits) {
    const int64_t t = (int64_t)((p.kb + splits - 1) / splits) * (p.pair ? 37 : 40);
    return t > SHORTEST ? t : SHORTEST;
}
int64_t ends_time(bool pair, int64_t parts) {
    return (pair ? 350 : 300) + (parts ? 500 + parts * (pair ? 256 : 128) * FFN_BN * 8 / 50000 : 0);
}

// The time of u1 units of t1 and then u2 of t2 on `slots`, and the second job's rounds for who had one more of the first.
int64_t two_jobs(int64_t u1, int64_t t1, int64_t u2, int64_t t2, int64_t slots, int &extra) {
    const int64_t all = u1 + u2 < slots ? u1 + u2 : slots, q = u1 / all, r = u1 % all;
    extra = 0;
    if (u2 == 0) return (q + (r > 0)) * t1;
    int64_t best = INT64_MAX;
    for (const int64_t less : {t1 / t2, (t1 + t2 - 1) / t2}) {
        int64_t w2 = (u2 + r * less + all - 1) / all, w1 = w2 - less;
        if (r == 0 || w1 < 0) w1 = 0, w2 = (u2 + all - r - 1) / (all - r);
        const int64_t first = r ? (q + 1) * t1 + w1 * t2 : 0, rest = q * t1 + w2 * t2, t = first > rest ? first : rest;
        if (t < best) best = t, extra = (int)w1;
    }
    return best;
}

}  // namespace

cudaError_t launch_ffn_product(const FfnMaps &maps, const FfnGemm &p, cudaStream_t stream) {
    return p.dtype == BF16 ? product_of<__nv_bfloat16>(maps, p, stream) : product_of<__half>(maps, p, stream);
}

// The quickest by the estimate.  What is cut: nothing, all tiles, or those of a last round that is half full at most; in four
// pieces of the summed axis at least, and only in parts that fit one round.
FfnPlan ffn_plan_one(FfnProduct what, int64_t tokens, int64_t dim, int64_t inner, int64_t &least) {
    FfnPlan best = {};
    least = INT64_MAX;
    for (const bool pair : {true, false}) {
        const FfnPlan p = plan_of(what, pair, tokens, dim, inner);
        const int64_t tiles = p.whole, slots = pair ? 76 : 152, all = unit_time(p, 1);
        auto consider = [&](int64_t whole, int splits, int64_t part) {
            const int64_t parts = (tiles - whole) * splits;
            const int64_t t = cut_in(whole, slots) * all + cut_in(parts, slots) * part + ends_time(pair, parts);
            if (t < least) least = t, best = p, best.whole = (int)whole, best.splits = splits;
        };
        consider(tiles, 1, 0);
        for (const int64_t whole : {(int64_t)0, tiles / slots * slots}) {
            const int64_t rest = tiles - whole;
            for (int splits = 2; rest > 0 && splits * rest <= slots && splits * 4 <= p.kb; ++splits) {
                const int64_t part = unit_time(p, splits);
                consider(whole, splits, part);
                if (part == SHORTEST) break;
            }
            if (tiles < slots) break;
        }
    }
    return best;
}

// dx and the weights' gradients in one launch, the longer units first, so that either fills what the other's last round leaves; or
// one after the other, where each has rounds enough: what runs side by side then shares less of L2 (8192 x 2048 x 8192: 682 us
// in one launch, 657 in two; 1537 x 1001 x 2731: 35 us in one, 63 in two).
FfnBackward ffn_plan_backward(int64_t tokens, int64_t dim, int64_t inner) {
    FfnBackward best = {};
    int64_t first, second;
    best.plan[0] = ffn_plan_one(FFN_DX, tokens, dim, inner, first), best.plan[1] = ffn_plan_one(FFN_DW, tokens, dim, inner, second);
    int64_t least = first + second;
    for (const bool pair : {true, false}) {
        FfnPlan one = plan_of(FFN_DX, pair, tokens, dim, inner), two = plan_of(FFN_DW, pair, tokens, dim, inner);
        const bool swap = two.kb > one.kb;
        if (swap) std::swap(one, two);
        const int64_t tiles1 = one.whole, tiles2 = two.whole, slots = pair ? 76 : 152;
        for (int s1 = 1; s1 == 1 || (tiles1 * s1 + tiles2 <= slots && s1 * 4 <= one.kb); ++s1) {
            const int64_t t1 = unit_time(one, s1);
            int s2 = 1;  // the second job's units no longer than the first's, where they can be cut
            while (s1 > 1 && unit_time(two, s2) > t1 && tiles1 * s1 + tiles2 * (s2 + 1) <= slots && (s2 + 1) * 4 <= two.kb) ++s2;
            int extra;
            const int64_t parts = (s1 > 1 ? tiles1 * s1 : 0) + (s2 > 1 ? tiles2 * s2 : 0);
            int64_t t = two_jobs(tiles1 * s1, t1, tiles2 * s2, unit_time(two, s2), slots, extra);
            if (tiles1 > slots && tiles2 > slots) t += t / 14;
            t += ends_time(pair, parts);
            if (t < least) {
                least = t;
                one.splits = s1, one.whole = s1 > 1 ? 0 : (int)tiles1, two.splits = s2, two.whole = s2 > 1 ? 0 : (int)tiles2;
                best = {{one, two}, true, swap, extra};
            }
            if (t1 == SHORTEST) break;
        }
    }
    return best;
}

size_t FfnPlan::partial_bytes() const { return (size_t)(units() - whole) * (pair ? 256 : 128) * FFN_BN * sizeof(float); }

}  // namespace gdr
