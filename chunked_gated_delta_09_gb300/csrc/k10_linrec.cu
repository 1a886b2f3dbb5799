// k10_linrec.cu -- the gated linear recurrence: cluster and grid, tensor maps, and choice by type.
#include <mutex>
#include <unordered_map>

#include "block_common.cuh"

namespace gdr {
namespace {

// For clusters of 1 to 16 CTAs: how many clusters of a kernel the device holds at a time (0: none).
struct Resident {
    int clusters[LR_MAX_CLUSTER + 1];
};
std::mutex g_mu;
std::unordered_map<const void *, Resident> g_resident[64];  // per device

cudaError_t resident(LinrecLaunch &l, Resident &out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(g_mu);
    if (dev >= 0 && dev < 64) {
        auto it = g_resident[dev].find(l.kernel);
        if (it != g_resident[dev].end()) {
            out = it->second;
            return cudaSuccess;
        }
    }
    if ((e = cudaFuncSetAttribute(l.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, l.smem)) != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(l.kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1)) != cudaSuccess) return e;
    for (int size = 1; size <= LR_MAX_CLUSTER; ++size) {
        l.cfg.gridDim = dim3((unsigned)size);
        l.attr.val.clusterDim.x = (unsigned)size;
        if (cudaOccupancyMaxActiveClusters(&out.clusters[size], l.kernel, &l.cfg) != cudaSuccess) {
            cudaGetLastError();
            out.clusters[size] = 0;
        }
    }
    if (out.clusters[1] < 1) return cudaErrorInvalidConfiguration;
    if (dev >= 0 && dev < 64) g_resident[dev][l.kernel] = out;
    return cudaSuccess;
}

}  // namespace

// Chooses the cluster's size and the grid for tiles of `rows_per_tile` rows x 32 channels; narrow: set instead where the
// largest clusters would put at most two CTAs on an SM and have several tiles in turn, for which larger CTAs do better.
cudaError_t linrec_plan(LinrecParams &p, LinrecLaunch &l, int rows_per_tile, bool *narrow, cudaStream_t stream) {
    l.cfg = {};
    l.cfg.blockDim = dim3((unsigned)l.threads);
    l.cfg.dynamicSmemBytes = (size_t)l.smem;
    l.cfg.stream = stream;
    l.attr.id = cudaLaunchAttributeClusterDimension;
    l.attr.val.clusterDim.x = l.attr.val.clusterDim.y = l.attr.val.clusterDim.z = 1;
    l.cfg.attrs = &l.attr;
    l.cfg.numAttrs = 1;
    Resident r;
    cudaError_t e = resident(l, r);
    if (e != cudaSuccess) return e;
    p.tiles = p.rows > 0 ? (p.rows + rows_per_tile - 1) / rows_per_tile : 1;
    p.per_seq = FastDiv::of((uint32_t)(p.tokens > 0 ? p.tokens : 1));
    const int64_t nblk = (p.dim + LR_CH - 1) / LR_CH;
    if (narrow && p.tiles > LR_MAX_CLUSTER && 5 * LR_MAX_CLUSTER * nblk <= 2 * r.clusters[1]) {
        *narrow = true;
        return cudaSuccess;
    }
    // The size whose clusters take the fewest tiles one after the other, all waves of them together.  A tile takes about 2 %
    // longer with each CTA more, from the exchange of the maps (48763 x 4096 bf16, backward: 6 CTAs, 127 tiles in turn,
    // 0.404 ms; 5 CTAs, 153 tiles, 0.426 ms; 10 CTAs in two waves, 154 tiles, 0.432 ms; 7 CTAs in two, 218, 0.497 ms); a wave
    // has to start and to end, which costs it about two more (4096 x 8192 bf16, forward: 2 CTAs in one wave, 16 tiles, 0.051
    // ms; 8 CTAs in three, 12 tiles, 0.056 ms).
    int64_t best = -1;
    for (int size = 1; size <= LR_MAX_CLUSTER; ++size) {
        if (r.clusters[size] < 1 || size > p.tiles) continue;
        const int64_t waves = (nblk + r.clusters[size] - 1) / r.clusters[size];
        const int64_t cost = waves * ((p.tiles + size - 1) / size + 2) * (50 + size);
        if (best < 0 || cost < best) best = cost, p.cluster = size;
    }
    p.supers = (p.tiles + p.cluster - 1) / p.cluster;
    l.cfg.gridDim = dim3((unsigned)(nblk * p.cluster));
    l.attr.val.clusterDim.x = (unsigned)p.cluster;
    // One CTA checks short lists in about the time of the other's first tile and sets the status word, which saves the launch that
    // clears it.  (Waits that a short limit makes expire may be noted before that.)
    p.clear = (!p.cu || p.N <= 1024) && p.spin >= (1u << 16);
    return p.clear ? cudaSuccess : cudaMemsetAsync(p.status, 0, sizeof(int), stream);
}

cudaError_t linrec_maps(const LinrecParams &p, LinrecMaps &maps, int rows_per_tile) {
    auto one = [&](CUtensorMap &map, const void *base, int dtype, int64_t stride) {
        // (one row has no distance to a next one: any that a map takes)
        return encode_matrix_map(&map, base, dtype, p.rows, p.dim, p.rows > 1 ? stride : (p.dim + 7) / 8 * 8, rows_per_tile, LR_CH);
    };
    cudaError_t e = one(maps.g, p.g, p.gate_dtype, p.g_ts);
    if (e == cudaSuccess) e = one(maps.x, p.x, p.dtype, p.x_ts);
    if (e == cudaSuccess && p.dh) e = one(maps.dh, p.dh, p.dtype, p.dh_ts);
    return e;
}

template <typename T, typename G> cudaError_t linrec_fwd_t(LinrecParams &, cudaStream_t);
template <typename T, typename G> cudaError_t linrec_bwd_t(LinrecParams &, cudaStream_t);
template <typename T, typename G> cudaError_t linrec_step_t(StepParams &, cudaStream_t);

#define BY_TYPES(p, CALL)                                                              \
    do {                                                                               \
        if (p.dtype == F32) return CALL(float, float);                                 \
        if (p.dtype == BF16 && p.gate_dtype == F32) return CALL(__nv_bfloat16, float); \
        if (p.dtype == BF16) return CALL(__nv_bfloat16, __nv_bfloat16);                \
        if (p.gate_dtype == F32) return CALL(__half, float);                           \
        return CALL(__half, __half);                                                   \
    } while (0)

cudaError_t launch_linrec_fwd(LinrecParams p, cudaStream_t stream) {
#define CALL(T, G) linrec_fwd_t<T, G>(p, stream)
    BY_TYPES(p, CALL);
#undef CALL
}
cudaError_t launch_linrec_bwd(LinrecParams p, cudaStream_t stream) {
#define CALL(T, G) linrec_bwd_t<T, G>(p, stream)
    BY_TYPES(p, CALL);
#undef CALL
}
cudaError_t launch_linrec_step(StepParams p, cudaStream_t stream) {
#define CALL(T, G) linrec_step_t<T, G>(p, stream)
    BY_TYPES(p, CALL);
#undef CALL
}

}  // namespace gdr
