// k10_linrec.cu -- the gated linear recurrence: workspace, grid, and choice by type.
#include "block_common.cuh"

namespace gdr {

// A sequence of up to this many tiles is walked by one CTA per block of channels: a tile takes it about 2 us, and the
// tree's cleared flags and hops cost more than that until there are as many.
constexpr int LR_WALK = 4;

namespace {
size_t up(size_t n) { return (n + 255) & ~size_t(255); }

// Records at each level of the tree over `tiles` tiles.
void tree_sizes(int64_t tiles, int64_t (&n)[4]) {
    for (int level = 0; level < 4; ++level) n[level] = (tiles + ((int64_t)1 << (3 * level)) - 1) >> (3 * level);
}
}  // namespace

// status and ticket, the flags (for the narrowest blocks, 32 channels), then the records
size_t linrec_workspace(int64_t rows, int64_t dim) {
    const int64_t tiles = (rows + LR_TILE - 1) / LR_TILE;
    if (tiles <= LR_WALK) return 256;
    int64_t n[4];
    tree_sizes(tiles, n);
    size_t bytes = 256;
    for (int level = 0; level < 4; ++level) bytes += up(sizeof(int) * (size_t)(n[level] * ((dim + 31) / 32)));
    for (int level = 0; level < 4; ++level) bytes += up(sizeof(float2) * (size_t)(n[level] * dim));
    return bytes;
}

// Places the tree in the workspace for blocks of `channels` and clears what has to start at zero.
cudaError_t linrec_blocks(LinrecParams &p, int channels, cudaStream_t stream) {
    p.tiles = p.rows > 0 ? (p.rows + LR_TILE - 1) / LR_TILE : 1;
    p.nblk = (p.dim + channels - 1) / channels;
    p.walk = p.tiles <= LR_WALK;
    p.blocks = FastDiv::of((uint32_t)p.nblk);
    p.per_seq = FastDiv::of((uint32_t)(p.tokens > 0 ? p.tokens : 1));
    if (p.walk) {
        p.grid = (unsigned)p.nblk;
        return cudaSuccess;
    }
    const int64_t grid = (int64_t)p.tiles * p.nblk;
    if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
    p.grid = (unsigned)grid;
    int64_t n[4];
    tree_sizes(p.tiles, n);
    char *at = reinterpret_cast<char *>(p.status) + 256;
    for (int level = 0; level < 4; ++level) {
        p.flags[level] = reinterpret_cast<int *>(at);
        at += up(sizeof(int) * (size_t)(n[level] * p.nblk));
    }
    const size_t cleared = at - reinterpret_cast<char *>(p.status);
    for (int level = 0; level < 4; ++level) {
        p.recs[level] = reinterpret_cast<float2 *>(at);
        at += up(sizeof(float2) * (size_t)(n[level] * p.dim));
    }
    p.ticket = p.status + 1;
    return cudaMemsetAsync(p.status, 0, cleared, stream);
}

template <typename T, typename G> cudaError_t linrec_fwd_t(LinrecParams &, cudaStream_t);
template <typename T, typename G> cudaError_t linrec_bwd_t(LinrecParams &, cudaStream_t);
template <typename T, typename G> cudaError_t linrec_step_t(StepParams &, cudaStream_t);

#define BY_TYPES(p, CALL)                                                       \
    do {                                                                        \
        if (p.dtype == F32) return CALL(float, float);                          \
        if (p.dtype == BF16 && p.gate_dtype == F32) return CALL(__nv_bfloat16, float); \
        if (p.dtype == BF16) return CALL(__nv_bfloat16, __nv_bfloat16);         \
        if (p.gate_dtype == F32) return CALL(__half, float);                    \
        return CALL(__half, __half);                                            \
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
