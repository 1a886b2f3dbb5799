// ffn.h -- parameters, work plans and launchers of the gated feed-forward (gdr_ffn_fwd, gdr_ffn_bwd).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/gdr_block.h"
#include "block_common.cuh"

namespace gdr {

// Tiles of the products: 256 columns of results, 128 rows for each CTA, 64 of the summed axis at a time.
constexpr int FFN_BM = 128, FFN_BN = 256, FFN_BK = 64;
// Up to this many tokens the forward pass streams the weights through registers instead (2048 x 8192: 32 tokens 17.5 us, 33 by
// tiles 20.5; 1024 x 4096: 8.0 and 12.0).
constexpr int FFN_FEW = GDR_FFN_FEW_TOKENS;

// The three products: h from x and the two weights (256 columns are 128 of each), dx from [dg du] and the weights,
// [dWg; dWu] from [dg du] and x.
enum FfnProduct { FFN_FWD = 0, FFN_DX = 1, FFN_DW = 2 };

// How a product is cut: mt x nt tiles and kb pieces of the summed axis.  The first `whole` tiles are worked on whole; the summed
// axis of the others is cut in `splits` parts, fp32 results that are added in order.
struct FfnPlan {
    int mt, nt, kb, whole, splits;
    // Tiles below each other that go together, so that the columns' operand stays in L2: 8192 x 2048 x 8192 forward 318 us by 16,
    // 326 by 4; the others 318 and 326 us by 4, 322 and 330 by 16.
    int group;
    bool pair;  // tiles of 256 rows for two CTAs
    __host__ __device__ int cut() const { return mt * nt - whole; }
    __host__ __device__ int units() const { return whole + cut() * splits; }
    size_t partial_bytes() const;
};
// The plan of a product by itself, and its estimated time in hundredths of a us.
FfnPlan ffn_plan_one(FfnProduct what, int64_t tokens, int64_t dim, int64_t inner, int64_t &time);
// Those of the backward's two, FFN_DX and FFN_DW: one after the other, or both in one launch, then the longer units first (FFN_DW
// where `swapped`), and how many rounds of the second the CTAs take that had a unit in the first one's last round.
struct FfnBackward {
    FfnPlan plan[2];
    bool joint, swapped;
    int extra;
};
FfnBackward ffn_plan_backward(int64_t tokens, int64_t dim, int64_t inner);

struct FfnMaps {
    CUtensorMap a[2][2], b[2][2];  // of each job: along the summed axis or the rows, its first and second half
};

struct FfnJob {
    FfnProduct what;
    FfnPlan plan;        // of no tiles: nothing to do
    int64_t rows, cols;  // of the result (FFN_DW: of each half of it); its rows are contiguous
    void *out[2];        // FFN_FWD: h; FFN_DX: dx; FFN_DW: dWg, dWu
    int piece;           // bytes that results are stored in: 32 or 16 where all rows are multiples of that
    int first_part;      // of the partial results
};

struct FfnGemm {
    FfnJob job[2];
    int extra;
    float *gate, *up;  // forward: kept for the backward, or null
    int piece32;       // bytes that those are stored in
    float *part;       // partial results: a tile's rows of 256 for each part of each tile that is cut
    int dtype, act;
    uint32_t spin;
    // Whether waits ran out: a byte for each CTA, which no other writes, so that clearing needs no order among them; or null: nobody
    // asks.  clear: what the bytes held is of an earlier call (else an earlier launch of this call has cleared them).
    uint8_t *status;
    bool clear;
};
cudaError_t launch_ffn_product(const FfnMaps &maps, const FfnGemm &p, cudaStream_t stream);

struct FfnFew {
    const void *x, *wg, *wu;
    void *h;
    float *gate, *up;
    int64_t x_ts, wg_rs, wu_rs;
    int tokens, dim, inner, dtype, act;
    bool vec;
};
cudaError_t launch_ffn_few(const FfnFew &p, cudaStream_t stream);

// dg = dh u act'(g), du = dh act(g) into rows `pitch` apart.
struct FfnAct {
    const void *dh;
    const float *gate, *up;
    void *dg, *du;
    int64_t dh_ts, tokens, inner, pitch;
    int dtype, act;
    bool vec;
    uint8_t *status;  // cleared
};
cudaError_t launch_ffn_act(const FfnAct &p, cudaStream_t stream);

// Up to three matrices of 16-bit rows of one width, copied to rows a multiple of 8 elements apart, zeros behind them.
struct FfnPad {
    const void *from[3];
    void *to[3];
    int64_t stride[3], rows[3];
    uint32_t warps[3];
    int count, cols;
    int64_t pitch;  // (64 bits: rows times pitch passes 2^32)
    FastDiv per_row;
    uint8_t *status;  // cleared
};
cudaError_t launch_ffn_pad(FfnPad p, cudaStream_t stream);

// Tensor map of 16-bit rows for boxes of box_rows x 64 elements with the 128-byte swizzle (16-byte piece j of row r lies at
// piece j ^ (r % 8)); what lies outside reads as zero.
cudaError_t encode_matrix_map_sw128(CUtensorMap *map, const void *base, int dtype, int64_t rows, int64_t cols, int64_t stride,
                                    int box_rows);

}  // namespace gdr
