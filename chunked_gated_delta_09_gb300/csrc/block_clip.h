// block_clip.h -- the table of tensors that the clip's kernels take as an argument, and their launchers.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace gdr {

constexpr int CLIP_TENSORS = 640;    // per launch; longer lists take more launches (kernel arguments end at 32,764 bytes)
constexpr int CLIP_PIECE = 16384;    // elements
// Many short CTAs, which the device spreads as they end (393 M bf16 gradients into fp32: 4 to an SM 0.507 ms, 8 0.493, 16 0.485).
constexpr int CLIP_CTAS = 152 * 16;

template <int N> struct ClipTable {
    const void *grad[N];
    void *out[N];
    int64_t size[N];
    int64_t first[N + 1];  // number of the tensor's first piece
    int64_t pieces;
    int count;
    uint8_t dtype[N], out_dtype[N];
};
static_assert(sizeof(ClipTable<CLIP_TENSORS>) <= 32000, "the table is a kernel argument");

cudaError_t launch_clip_sumsq(const ClipTable<CLIP_TENSORS> &t, double *part, int parts, cudaStream_t stream);
// Whether all tensors together are few enough for one launch, which then does everything.
bool clip_is_small(const ClipTable<CLIP_TENSORS> &t);
cudaError_t launch_clip_small(const ClipTable<CLIP_TENSORS> &t, float *norm, bool scale, float max_norm, float eps,
                              cudaStream_t stream);
cudaError_t launch_clip_norm(const double *part, int parts, float *norm, cudaStream_t stream);
cudaError_t launch_clip_scale(const ClipTable<CLIP_TENSORS> &t, const double *part, int parts, float *norm, float max_norm,
                              float eps, cudaStream_t stream);

}  // namespace gdr
