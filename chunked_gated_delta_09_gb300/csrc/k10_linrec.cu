// k10_linrec.cu -- the gated linear recurrence h_t = a_t h_{t-1} + b_t over packed or dense sequences, its backward
// and its single-token step.
#include "block_common.cuh"

namespace gdr {
namespace {

constexpr int LR_TILE = 64;  // rows between saved states

// a = exp(g) and, where the input is weighted by it, 1 - a.
__device__ __forceinline__ void decay(float g, float &a, float &rest) {
    const float e = expm1f(g);
    a = g > -0.5f ? 1.f + e : expf(g);
    rest = -e;
}

__device__ __forceinline__ void lr_range(const LinrecParams &p, int s, int &bos, int &eos) {
    bos = p.cu ? p.cu[s] : s * p.tokens;
    eos = p.cu ? p.cu[s + 1] : bos + p.tokens;
    bos = max(0, min(bos, p.rows));
    eos = max(bos, min(eos, p.rows));
}

// One thread walks one channel of one sequence.
__global__ void k10_fwd(const LinrecParams p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, s = blockIdx.y;
    if (p.cu && c == 0 && s == 0 && (p.cu[0] != 0 || p.cu[p.N] != p.rows)) atomicOr(p.status, ST_BAD_SEQLENS);
    if (p.cu && c == 0 && p.cu[s + 1] < p.cu[s]) atomicOr(p.status, ST_BAD_SEQLENS);
    if (c >= p.dim) return;
    int bos, eos;
    lr_range(p, s, bos, eos);
    float h = p.h0 ? p.h0[(size_t)s * p.dim + c] : 0.f;
    for (int t = bos; t < eos; ++t) {
        float a, rest;
        decay(load_scalar(p.g, (size_t)t * p.g_ts + c, p.gate_dtype), a, rest);
        const float x = load_scalar(p.x, (size_t)t * p.x_ts + c, p.dtype);
        if (p.states && t % LR_TILE == 0) p.states[(size_t)(t / LR_TILE) * p.dim + c] = h;
        h = fmaf(a, h, p.complement ? rest * x : x);
        if (p.h) store_scalar(p.h, (size_t)t * p.dim + c, h, p.dtype);
    }
    if (p.ht) p.ht[(size_t)s * p.dim + c] = h;
}

__global__ void k10_bwd(const LinrecParams p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x, s = blockIdx.y;
    if (p.cu && c == 0 && s == 0 && (p.cu[0] != 0 || p.cu[p.N] != p.rows)) atomicOr(p.status, ST_BAD_SEQLENS);
    if (p.cu && c == 0 && p.cu[s + 1] < p.cu[s]) atomicOr(p.status, ST_BAD_SEQLENS);
    if (c >= p.dim) return;
    int bos, eos;
    lr_range(p, s, bos, eos);
    float mu = p.dht ? p.dht[(size_t)s * p.dim + c] : 0.f, before[LR_TILE];
    for (int end = eos; end > bos;) {
        const int start = max(bos, (end - 1) / LR_TILE * LR_TILE);
        float h = start == bos ? (p.h0 ? p.h0[(size_t)s * p.dim + c] : 0.f) : p.states[(size_t)(start / LR_TILE) * p.dim + c];
        for (int t = start; t < end; ++t) {
            float a, rest;
            decay(load_scalar(p.g, (size_t)t * p.g_ts + c, p.gate_dtype), a, rest);
            const float x = load_scalar(p.x, (size_t)t * p.x_ts + c, p.dtype);
            before[t - start] = h;
            h = fmaf(a, h, p.complement ? rest * x : x);
        }
        for (int t = end - 1; t >= start; --t) {
            float a, rest;
            decay(load_scalar(p.g, (size_t)t * p.g_ts + c, p.gate_dtype), a, rest);
            const float x = load_scalar(p.x, (size_t)t * p.x_ts + c, p.dtype);
            const float lam = load_scalar(p.dh, (size_t)t * p.dh_ts + c, p.dtype) + mu;
            const float prev = p.complement ? before[t - start] - x : before[t - start];
            mu = a * lam;
            store_scalar(p.dx, (size_t)t * p.dim + c, p.complement ? rest * lam : lam, p.dtype);
            store_scalar(p.dg, (size_t)t * p.dim + c, mu * prev, p.gate_dtype);
        }
        end = start;
    }
    if (p.dh0) p.dh0[(size_t)s * p.dim + c] = mu;
}

__global__ void k10_step(const StepParams p) {
    const int c = blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t i = blockIdx.y;
    if (c >= p.dim) return;
    const int64_t slot = p.slots ? p.slots[i] : i;
    float y = 0.f;
    if (slot >= 0 && slot < p.num_slots) {
        float a, rest;
        decay(load_scalar(p.g, (size_t)i * p.g_ts + c, p.gate_dtype), a, rest);
        const float x = load_scalar(p.x, (size_t)i * p.x_ts + c, p.dtype);
        float *h = p.state + (size_t)slot * p.dim + c;
        y = fmaf(a, *h, p.complement ? rest * x : x);
        *h = y;
    }
    store_scalar(p.y, (size_t)i * p.dim + c, y, p.dtype);
}

}  // namespace

cudaError_t launch_linrec_fwd(const LinrecParams &p, cudaStream_t stream) {
    k10_fwd<<<dim3((p.dim + 127) / 128, p.N), 128, 0, stream>>>(p);
    return cudaGetLastError();
}
cudaError_t launch_linrec_bwd(const LinrecParams &p, cudaStream_t stream) {
    k10_bwd<<<dim3((p.dim + 127) / 128, p.N), 128, 0, stream>>>(p);
    return cudaGetLastError();
}
cudaError_t launch_linrec_step(const StepParams &p, cudaStream_t stream) {
    k10_step<<<dim3((p.dim + 127) / 128, (unsigned)p.batch), 128, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace gdr
