// ffn_api.cu -- the C entries of the gated feed-forward: argument checks, workspace and launches.
#include <stdlib.h>

#include "block_args.h"
#include "ffn.h"
#include "ffn_act.cuh"

using namespace gdr;

namespace {

int64_t round8(int64_t n) { return (n + 7) / 8 * 8; }
size_t region(size_t bytes) { return (bytes + 255) / 256 * 256; }

// Sizes that the calls take: 0 fine, otherwise the status to return.
gdr_status sizes(int64_t tokens, int64_t dim, int64_t inner) {
    if (tokens < 0 || dim < 1 || inner < 1) return GDR_ERR_INVALID_ARG;
    if (tokens > kMaxRows || dim > GDR_FFN_MAX_DIM || inner > GDR_FFN_MAX_DIM || tokens * (round8(dim) / 8) > kMaxRows ||
        tokens * (round8(inner) / 8) > kMaxRows || inner * (round8(dim) / 8) > kMaxRows)
        return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Whether a tensor map takes rows of 16-bit elements as they are.
bool mappable(const void *p, int64_t stride, int64_t rows, int64_t cols) {
    return at(p, 16) && (rows <= 1 || (stride % 8 == 0 && stride >= cols && stride < (1ll << 36)));
}

// Workspace, in 256-byte regions: status | x, Wg, Wu brought to 16-byte boundaries (calls with `copies`) | backward:
// dg, du | partial results.
struct Layout {
    size_t x, wg, wu, dg, du, part, total;
    FfnPlan forward;
    FfnBackward backward;
    Layout(int64_t tokens, int64_t dim, int64_t inner, bool copies, bool bwd) {
        size_t at = GDR_FFN_STATUS_BYTES;
        auto take = [&](size_t bytes) {
            const size_t o = at;
            at += region(bytes);
            return o;
        };
        const size_t w = copies ? (size_t)(inner * round8(dim)) * 2 : 0, d = bwd ? (size_t)(tokens * round8(inner)) * 2 : 0;
        x = take(copies ? (size_t)(tokens * round8(dim)) * 2 : 0), wg = take(w), wu = take(w), dg = take(d), du = take(d);
        if (bwd) {
            backward = ffn_plan_backward(tokens, dim, inner);
            part = take(backward.plan[0].partial_bytes() + backward.plan[1].partial_bytes());
        } else {
            int64_t time;
            forward = ffn_plan_one(FFN_FWD, tokens, dim, inner, time);
            part = take(forward.partial_bytes());
        }
        total = at;
    }
};

uint32_t spin_limit() {
    const char *spin = getenv("GDR_SPIN_LIMIT");  // a test knob, as for the delta rule's plans
    return spin && atol(spin) > 0 ? (uint32_t)atol(spin) : WAIT_LIMIT_DEFAULT;
}

// Rows as a tensor map takes them: where they are, or copied to `copy`.
struct Rows {
    const void *p;
    int64_t stride;
};
void to_rows(FfnPad &pad, Rows &r, void *copy, int64_t rows, int64_t cols) {
    if (mappable(r.p, r.stride, rows, cols)) return;
    const int m = pad.count++;
    pad.from[m] = r.p, pad.to[m] = copy, pad.stride[m] = r.stride, pad.rows[m] = rows, pad.cols = (int)cols;
    r = {copy, round8(cols)};
}
cudaError_t map_of(CUtensorMap &m, Rows r, int dtype, int64_t rows, int64_t cols, int box_rows) {
    return encode_matrix_map_sw128(&m, r.p, dtype, rows, cols, rows > 1 ? r.stride : round8(cols), box_rows);
}

// The status in the workspace of a call in which nothing waits, where it is given one.
cudaError_t clear_status(void *ws, uint64_t bytes, cudaStream_t stream) {
    if (!ws || !at(ws, 256) || bytes < GDR_FFN_STATUS_BYTES) return cudaSuccess;
    return cudaMemsetAsync(ws, 0, GDR_FFN_STATUS_BYTES, stream);
}

int piece_of(const void *t, const void *u, int64_t row_bytes) {
    int n = 32;
    while (n > 8 && !(at(t, n) && at(u, n) && row_bytes % n == 0)) n /= 2;
    return n;
}
FfnJob job_of(FfnProduct what, const FfnPlan &plan, void *out0, void *out1, int64_t rows, int64_t cols) {
    return {what, plan, rows, cols, {out0, out1}, piece_of(out0, out1, cols * 2), 0};
}

}  // namespace

extern "C" {

size_t gdr_ffn_workspace_bytes(int64_t tokens, int64_t dim, int64_t inner, int copies, int backward) {
    if (sizes(tokens, dim, inner) != GDR_OK || tokens == 0) return 0;
    if (!backward && tokens <= FFN_FEW) return 0;
    return Layout(tokens, dim, inner, copies != 0, backward != 0).total;
}

gdr_status gdr_ffn_fwd(const gdr_ffn_fwd_args *a, void *stream_) {
    if (!a) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    const gdr_status st = sizes(a->tokens, a->dim, a->inner);
    if (st != GDR_OK) return st;
    if ((a->dtype != GDR_BF16 && a->dtype != GDR_F16) || a->activation < 0 || a->activation > GDR_FFN_GELU_TANH ||
        !a->gate != !a->up || (!a->h && !a->gate))
        return a->dtype == GDR_F32 ? GDR_ERR_UNSUPPORTED : GDR_ERR_INVALID_ARG;
    if (a->tokens == 0) return done(clear_status(a->workspace, a->workspace_bytes, stream));
    if (!a->x || !a->w_gate || !a->w_up || a->x_token_stride < 0 || a->w_gate_row_stride < 0 || a->w_up_row_stride < 0)
        return GDR_ERR_INVALID_ARG;
    if (!at(a->x, 2) || !at(a->w_gate, 2) || !at(a->w_up, 2) || !at(a->h, 2) || !at(a->gate, 4) || !at(a->up, 4))
        return GDR_ERR_INVALID_ARG;
    if (a->tokens <= FFN_FEW) {
        VecRule v(8, a->dim);
        v.tensor(a->x, a->dtype, a->x_token_stride);
        v.tensor(a->w_gate, a->dtype, a->w_gate_row_stride);
        v.tensor(a->w_up, a->dtype, a->w_up_row_stride);
        FfnFew p = {};
        p.x = a->x, p.wg = a->w_gate, p.wu = a->w_up, p.h = a->h, p.gate = a->gate, p.up = a->up;
        p.x_ts = a->x_token_stride, p.wg_rs = a->w_gate_row_stride, p.wu_rs = a->w_up_row_stride;
        p.tokens = (int)a->tokens, p.dim = (int)a->dim, p.inner = (int)a->inner, p.dtype = a->dtype, p.act = a->activation;
        p.vec = v.ok;
        const cudaError_t e = clear_status(a->workspace, a->workspace_bytes, stream);
        return done(e != cudaSuccess ? e : launch_ffn_few(p, stream));
    }
    Rows x = {a->x, a->x_token_stride}, wg = {a->w_gate, a->w_gate_row_stride}, wu = {a->w_up, a->w_up_row_stride};
    const bool copies = !mappable(x.p, x.stride, a->tokens, a->dim) || !mappable(wg.p, wg.stride, a->inner, a->dim) ||
                        !mappable(wu.p, wu.stride, a->inner, a->dim);
    const Layout l(a->tokens, a->dim, a->inner, copies, false);
    const bool status_alone = l.total == GDR_FFN_STATUS_BYTES;
    if (!(status_alone && !a->workspace) && (!a->workspace || !at(a->workspace, 256) || a->workspace_bytes < l.total))
        return GDR_ERR_INVALID_ARG;
    char *ws = (char *)a->workspace;
    FfnPad pad = {};
    pad.status = (uint8_t *)ws;
    to_rows(pad, x, ws + l.x, a->tokens, a->dim);
    to_rows(pad, wg, ws + l.wg, a->inner, a->dim);
    to_rows(pad, wu, ws + l.wu, a->inner, a->dim);
    cudaError_t e = pad.count ? launch_ffn_pad(pad, stream) : cudaSuccess;
    FfnMaps maps;
    if (e == cudaSuccess) e = map_of(maps.a[0][0], x, a->dtype, a->tokens, a->dim, FFN_BM);
    if (e == cudaSuccess) e = map_of(maps.b[0][0], wg, a->dtype, a->inner, a->dim, FFN_BN / 2);
    if (e == cudaSuccess) e = map_of(maps.b[0][1], wu, a->dtype, a->inner, a->dim, FFN_BN / 2);
    if (e != cudaSuccess) return GDR_ERR_CUDA;
    FfnGemm p = {};
    p.job[0] = job_of(FFN_FWD, l.forward, a->h, nullptr, a->tokens, a->inner);
    p.gate = a->gate, p.up = a->up, p.piece32 = piece_of(a->gate, a->up, a->inner * 4), p.part = (float *)(ws + l.part);
    p.dtype = a->dtype, p.act = a->activation, p.spin = spin_limit(), p.status = (uint8_t *)ws, p.clear = ws && pad.count == 0;
    return done(launch_ffn_product(maps, p, stream));
}

gdr_status gdr_ffn_bwd(const gdr_ffn_bwd_args *a, void *stream_) {
    if (!a) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    const gdr_status st = sizes(a->tokens, a->dim, a->inner);
    if (st != GDR_OK) return st;
    if ((a->dtype != GDR_BF16 && a->dtype != GDR_F16) || a->activation < 0 || a->activation > GDR_FFN_GELU_TANH ||
        !a->dw_gate != !a->dw_up)
        return a->dtype == GDR_F32 ? GDR_ERR_UNSUPPORTED : GDR_ERR_INVALID_ARG;
    if (!at(a->dx, 2) || !at(a->dw_gate, 2) || !at(a->dw_up, 2)) return GDR_ERR_INVALID_ARG;
    if (a->tokens == 0 || (!a->dx && !a->dw_gate)) {
        const size_t bytes = (size_t)(a->inner * a->dim) * 2;
        cudaError_t e = clear_status(a->workspace, a->workspace_bytes, stream);
        if (e == cudaSuccess && a->dw_gate) e = cudaMemsetAsync(a->dw_gate, 0, bytes, stream);
        if (e == cudaSuccess && a->dw_gate) e = cudaMemsetAsync(a->dw_up, 0, bytes, stream);
        return done(e);
    }
    if (!a->dh || !a->gate || !a->up || (a->dw_gate && !a->x) || (a->dx && (!a->w_gate || !a->w_up)) || a->dh_token_stride < 0 ||
        a->x_token_stride < 0 || a->w_gate_row_stride < 0 || a->w_up_row_stride < 0)
        return GDR_ERR_INVALID_ARG;
    if (!at(a->dh, 2) || !at(a->gate, 4) || !at(a->up, 4) || !at(a->x, 2) || !at(a->w_gate, 2) || !at(a->w_up, 2))
        return GDR_ERR_INVALID_ARG;
    Rows x = {a->x, a->x_token_stride}, wg = {a->w_gate, a->w_gate_row_stride}, wu = {a->w_up, a->w_up_row_stride};
    const bool copies = (a->dw_gate && !mappable(x.p, x.stride, a->tokens, a->dim)) ||
                        (a->dx && (!mappable(wg.p, wg.stride, a->inner, a->dim) || !mappable(wu.p, wu.stride, a->inner, a->dim)));
    const Layout l(a->tokens, a->dim, a->inner, copies, true);
    if (!a->workspace || !at(a->workspace, 256) || a->workspace_bytes < l.total) return GDR_ERR_INVALID_ARG;
    char *ws = (char *)a->workspace;
    VecRule v(8, a->inner);
    v.tensor(a->dh, a->dtype, a->dh_token_stride);
    v.tensor(a->gate, GDR_F32, a->inner);
    v.tensor(a->up, GDR_F32, a->inner);
    FfnAct act = {};
    act.dh = a->dh, act.gate = a->gate, act.up = a->up, act.dg = ws + l.dg, act.du = ws + l.du;
    act.dh_ts = a->dh_token_stride, act.tokens = a->tokens, act.inner = a->inner, act.pitch = round8(a->inner);
    act.dtype = a->dtype, act.act = a->activation, act.vec = v.ok, act.status = (uint8_t *)ws;
    cudaError_t e = launch_ffn_act(act, stream);
    FfnPad pad = {};
    pad.status = (uint8_t *)ws;
    if (a->dx) to_rows(pad, wg, ws + l.wg, a->inner, a->dim), to_rows(pad, wu, ws + l.wu, a->inner, a->dim);
    if (a->dw_gate) to_rows(pad, x, ws + l.x, a->tokens, a->dim);
    if (e == cudaSuccess && pad.count) e = launch_ffn_pad(pad, stream);
    if (e != cudaSuccess) return GDR_ERR_CUDA;
    const Rows d[2] = {{act.dg, act.pitch}, {act.du, act.pitch}};
    FfnMaps maps;
    FfnGemm p = {};
    p.part = (float *)(ws + l.part), p.dtype = a->dtype, p.spin = spin_limit(), p.status = (uint8_t *)ws;
    int jobs = 0;
    for (int j = 0; j < 2; ++j) {
        const bool dx = (j == 0) != l.backward.swapped;
        if (!(dx ? a->dx : a->dw_gate)) continue;  // not wanted
        FfnJob &job = p.job[jobs];
        job = dx ? job_of(FFN_DX, l.backward.plan[j], a->dx, nullptr, a->tokens, a->dim)
                 : job_of(FFN_DW, l.backward.plan[j], a->dw_gate, a->dw_up, a->inner, a->dim);
        for (int i = 0; i < 2 && e == cudaSuccess; ++i) {
            e = map_of(maps.a[jobs][i], d[i], a->dtype, a->tokens, a->inner, dx ? FFN_BM : FFN_BK);
            if (e == cudaSuccess && dx) e = map_of(maps.b[jobs][i], i ? wu : wg, a->dtype, a->inner, a->dim, FFN_BK);
        }
        if (e == cudaSuccess && !dx) e = map_of(maps.b[jobs][0], x, a->dtype, a->tokens, a->dim, FFN_BK);
        if (jobs == 1) job.first_part = p.job[0].plan.units() - p.job[0].plan.whole, p.extra = l.backward.extra;
        if (l.backward.joint) ++jobs;
        else if (e == cudaSuccess) e = launch_ffn_product(maps, p, stream);
    }
    if (e == cudaSuccess && jobs) e = launch_ffn_product(maps, p, stream);
    return done(e);
}

gdr_status gdr_ffn_get_status(void *workspace, void *stream_) {
    if (!workspace || !at(workspace, 256)) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    uint8_t status[GDR_FFN_STATUS_BYTES] = {};
    // all of it on the caller's stream, and done on return: the workspace may be given away then
    if (cudaMemcpyAsync(status, workspace, sizeof(status), cudaMemcpyDeviceToHost, stream) != cudaSuccess) return GDR_ERR_CUDA;
    if (cudaMemsetAsync(workspace, 0, sizeof(status), stream) != cudaSuccess) return GDR_ERR_CUDA;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return GDR_ERR_CUDA;
    for (const uint8_t ran_out : status)
        if (ran_out) return GDR_ERR_TIMEOUT;
    return GDR_OK;
}

}  // extern "C"
