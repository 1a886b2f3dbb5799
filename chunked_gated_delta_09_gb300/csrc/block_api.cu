// block_api.cu -- the C entries of include/gdr_block.h: argument checks and launches.  No device memory is allocated.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <stdlib.h>

#include <memory>
#include <new>

#include "../../include/gdr_block.h"
#include "block_clip.h"
#include "block_common.cuh"

using namespace gdr;

namespace {

constexpr int64_t kMaxRows = 1ll << 30;

bool type_ok(int d) { return d == GDR_F32 || d == GDR_BF16 || d == GDR_F16; }
int64_t type_size(int d) { return d == GDR_F32 ? 4 : 2; }
bool at(const void *p, int64_t a) { return (uintptr_t)p % (uintptr_t)a == 0; }

// Collects whether every tensor of a call can be moved in pieces of `n` elements (16 bytes at most at a time).  The width is
// part of the rule by itself: a thread has whole pieces, also in a call whose outputs, of stride `dim`, are all absent.
struct VecRule {
    int64_t n;
    bool ok, natural = true;
    VecRule(int64_t n_, int64_t dim) : VecRule(n_, dim, n_) {}
    VecRule(int64_t n_, int64_t dim, int64_t whole) : n(n_), ok(dim % whole == 0) {}  // whole: elements that a thread stores together
    void tensor(const void *p, int dtype, int64_t stride0 = 0, int64_t stride1 = 0) {
        if (!p) return;
        const int64_t s = type_size(dtype), need = n * s < 16 ? n * s : 16;
        natural = natural && at(p, s);
        ok = ok && at(p, need) && stride0 * s % need == 0 && stride1 * s % need == 0;
    }
};

// The largest pieces of rows of `dim` elements, 4, 2 or 1 of them, that start at multiples of their size in every tensor.
struct Pieces {
    int n;
    explicit Pieces(int64_t dim) : n(dim % 4 == 0 ? 4 : dim % 2 == 0 ? 2 : 1) {}
    void tensor(const void *p, int dtype, int64_t stride) {
        const int64_t s = type_size(dtype);
        while (n > 1 && !(at(p, n * s) && stride % n == 0)) n /= 2;
    }
};

gdr_status done(cudaError_t e) { return e == cudaSuccess ? GDR_OK : GDR_ERR_CUDA; }

// Rows (token, head) of a strided tensor as rows of one stride where that is possible.
bool collapses(int64_t ts, int64_t hs, int64_t tokens, int64_t heads) {
    return heads == 1 || tokens <= 1 || ts == heads * hs;
}

// Sizes that the norms take: 0 fine, otherwise the status to return.
gdr_status norm_sizes(int64_t tokens, int64_t heads, int64_t dim) {
    if (tokens < 0 || heads < 1 || dim < 1) return GDR_ERR_INVALID_ARG;
    if (dim > GDR_NORM_MAX_DIM || tokens > kMaxRows || heads > kMaxRows || tokens * heads > kMaxRows)
        return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

gdr_status clear_sum(void *out, int64_t dim, int dtype, cudaStream_t stream) {
    return out ? done(cudaMemsetAsync(out, 0, (size_t)(dim * type_size(dtype)), stream)) : GDR_OK;
}

}  // namespace

extern "C" {

size_t gdr_norm_workspace_bytes(int64_t rows, int64_t dim, int sums) {
    if (rows < 0 || dim < 1 || dim > GDR_NORM_MAX_DIM || sums < 0 || sums > 2) return 0;
    return (size_t)norm_parts(rows, dim) * (size_t)dim * (size_t)sums * sizeof(float);
}

gdr_status gdr_gated_norm_fwd(const gdr_gated_norm_fwd_args *a, void *stream) {
    if (!a) return GDR_ERR_INVALID_ARG;
    const gdr_status st = norm_sizes(a->tokens, a->heads, a->dim);
    if (st != GDR_OK) return st;
    if (!type_ok(a->dtype) || (a->weight && !type_ok(a->weight_dtype)) || (a->activation != 0 && a->activation != 1))
        return GDR_ERR_INVALID_ARG;
    if (a->tokens == 0) return GDR_OK;
    if (!a->x || !a->y) return GDR_ERR_INVALID_ARG;
    if (a->x_token_stride < 0 || a->x_head_stride < 0 || a->z_token_stride < 0 || a->z_head_stride < 0)
        return GDR_ERR_INVALID_ARG;
    VecRule v(16 / type_size(a->dtype), a->dim);
    v.tensor(a->x, a->dtype, a->x_token_stride, a->x_head_stride);
    v.tensor(a->z, a->dtype, a->z_token_stride, a->z_head_stride);
    v.tensor(a->y, a->dtype, a->dim);
    if (!v.natural || (a->weight && !at(a->weight, type_size(a->weight_dtype)))) return GDR_ERR_INVALID_ARG;
    GatedNormParams p = {};
    p.x = a->x, p.z = a->z, p.weight = a->weight, p.y = a->y;
    const bool flat = collapses(a->x_token_stride, a->x_head_stride, a->tokens, a->heads) &&
                      (!a->z || collapses(a->z_token_stride, a->z_head_stride, a->tokens, a->heads));
    p.heads = FastDiv::of(flat ? 1 : (uint32_t)a->heads);
    p.xm = {flat && a->heads > 1 ? a->x_head_stride : a->x_token_stride, a->x_head_stride};
    p.zm = {flat && a->heads > 1 ? a->z_head_stride : a->z_token_stride, a->z_head_stride};
    p.rows = (uint32_t)(a->tokens * a->heads), p.dim = (int)a->dim;
    p.dtype = a->dtype, p.weight_dtype = a->weight_dtype, p.act = a->activation, p.eps = a->eps;
    p.vec = v.ok;
    return done(launch_gated_norm_fwd(p, (cudaStream_t)stream));
}

gdr_status gdr_gated_norm_bwd(const gdr_gated_norm_bwd_args *a, void *stream_) {
    if (!a) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    const gdr_status st = norm_sizes(a->tokens, a->heads, a->dim);
    if (st != GDR_OK) return st;
    if (!type_ok(a->dtype) || ((a->weight || a->dweight) && !type_ok(a->weight_dtype)) ||
        (a->activation != 0 && a->activation != 1))
        return GDR_ERR_INVALID_ARG;
    if ((a->dweight && !a->weight) || (a->dz && !a->z)) return GDR_ERR_INVALID_ARG;
    if (a->dweight && !at(a->dweight, type_size(a->weight_dtype))) return GDR_ERR_INVALID_ARG;
    if (a->tokens == 0) return clear_sum(a->dweight, a->dim, a->weight_dtype, stream);
    if (!a->dy || !a->x || !a->dx || (a->z && !a->dz)) return GDR_ERR_INVALID_ARG;
    if (a->dweight && (!a->workspace || !at(a->workspace, 16) ||
                       a->workspace_bytes < gdr_norm_workspace_bytes(a->tokens * a->heads, a->dim, 1)))
        return GDR_ERR_INVALID_ARG;
    if (a->x_token_stride < 0 || a->x_head_stride < 0 || a->z_token_stride < 0 || a->z_head_stride < 0 ||
        a->dy_token_stride < 0 || a->dy_head_stride < 0)
        return GDR_ERR_INVALID_ARG;
    VecRule v(16 / type_size(a->dtype), a->dim);
    v.tensor(a->dy, a->dtype, a->dy_token_stride, a->dy_head_stride);
    v.tensor(a->x, a->dtype, a->x_token_stride, a->x_head_stride);
    v.tensor(a->z, a->dtype, a->z_token_stride, a->z_head_stride);
    v.tensor(a->dx, a->dtype, a->dim);
    v.tensor(a->dz, a->dtype, a->dim);
    if (!v.natural || (a->weight && !at(a->weight, type_size(a->weight_dtype)))) return GDR_ERR_INVALID_ARG;
    GatedNormParams p = {};
    p.dy = a->dy, p.x = a->x, p.z = a->z, p.weight = a->weight;
    p.dx = a->dx, p.dz = a->dz, p.dweight = a->dweight, p.part = (float *)a->workspace;
    const bool flat = collapses(a->x_token_stride, a->x_head_stride, a->tokens, a->heads) &&
                      collapses(a->dy_token_stride, a->dy_head_stride, a->tokens, a->heads) &&
                      (!a->z || collapses(a->z_token_stride, a->z_head_stride, a->tokens, a->heads));
    p.heads = FastDiv::of(flat ? 1 : (uint32_t)a->heads);
    p.dym = {flat && a->heads > 1 ? a->dy_head_stride : a->dy_token_stride, a->dy_head_stride};
    p.xm = {flat && a->heads > 1 ? a->x_head_stride : a->x_token_stride, a->x_head_stride};
    p.zm = {flat && a->heads > 1 ? a->z_head_stride : a->z_token_stride, a->z_head_stride};
    p.rows = (uint32_t)(a->tokens * a->heads), p.dim = (int)a->dim;
    p.dtype = a->dtype, p.weight_dtype = a->weight_dtype, p.act = a->activation, p.eps = a->eps;
    p.vec = v.ok;
    return done(launch_gated_norm_bwd(p, stream));
}

gdr_status gdr_add_norm_fwd(const gdr_add_norm_fwd_args *a, void *stream) {
    if (!a) return GDR_ERR_INVALID_ARG;
    const gdr_status st = norm_sizes(a->tokens, 1, a->dim);
    if (st != GDR_OK) return st;
    if (!type_ok(a->dtype) || (a->residual_dtype != a->dtype && a->residual_dtype != GDR_F32) ||
        (a->weight && !type_ok(a->weight_dtype)) || (a->scale_vec && !type_ok(a->scale_dtype)))
        return GDR_ERR_INVALID_ARG;
    if (a->tokens == 0) return GDR_OK;
    if (!a->x || !a->y) return GDR_ERR_INVALID_ARG;
    if (a->x_token_stride < 0 || a->residual_token_stride < 0 ||
        (a->residual_out && !(a->tokens <= 1 || a->residual_out_token_stride >= a->dim)))
        return GDR_ERR_INVALID_ARG;
    VecRule v(16 / type_size(a->dtype), a->dim);
    v.tensor(a->x, a->dtype, a->x_token_stride);
    v.tensor(a->residual, a->residual_dtype, a->residual_token_stride);
    v.tensor(a->residual_out, a->residual_dtype, a->residual_out_token_stride);
    v.tensor(a->y, a->dtype, a->dim);
    if (!v.natural || (a->weight && !at(a->weight, type_size(a->weight_dtype))) ||
        (a->scale_vec && !at(a->scale_vec, type_size(a->scale_dtype))))
        return GDR_ERR_INVALID_ARG;
    AddNormParams p = {};
    p.x = a->x, p.residual = a->residual, p.weight = a->weight, p.scale_vec = a->scale_vec;
    p.y = a->y, p.residual_out = a->residual_out;
    p.x_ts = a->x_token_stride, p.r_ts = a->residual_token_stride, p.ro_ts = a->residual_out_token_stride;
    p.rows = (uint32_t)a->tokens, p.dim = (int)a->dim;
    p.dtype = a->dtype, p.residual_dtype = a->residual_dtype;
    p.weight_dtype = a->weight_dtype, p.scale_dtype = a->scale_dtype;
    p.scale = a->scale, p.eps = a->eps;
    p.vec = v.ok;
    return done(launch_add_norm_fwd(p, (cudaStream_t)stream));
}

gdr_status gdr_add_norm_bwd(const gdr_add_norm_bwd_args *a, void *stream_) {
    if (!a) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    const gdr_status st = norm_sizes(a->tokens, 1, a->dim);
    if (st != GDR_OK) return st;
    if (!type_ok(a->dtype) || (a->residual_dtype != a->dtype && a->residual_dtype != GDR_F32) ||
        (a->weight && !type_ok(a->weight_dtype)) || (a->scale_vec && !type_ok(a->scale_dtype)))
        return GDR_ERR_INVALID_ARG;
    if ((a->dweight && !a->weight) || (a->dscale && !a->scale_vec)) return GDR_ERR_INVALID_ARG;
    if ((a->dweight && !at(a->dweight, type_size(a->weight_dtype))) ||
        (a->dscale && !at(a->dscale, type_size(a->scale_dtype))))
        return GDR_ERR_INVALID_ARG;
    if (a->tokens == 0) {
        const gdr_status e = clear_sum(a->dweight, a->dim, a->weight_dtype, stream);
        return e != GDR_OK ? e : clear_sum(a->dscale, a->dim, a->scale_dtype, stream);
    }
    if (!a->dy || !a->residual_out || (a->dscale && !a->x)) return GDR_ERR_INVALID_ARG;
    const int sums = (a->dweight ? 1 : 0) + (a->dscale ? 1 : 0);
    if (sums && (!a->workspace || !at(a->workspace, 16) ||
                 a->workspace_bytes < gdr_norm_workspace_bytes(a->tokens, a->dim, sums)))
        return GDR_ERR_INVALID_ARG;
    if (a->dy_token_stride < 0 || a->dres_token_stride < 0 || a->residual_out_token_stride < 0 || a->x_token_stride < 0)
        return GDR_ERR_INVALID_ARG;
    VecRule v(16 / type_size(a->dtype), a->dim);
    v.tensor(a->dy, a->dtype, a->dy_token_stride);
    v.tensor(a->dres, a->residual_dtype, a->dres_token_stride);
    v.tensor(a->residual_out, a->residual_dtype, a->residual_out_token_stride);
    if (a->dscale) v.tensor(a->x, a->dtype, a->x_token_stride);
    v.tensor(a->dx, a->dtype, a->dim);
    v.tensor(a->dresidual, a->residual_dtype, a->dim);
    if (!v.natural || (a->weight && !at(a->weight, type_size(a->weight_dtype))) ||
        (a->scale_vec && !at(a->scale_vec, type_size(a->scale_dtype))))
        return GDR_ERR_INVALID_ARG;
    AddNormParams p = {};
    p.dy = a->dy, p.dres = a->dres, p.x = a->x, p.weight = a->weight, p.scale_vec = a->scale_vec;
    p.residual_out = const_cast<void *>(a->residual_out);
    p.dx = a->dx, p.dresidual = a->dresidual, p.dweight = a->dweight, p.dscale = a->dscale;
    p.part = (float *)a->workspace;
    p.dy_ts = a->dy_token_stride, p.dres_ts = a->dres_token_stride, p.x_ts = a->x_token_stride;
    p.ro_ts = a->residual_out_token_stride;
    p.rows = (uint32_t)a->tokens, p.dim = (int)a->dim;
    p.dtype = a->dtype, p.residual_dtype = a->residual_dtype;
    p.weight_dtype = a->weight_dtype, p.scale_dtype = a->scale_dtype;
    p.scale = a->scale, p.eps = a->eps;
    p.vec = v.ok;
    return done(launch_add_norm_bwd(p, stream));
}

// ---------------------------------------------------------------- gated linear recurrence
size_t gdr_linrec_workspace_bytes(int64_t rows, int64_t dim) {
    if (rows < 0 || rows > kMaxRows || dim < 1) return 0;
    return 256;  // the status word
}

static gdr_status linrec_sizes(int64_t batch, int64_t tokens, int64_t dim, int64_t num_seqs, int dtype, int gate_dtype,
                               int complement) {
    if (batch < 1 || tokens < 0 || dim < 1 || num_seqs < 0 || (num_seqs > 0 && batch != 1)) return GDR_ERR_INVALID_ARG;
    if (!type_ok(dtype) || (gate_dtype != dtype && gate_dtype != GDR_F32) || (complement != 0 && complement != 1))
        return GDR_ERR_INVALID_ARG;
    if (batch > kMaxRows || tokens > kMaxRows || batch * tokens > kMaxRows || dim > (1 << 20) || num_seqs > (1 << 24))
        return GDR_ERR_UNSUPPORTED;
    return GDR_OK;
}

// Rows that a tensor map can describe: apart from each other, at a distance that its 40 bits hold.
static bool map_rows(int64_t stride, int64_t rows, int64_t dim) {
    return rows <= 1 || (stride >= dim && stride < (1ll << 36));
}

static uint32_t spin_limit() {
    const char *spin = getenv("GDR_SPIN_LIMIT");  // a test knob, as for the delta rule's plans
    return spin && atol(spin) > 0 ? (uint32_t)atol(spin) : WAIT_LIMIT_DEFAULT;
}

gdr_status gdr_linrec_fwd(const gdr_linrec_fwd_args *a, void *stream_) {
    if (!a) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    const gdr_status st =
        linrec_sizes(a->batch, a->tokens, a->dim, a->num_seqs, a->dtype, a->gate_dtype, a->complement);
    if (st != GDR_OK) return st;
    const int64_t rows = a->batch * a->tokens;
    if ((rows > 0 && (!a->x || !a->g)) || (a->num_seqs > 0 && !a->cu_seqlens)) return GDR_ERR_INVALID_ARG;
    if (a->x_token_stride < 0 || a->g_token_stride < 0) return GDR_ERR_INVALID_ARG;
    if (!a->workspace || !at(a->workspace, 256) || a->workspace_bytes < gdr_linrec_workspace_bytes(rows, a->dim))
        return GDR_ERR_INVALID_ARG;
    if (!at(a->h0, 4) || !at(a->ht, 4) || !at(a->states, 4) || !at(a->cu_seqlens, 4)) return GDR_ERR_INVALID_ARG;
    VecRule v(8, a->dim, 4);  // tensor maps take multiples of 16 bytes, lanes have 4 channels at most
    v.tensor(a->x, a->dtype, a->x_token_stride);
    v.tensor(a->g, a->gate_dtype, a->g_token_stride);
    v.tensor(a->h, a->dtype, a->dim);
    v.tensor(a->h0, GDR_F32, a->dim);
    v.tensor(a->ht, GDR_F32, a->dim);
    v.tensor(a->states, GDR_F32, a->dim);
    if (!v.natural) return GDR_ERR_INVALID_ARG;
    LinrecParams p = {};
    p.x = a->x, p.g = a->g, p.h0 = a->h0, p.cu = a->num_seqs > 0 ? a->cu_seqlens : nullptr;
    p.h = a->h, p.ht = a->ht, p.states = a->states;
    p.x_ts = a->x_token_stride, p.g_ts = a->g_token_stride;
    p.rows = (int)rows, p.tokens = (int)a->tokens, p.dim = (int)a->dim;
    p.N = (int)(a->num_seqs > 0 ? a->num_seqs : a->batch), p.complement = a->complement;
    p.dtype = a->dtype, p.gate_dtype = a->gate_dtype;
    p.vec = v.ok && rows > 0 && map_rows(a->x_token_stride, rows, a->dim) && map_rows(a->g_token_stride, rows, a->dim);
    Pieces x(a->dim), g(a->dim);
    x.tensor(a->x, a->dtype, a->x_token_stride), x.tensor(a->h, a->dtype, a->dim);
    g.tensor(a->g, a->gate_dtype, a->g_token_stride);
    p.x_piece = x.n, p.g_piece = g.n;
    p.status = (int *)a->workspace, p.spin = spin_limit();
    return done(launch_linrec_fwd(p, stream));
}

gdr_status gdr_linrec_bwd(const gdr_linrec_bwd_args *a, void *stream_) {
    if (!a) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    const gdr_status st =
        linrec_sizes(a->batch, a->tokens, a->dim, a->num_seqs, a->dtype, a->gate_dtype, a->complement);
    if (st != GDR_OK) return st;
    const int64_t rows = a->batch * a->tokens;
    if (rows > 0 && (!a->x || !a->g || !a->dh || !a->dx || !a->dg || !a->states)) return GDR_ERR_INVALID_ARG;
    if (a->num_seqs > 0 && !a->cu_seqlens) return GDR_ERR_INVALID_ARG;
    if (a->x_token_stride < 0 || a->g_token_stride < 0 || a->dh_token_stride < 0) return GDR_ERR_INVALID_ARG;
    if (!a->workspace || !at(a->workspace, 256) || a->workspace_bytes < gdr_linrec_workspace_bytes(rows, a->dim))
        return GDR_ERR_INVALID_ARG;
    if (!at(a->h0, 4) || !at(a->dht, 4) || !at(a->states, 4) || !at(a->dh0, 4) || !at(a->cu_seqlens, 4))
        return GDR_ERR_INVALID_ARG;
    VecRule v(8, a->dim, 4);  // tensor maps take multiples of 16 bytes, lanes have 4 channels at most
    v.tensor(a->x, a->dtype, a->x_token_stride);
    v.tensor(a->g, a->gate_dtype, a->g_token_stride);
    v.tensor(a->dh, a->dtype, a->dh_token_stride);
    v.tensor(a->dx, a->dtype, a->dim);
    v.tensor(a->dg, a->gate_dtype, a->dim);
    v.tensor(a->h0, GDR_F32, a->dim);
    v.tensor(a->dht, GDR_F32, a->dim);
    v.tensor(a->dh0, GDR_F32, a->dim);
    v.tensor(a->states, GDR_F32, a->dim);
    if (!v.natural) return GDR_ERR_INVALID_ARG;
    LinrecParams p = {};
    p.x = a->x, p.g = a->g, p.dh = a->dh, p.h0 = a->h0, p.dht = a->dht;
    p.cu = a->num_seqs > 0 ? a->cu_seqlens : nullptr;
    p.dx = a->dx, p.dg = a->dg, p.dh0 = a->dh0, p.states = const_cast<float *>(a->states);
    p.x_ts = a->x_token_stride, p.g_ts = a->g_token_stride, p.dh_ts = a->dh_token_stride;
    p.rows = (int)rows, p.tokens = (int)a->tokens, p.dim = (int)a->dim;
    p.N = (int)(a->num_seqs > 0 ? a->num_seqs : a->batch), p.complement = a->complement;
    p.dtype = a->dtype, p.gate_dtype = a->gate_dtype;
    p.vec = v.ok && rows > 0 && map_rows(a->x_token_stride, rows, a->dim) && map_rows(a->g_token_stride, rows, a->dim) &&
            map_rows(a->dh_token_stride, rows, a->dim);
    Pieces x(a->dim), g(a->dim);
    x.tensor(a->x, a->dtype, a->x_token_stride), x.tensor(a->dh, a->dtype, a->dh_token_stride);
    x.tensor(a->dx, a->dtype, a->dim);
    g.tensor(a->g, a->gate_dtype, a->g_token_stride), g.tensor(a->dg, a->gate_dtype, a->dim);
    p.x_piece = x.n, p.g_piece = g.n;
    p.status = (int *)a->workspace, p.spin = spin_limit();
    return done(launch_linrec_bwd(p, stream));
}

gdr_status gdr_linrec_get_status(void *workspace, void *stream_) {
    if (!workspace || !at(workspace, 256)) return GDR_ERR_INVALID_ARG;
    cudaStream_t stream = (cudaStream_t)stream_;
    int word = 0;
    // all of it on the caller's stream, and done on return: the workspace may be given away then
    if (cudaMemcpyAsync(&word, workspace, sizeof(int), cudaMemcpyDeviceToHost, stream) != cudaSuccess) return GDR_ERR_CUDA;
    if (cudaMemsetAsync(workspace, 0, sizeof(int), stream) != cudaSuccess) return GDR_ERR_CUDA;
    if (cudaStreamSynchronize(stream) != cudaSuccess) return GDR_ERR_CUDA;
    if (word & ST_TIMEOUT) return GDR_ERR_TIMEOUT;
    return word & ST_BAD_SEQLENS ? GDR_ERR_DEVICE : GDR_OK;
}

gdr_status gdr_linrec_step(const gdr_linrec_step_args *a, void *stream) {
    if (!a) return GDR_ERR_INVALID_ARG;
    if (a->batch < 0 || a->dim < 1 || a->num_slots < 0 || !type_ok(a->dtype) ||
        (a->gate_dtype != a->dtype && a->gate_dtype != GDR_F32) || (a->complement != 0 && a->complement != 1))
        return GDR_ERR_INVALID_ARG;
    if (a->dim > (1 << 20) || a->num_slots > 0x7fffffffll || a->batch > kMaxRows || a->batch * a->dim > kMaxRows)
        return GDR_ERR_UNSUPPORTED;
    if (!a->slots && a->num_slots < a->batch) return GDR_ERR_INVALID_ARG;
    if (a->batch == 0) return GDR_OK;
    if (!a->x || !a->g || !a->y || (a->num_slots > 0 && !a->state)) return GDR_ERR_INVALID_ARG;
    if (a->x_token_stride < 0 || a->g_token_stride < 0 || !at(a->slots, 4) || !at(a->state, 4))
        return GDR_ERR_INVALID_ARG;
    VecRule v(4, a->dim);
    v.tensor(a->x, a->dtype, a->x_token_stride);
    v.tensor(a->g, a->gate_dtype, a->g_token_stride);
    v.tensor(a->y, a->dtype, a->dim);
    v.tensor(a->state, GDR_F32, a->dim);
    if (!v.natural) return GDR_ERR_INVALID_ARG;
    StepParams p = {};
    p.x = a->x, p.g = a->g, p.slots = a->slots, p.state = a->state, p.y = a->y;
    p.x_ts = a->x_token_stride, p.g_ts = a->g_token_stride, p.batch = a->batch, p.num_slots = a->num_slots;
    p.dim = (int)a->dim, p.dtype = a->dtype, p.gate_dtype = a->gate_dtype, p.complement = a->complement;
    p.vec = v.ok;
    return done(launch_linrec_step(p, (cudaStream_t)stream));
}

// ---------------------------------------------------------------- gradient norm and clip
size_t gdr_clip_workspace_bytes(int64_t count, int64_t elements) {
    if (count < 0 || elements < 0) return 0;
    const int64_t launches = count / CLIP_TENSORS + 1;
    return sizeof(double) * (size_t)launches * CLIP_CTAS;
}

static gdr_status clip_impl(const gdr_clip_args *a, bool scale, cudaStream_t stream) {
    if (!a || a->count < 0 || !a->norm || !at(a->norm, 4)) return GDR_ERR_INVALID_ARG;
    if (scale && !(a->max_norm >= 0.f)) return GDR_ERR_INVALID_ARG;
    if (scale && !(a->eps >= 0.f)) return GDR_ERR_INVALID_ARG;
    if (a->count > 0 && (!a->grads || !a->sizes || !a->dtypes || (scale && a->outs && !a->out_dtypes)))
        return GDR_ERR_INVALID_ARG;
    int64_t total = 0;
    for (int64_t i = 0; i < a->count; ++i) {
        const int64_t n = a->sizes[i];
        if (n < 0 || !type_ok(a->dtypes[i])) return GDR_ERR_INVALID_ARG;
        if (n > (1ll << 46) || total > (1ll << 46)) return GDR_ERR_UNSUPPORTED;
        total += n;
        if (n == 0) continue;
        if (!a->grads[i] || !at(a->grads[i], type_size(a->dtypes[i]))) return GDR_ERR_INVALID_ARG;
        if (scale && a->outs &&
            (!type_ok(a->out_dtypes[i]) || !a->outs[i] || !at(a->outs[i], type_size(a->out_dtypes[i]))))
            return GDR_ERR_INVALID_ARG;
        if (scale && a->outs && a->outs[i] == a->grads[i] && a->out_dtypes[i] != a->dtypes[i]) return GDR_ERR_INVALID_ARG;
    }
    if (!a->workspace || !at(a->workspace, 16) || a->workspace_bytes < gdr_clip_workspace_bytes(a->count, total))
        return GDR_ERR_INVALID_ARG;
    double *part = (double *)a->workspace;
    std::unique_ptr<ClipTable<CLIP_TENSORS>> t(new (std::nothrow) ClipTable<CLIP_TENSORS>);
    if (!t) return GDR_ERR_OOM;
    int parts = 0;
    for (int pass = 0; pass < (scale ? 2 : 1); ++pass) {
        for (int64_t i = 0; i < a->count || (pass == 1 && i == 0);) {
            t->count = 0, t->pieces = 0;
            for (; i < a->count && t->count < CLIP_TENSORS; ++i) {
                if (a->sizes[i] == 0) continue;
                const int k = t->count++;
                t->grad[k] = a->grads[i];
                t->out[k] = a->outs ? a->outs[i] : const_cast<void *>(a->grads[i]);
                t->size[k] = a->sizes[i];
                t->dtype[k] = (uint8_t)a->dtypes[i];
                t->out_dtype[k] = (uint8_t)(scale && a->outs ? a->out_dtypes[i] : a->dtypes[i]);
                t->first[k] = t->pieces;
                t->pieces += (a->sizes[i] + CLIP_PIECE - 1) / CLIP_PIECE;
            }
            t->first[t->count] = t->pieces;
            cudaError_t e = cudaSuccess;
            if (pass == 0 && i == a->count && parts == 0 && clip_is_small(*t))
                return done(launch_clip_small(*t, a->norm, scale, a->max_norm, a->eps, stream));
            if (pass == 0) {
                if (t->pieces == 0) continue;
                const int n = (int)(t->pieces < CLIP_CTAS ? t->pieces : CLIP_CTAS);
                e = launch_clip_sumsq(*t, part + parts, n, stream);
                parts += n;
            } else {
                e = launch_clip_scale(*t, part, parts, a->norm, a->max_norm, a->eps, stream);
            }
            if (e != cudaSuccess) return GDR_ERR_CUDA;
            if (a->count == 0) break;
        }
    }
    if (!scale) return done(launch_clip_norm(part, parts, a->norm, stream));
    return GDR_OK;
}

gdr_status gdr_clip_grad_norm(const gdr_clip_args *a, void *stream) { return clip_impl(a, true, (cudaStream_t)stream); }
gdr_status gdr_grad_norm(const gdr_clip_args *a, void *stream) { return clip_impl(a, false, (cudaStream_t)stream); }

}  // extern "C"
