/*
 * gdr_block.h -- C ABI of the operators around the delta rule (libgdrbwd.so): the norms before and after a
 * block, the gated linear recurrence with its backward and its single-token step, and the gradient clip that
 * closes a training step.
 *
 * Conventions are those of gdr_bwd.h: plain device pointers owned by the caller, every call asynchronous on the
 * caller's stream and returning a gdr_status, arguments checked on the host before anything is launched
 * (GDR_ERR_INVALID_ARG, or GDR_ERR_UNSUPPORTED for a valid request outside the limits named here), no device
 * memory allocated by the library, outputs fully overwritten.  Sums, norms and states are held in fp32; an
 * output of a 16-bit type is rounded once, to nearest even.  All results are bit-identical from run to run.
 *
 * Rows: the last axis of every tensor is contiguous; a "token stride" or "head stride" is the distance in
 * elements from one token or head to the next.  Pointers are aligned to their element type.  Rows whose
 * pointers, strides and widths are multiples of 16 bytes are moved in 16-byte pieces, others element by element (by
 * the recurrence in pieces of 4 or 2 elements where those are aligned).
 * Outputs without a stride argument are contiguous.  Inputs and outputs must not overlap unless said.
 * A call with no tokens (or no elements) is valid: sums over tokens are then zero.
 */
#ifndef GDR_BLOCK_H_
#define GDR_BLOCK_H_

#include "gdr_bwd.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Longest normalised row. */
#define GDR_NORM_MAX_DIM 16384

typedef enum { GDR_ACT_SILU = 0, GDR_ACT_SIGMOID = 1 } gdr_activation;

/* ---- Norm after a block, fused with its output gate, over each head of `dim` channels:
 *     y = weight * x / sqrt(mean(x^2) + eps) * act(z)
 * x, z, y, dy, dx, dz: [tokens, heads, dim] in `dtype`; weight, dweight: [dim] in weight_dtype.
 * weight NULL means 1 (dweight must be NULL too); z NULL means no gate (dz must be NULL too). */
typedef struct {
    const void *x, *z, *weight;
    void *y;
    int64_t tokens, heads, dim;
    int64_t x_token_stride, x_head_stride, z_token_stride, z_head_stride;
    int32_t dtype, weight_dtype, activation;
    float eps;
} gdr_gated_norm_fwd_args;
gdr_status gdr_gated_norm_fwd(const gdr_gated_norm_fwd_args *args, void *stream);

/* Gradients of sum(y * dy).  dweight may be NULL (not returned); with it, `workspace` holds
 * gdr_norm_workspace_bytes(tokens * heads, dim, 1) bytes, 16-byte aligned. */
typedef struct {
    const void *dy, *x, *z, *weight;
    void *dx, *dz, *dweight, *workspace;
    int64_t tokens, heads, dim;
    int64_t dy_token_stride, dy_head_stride, x_token_stride, x_head_stride, z_token_stride, z_head_stride;
    uint64_t workspace_bytes;
    int32_t dtype, weight_dtype, activation;
    float eps;
} gdr_gated_norm_bwd_args;
gdr_status gdr_gated_norm_bwd(const gdr_gated_norm_bwd_args *args, void *stream);

/* ---- Norm before a block, fused with the residual stream that it reads:
 *     r' = residual + scale * x ,     y = weight * r' / sqrt(mean(r'^2) + eps)
 * x, y [tokens, dim] in dtype; residual, residual_out = r' [tokens, dim] in residual_dtype (dtype or GDR_F32);
 * y is formed from r' before its rounding.  residual NULL: the stream starts here, r' = scale * x.
 * scale_vec [dim] in scale_dtype, or NULL: the number `scale`.  weight NULL means 1.  residual_out may be
 * `residual` itself (same stride), or NULL (not returned). */
typedef struct {
    const void *x, *residual, *weight, *scale_vec;
    void *y, *residual_out;
    int64_t tokens, dim, x_token_stride, residual_token_stride, residual_out_token_stride;
    int32_t dtype, residual_dtype, weight_dtype, scale_dtype;
    float scale, eps;
} gdr_add_norm_fwd_args;
gdr_status gdr_add_norm_fwd(const gdr_add_norm_fwd_args *args, void *stream);

/* Gradients of sum(y * dy) + sum(r' * dres), taken at the stored residual_out:
 *     dresidual = d r' (residual_dtype),  dx = scale * dresidual (dtype),  dweight [dim] (weight_dtype),
 *     dscale [dim] (scale_dtype) = sum over tokens of dresidual * x.
 * dres NULL means zero.  x is read for dscale alone.  dx, dresidual, dweight and dscale may each be NULL (not
 * returned); dscale needs scale_vec and x, dweight needs weight.  With n of dweight and dscale wanted,
 * `workspace` holds gdr_norm_workspace_bytes(tokens, dim, n) bytes, 16-byte aligned. */
typedef struct {
    const void *dy, *dres, *residual_out, *x, *weight, *scale_vec;
    void *dx, *dresidual, *dweight, *dscale, *workspace;
    int64_t tokens, dim, dy_token_stride, dres_token_stride, residual_out_token_stride, x_token_stride;
    uint64_t workspace_bytes;
    int32_t dtype, residual_dtype, weight_dtype, scale_dtype;
    float scale, eps;
} gdr_add_norm_bwd_args;
gdr_status gdr_add_norm_bwd(const gdr_add_norm_bwd_args *args, void *stream);

/* Workspace of the two backward calls for `sums` column sums over `rows` rows of `dim` (0 for bad sizes). */
size_t gdr_norm_workspace_bytes(int64_t rows, int64_t dim, int sums);

/* ---- Gated linear recurrence, for every channel by itself:
 *     h_t = a_t h_{t-1} + b_t ,   a_t = exp(g_t) ,   b_t = x_t   or (complement)   (1 - a_t) x_t
 * x, h [batch, tokens, dim] in dtype, g [batch, tokens, dim] (raw log-gate) in gate_dtype (dtype or GDR_F32);
 * h0, ht [N, dim] fp32: the state before the first and after the last token of each sequence, h0 NULL means
 * zero, ht NULL not returned.  N = batch, or num_seqs when > 0 (varlen: batch 1, cu_seqlens as in gdr_bwd.h;
 * empty sequences give ht = h0).  batch * tokens is at most 2^30.
 * Gates are taken to [-88, 88.3] (16-bit ones to [-88, 88]); below -87.7 a is 0.  What the decays of up to 256
 * successive rows leave of a state below 2^-126 of it counts as zero.  Gates above 0 grow: channels that have
 * such, or whose states become infinite, are followed token by token, several times slower; a state that becomes
 * infinite may be a nan instead in the rest of a sequence that ends within 256 rows.
 * states, if not NULL: fp32 [ceil(batch tokens / GDR_LINREC_SAVE), dim], the state that enters each GDR_LINREC_SAVE
 * rows (of no meaning where a sequence starts on the first of them); the backward takes them.  h may be NULL (states and ht alone).
 * workspace: gdr_linrec_workspace_bytes(batch * tokens, dim) bytes, 256-byte aligned, not used by another call
 * that may run at the same time.  Malformed cu_seqlens and waits that expire are read with
 * gdr_linrec_get_status. */
#define GDR_LINREC_SAVE 16
typedef struct {
    const void *x, *g;
    const float *h0;
    const int32_t *cu_seqlens;
    void *h;
    float *ht, *states;
    void *workspace;
    int64_t batch, tokens, dim, num_seqs, x_token_stride, g_token_stride;
    uint64_t workspace_bytes;
    int32_t dtype, gate_dtype, complement, reserved;
} gdr_linrec_fwd_args;
gdr_status gdr_linrec_fwd(const gdr_linrec_fwd_args *args, void *stream);

/* Gradients of sum(h * dh) + sum(ht * dht): dx (dtype), dg (gate_dtype), dh0 fp32 [N, dim] or NULL.
 * states is what the forward call on the same x, g, h0 wrote.  dht NULL means zero. */
typedef struct {
    const void *x, *g, *dh;
    const float *h0, *dht, *states;
    const int32_t *cu_seqlens;
    void *dx, *dg;
    float *dh0;
    void *workspace;
    int64_t batch, tokens, dim, num_seqs, x_token_stride, g_token_stride, dh_token_stride;
    uint64_t workspace_bytes;
    int32_t dtype, gate_dtype, complement, reserved;
} gdr_linrec_bwd_args;
gdr_status gdr_linrec_bwd(const gdr_linrec_bwd_args *args, void *stream);

size_t gdr_linrec_workspace_bytes(int64_t rows, int64_t dim);

/* As gdr_bwd_get_status, for the last recurrence call on this workspace: synchronises `stream`, returns GDR_OK,
 * GDR_ERR_TIMEOUT or GDR_ERR_DEVICE and clears the word. */
gdr_status gdr_linrec_get_status(void *workspace, void *stream);

/* One token for each of `batch` sequences: state = a state + b in place, y = state (dtype).
 * x, y [batch, dim] in dtype, g [batch, dim] in gate_dtype, state fp32 [num_slots, dim].  Sequence i owns row
 * slots[i] of state (int32, device; NULL: row i, num_slots >= batch).  A slot that is negative or not below
 * num_slots is skipped: its y row is zero.  The other slots must be distinct. */
typedef struct {
    const void *x, *g;
    const int32_t *slots;
    float *state;
    void *y;
    int64_t batch, dim, num_slots, x_token_stride, g_token_stride;
    int32_t dtype, gate_dtype, complement, reserved;
} gdr_linrec_step_args;
gdr_status gdr_linrec_step(const gdr_linrec_step_args *args, void *stream);

/* ---- Global gradient norm over `count` tensors, and clipping:
 *     norm = sqrt(sum of all squares) ,   out_i = grad_i * min(1, max_norm / (norm + eps))
 * grads, outs, sizes, dtypes, out_dtypes: host arrays of `count` entries (read before the call returns); the
 * tensors themselves are contiguous device memory and may be empty.  outs NULL: in place (out_dtypes unused);
 * an entry of outs may be the same entry of grads when the types agree.  norm: one fp32 on the device.
 * A norm that is not finite gives what the formula gives: all finite gradients become 0 for an infinite norm,
 * everything becomes nan for a nan norm.  Squares are formed in fp32 and added in fp32 32 at a time, in fp64 from there:
 * a value above 1.8e19 makes the norm infinite, values below 1e-23 count as zero.  gdr_grad_norm computes the norm
 * alone.
 * workspace: gdr_clip_workspace_bytes(count, total number of elements) bytes, 16-byte aligned. */
typedef struct {
    const void *const *grads;
    void *const *outs;
    const int64_t *sizes;
    const int32_t *dtypes, *out_dtypes;
    float *norm;
    void *workspace;
    int64_t count;
    uint64_t workspace_bytes;
    float max_norm, eps;
} gdr_clip_args;
gdr_status gdr_clip_grad_norm(const gdr_clip_args *args, void *stream);
gdr_status gdr_grad_norm(const gdr_clip_args *args, void *stream);
size_t gdr_clip_workspace_bytes(int64_t count, int64_t elements);

#ifdef __cplusplus
}
#endif

#endif /* GDR_BLOCK_H_ */
