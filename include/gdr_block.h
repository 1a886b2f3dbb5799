/*
 * gdr_block.h -- C ABI of the operators around the delta rule (libgdrbwd.so): the norms before and after a
 * block, the gated linear recurrence with its backward and its single-token step, the gradient clip that
 * closes a training step, the rule itself token by token on a pool of states, such states kept in 8 bits, and
 * the gated feed-forward with its backward.
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

/* ---- The gated delta rule token by token, on a pool of states (the recurrent form of gdr_fwd_run's rule): for each of
 * `batch` sequences, each value head h (key head h / (v_heads / k_heads)) and each of its tokens in turn
 *     S' = S diag(exp(g)) ,   S = S' + beta (v - S' k) k^T ,   o = scale S q
 * q, k [batch, tokens, k_heads, K], v, o [batch, tokens, v_heads, V] in dtype; beta [batch, tokens, v_heads] in beta_dtype
 * (dtype or GDR_F32); g fp32 [batch, tokens, v_heads], or with gate_per_channel [batch, tokens, v_heads, K]: the raw
 * log-gates, <= 0 (products of exp(g) over up to 8 successive tokens are formed, and must not leave fp32).  A state or input
 * that is not finite makes the rows that it meets not finite.
 * K and V are multiples of 8 up to 128.  scale 0 means 1 / sqrt(K).  `batch tokens` rows lie at one distance ("token stride").
 * state: fp32 [num_slots] times [v_heads, V, K], each contiguous and 16-byte aligned, state_slot_stride apart.
 * Sequence i owns state slots[i] (int32, device; NULL: state i, num_slots >= batch).  A slot that is negative or not below
 * num_slots is skipped, with zero rows of o.  The other slots must be distinct when update is 1.
 * lengths (int32 [batch], device; NULL: all `tokens`): the first lengths[i] tokens, taken to [0, tokens], of sequence i are
 * used; the rows of o behind them are zero.  update 0 leaves the pool as it was: the outputs of drafted tokens.  q and o NULL
 * (with update 1): the states alone.  With `lengths` the number of accepted tokens, that moves them over the accepted ones. */
typedef struct {
    const void *q, *k, *v, *beta;
    const float *g;
    float *state;
    const int32_t *slots, *lengths;
    void *o;
    int64_t batch, tokens, k_heads, v_heads, K, V, num_slots, state_slot_stride;
    int64_t q_token_stride, q_head_stride, k_token_stride, k_head_stride, v_token_stride, v_head_stride;
    int64_t beta_token_stride, g_token_stride, g_head_stride;
    int32_t dtype, beta_dtype, gate_per_channel, update;
    float scale;
} gdr_step_args;
gdr_status gdr_step(const gdr_step_args *args, void *stream);

/* ---- States kept in 8 bits: of each pair i < count, state slots[i] of a pool is written to entry entries[i] of a cache, or
 * read back from it.  A state is `rows` contiguous rows of `width` fp32 values, state_slot_stride apart; an entry is as many
 * codes (cache_stride apart, in codes) and a scale for each row (scales_stride apart).  Each row has
 *     scale = 2^e ,  e = the least integer >= -126 with max |x| <= Q 2^e ,   code = round(x / scale) ,   x ~ code scale
 * with codes int8 and Q = 127 (GDR_CODE_INT8) or e4m3 and Q = 448 (GDR_CODE_E4M3); ties go to even, and a code whose
 * value would leave fp32 (2^128) is the next smaller one.  A state that was read
 * back and is saved again gives the same values.  A row with a value that is not finite gets the scale nan, and reads
 * back as nan.  slots, entries: int32, device, or NULL: i.  Pairs with a slot or an entry out of range are skipped.
 * What a call writes to (entries of a save, slots of a load) must be distinct; what it reads from need not be. */
typedef enum { GDR_CODE_INT8 = 0, GDR_CODE_E4M3 = 1 } gdr_code;
typedef struct {
    float *state;
    void *cache;
    float *scales;
    const int32_t *slots, *entries;
    int64_t count, rows, width, num_slots, num_entries, state_slot_stride, cache_stride, scales_stride;
    int32_t code, reserved;
} gdr_state_cache_args;
gdr_status gdr_save_states(const gdr_state_cache_args *args, void *stream);
gdr_status gdr_load_states(const gdr_state_cache_args *args, void *stream);

/* ---- Gated feed-forward: both projections, the activation and the product,
 *     g = x w_gate^T ,   u = x w_up^T ,   h = act(g) u
 * x [tokens, dim], w_gate, w_up [inner, dim] (rows at a "row stride"), h [tokens, inner], all in dtype: GDR_BF16 or GDR_F16
 * (GDR_F32 is GDR_ERR_UNSUPPORTED).  Products are summed in fp32.  Activations: silu, sigmoid, gelu with the tanh
 * formula, g (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) / 2.
 * gate, up fp32 [tokens, inner], both or neither (NULL): g and u for the backward.  h may be NULL with them.
 * workspace: gdr_ffn_workspace_bytes bytes, 256-byte aligned, not used by another call that may run at the same time; NULL
 * where that is 0, or GDR_FFN_STATUS_BYTES: the status alone.  Waits that expire are read with gdr_ffn_get_status; calls in which
 * nothing waits (few tokens, none, or no result wanted) clear the status of a workspace
 * of GDR_FFN_STATUS_BYTES or more that they are given all the same. */
#define GDR_FFN_MAX_DIM (1 << 20)
/* Forward calls of up to so many tokens take no workspace. */
#define GDR_FFN_FEW_TOKENS 32
#define GDR_FFN_STATUS_BYTES 256
typedef enum { GDR_FFN_SILU = 0, GDR_FFN_SIGMOID = 1, GDR_FFN_GELU_TANH = 2 } gdr_ffn_activation;
typedef struct {
    const void *x, *w_gate, *w_up;
    void *h;
    float *gate, *up;
    void *workspace;
    int64_t tokens, dim, inner, x_token_stride, w_gate_row_stride, w_up_row_stride;
    uint64_t workspace_bytes;
    int32_t dtype, activation;
} gdr_ffn_fwd_args;
gdr_status gdr_ffn_fwd(const gdr_ffn_fwd_args *args, void *stream);

/* Gradients of sum(h * dh): with dg = dh u act'(g) and du = dh act(g), rounded to dtype (and within its range),
 *     dx = dg w_gate + du w_up [tokens, dim] ,   dw_gate = dg^T x ,  dw_up = du^T x [inner, dim]   (all in dtype)
 * gate and up are what the forward call wrote.  dx may be NULL (not returned, the weights are not read), and so may dw_gate
 * and dw_up together (x is not read). */
typedef struct {
    const void *dh, *x, *w_gate, *w_up;
    const float *gate, *up;
    void *dx, *dw_gate, *dw_up, *workspace;
    int64_t tokens, dim, inner, dh_token_stride, x_token_stride, w_gate_row_stride, w_up_row_stride;
    uint64_t workspace_bytes;
    int32_t dtype, activation;
} gdr_ffn_bwd_args;
gdr_status gdr_ffn_bwd(const gdr_ffn_bwd_args *args, void *stream);

/* Workspace of a forward (backward 0) or backward call.  copies: whether any of x, w_gate and w_up has rows that do not all
 * start at multiples of 16 bytes (such are brought there first).  0 for bad sizes, and for forward calls of few tokens. */
size_t gdr_ffn_workspace_bytes(int64_t tokens, int64_t dim, int64_t inner, int copies, int backward);

/* Of the last feed-forward call on this workspace: synchronises `stream`, returns GDR_OK or GDR_ERR_TIMEOUT and clears the
 * status, the workspace's first GDR_FFN_STATUS_BYTES. */
gdr_status gdr_ffn_get_status(void *workspace, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_BLOCK_H_ */
