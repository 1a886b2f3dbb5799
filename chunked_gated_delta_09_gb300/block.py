"""Torch-facing calls of the operators around the delta rule (include/gdr_block.h):

* ``gated_norm``  y = weight * x / rms(x) * act(z) over each head: the norm after a block, with its output gate;
* ``add_norm``    r' = residual + scale * x, y = weight * r' / rms(r'): the residual stream and the norm before a block;
* ``linear_recurrence``  h_t = a_t h_{t-1} + b_t with a = exp(g), per channel; ``linrec_step`` does single tokens;
* ``clip_grad_norm`` / ``grad_norm``  the norm over many gradients, and clipping.

As in :mod:`ops`, everything is computed by libgdrbwd.so's kernels: this module checks tensors, allocates outputs and
workspace with torch and passes raw pointers.  ``*_fwd`` and ``*_bwd`` are the plain calls, the names without a suffix
are differentiable, once: a second derivative through them is an error.  ``stream`` (default: torch's current stream) queues the call there, with its outputs allocated for
that stream; the caller orders it after the work that made the inputs.
"""
from __future__ import annotations

import contextlib
from array import array
from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable
from torch.autograd.graph import increment_version

from . import _lib
from ._lib import GdrError

_DT = {torch.float32: _lib.GDR_F32, torch.bfloat16: _lib.GDR_BF16, torch.float16: _lib.GDR_F16}
_ACT = {"silu": 0, "sigmoid": 1}
_F32 = torch.float32

_pack_gated_fwd = _lib.packer(_lib.GdrGatedNormFwdArgs)
_pack_gated_bwd = _lib.packer(_lib.GdrGatedNormBwdArgs)
_pack_add_fwd = _lib.packer(_lib.GdrAddNormFwdArgs)
_pack_add_bwd = _lib.packer(_lib.GdrAddNormBwdArgs)
_pack_linrec_fwd = _lib.packer(_lib.GdrLinrecFwdArgs)
_pack_linrec_bwd = _lib.packer(_lib.GdrLinrecBwdArgs)
_pack_linrec_step = _lib.packer(_lib.GdrLinrecStepArgs)
_pack_clip = _lib.packer(_lib.GdrClipArgs)

# the current stream's handle as an integer; torch.cuda.current_stream builds an object first, at ten times the cost
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
if _raw_stream is None:  # pragma: no cover
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _need(ok: bool, what: str):
    if not ok:
        raise ValueError(what)


_entries = {}  # the library's functions by name, once it is loaded


def _entry(name: str):
    fn = _entries.get(name)
    if fn is None:
        fn = _entries[name] = getattr(_lib.load(), name)
    return fn


def _queue(name: str, packed: bytes, index: int):
    """Call the C entry on torch's current stream of device ``index``."""
    fn = _entry(name)
    if torch.cuda.current_device() != index:
        with torch.cuda.device(index):
            st = fn(packed, _raw_stream(index))
    else:
        st = fn(packed, _raw_stream(index))
    if st:
        raise GdrError(st, name)


@contextlib.contextmanager
def _on(stream, tensors):
    """Run a call on ``stream``: what is allocated inside belongs to it, and the inputs stay alive for it."""
    with torch.cuda.stream(stream):
        yield
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _cuda(x: torch.Tensor, name: str) -> int:
    if not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (the operators have no CPU path)")
    if x.dtype not in _DT:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    return x.get_device()


def _like(t: torch.Tensor, name: str, index: int, shape, *dtypes):
    if t.get_device() != index or t.shape != shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a tensor of shape {tuple(shape)} and type "
                         f"{' or '.join(str(d) for d in dtypes)} on cuda:{index}, "
                         f"got {tuple(t.shape)}, {t.dtype} on {t.device}")


def _vector(t: Optional[torch.Tensor], name: str, index: int, dim: int):
    if t is None:
        return
    if t.get_device() != index or t.dim() != 1 or t.shape[0] != dim or t.dtype not in _DT:
        raise ValueError(f"{name} must be a floating tensor [{dim}] on cuda:{index}")
    if dim > 1 and not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _token_stride(t: torch.Tensor, name: str) -> int:
    """Distance between the rows of [..., D] when they all lie at one distance from the next."""
    if t.is_contiguous():
        return t.shape[-1]
    return _strides(t, name, 1)[0]


def _strides(t: torch.Tensor, name: str, inner: int):
    """(distance between tokens, distance between heads) of [..., heads, D] (inner = 2) or [..., D] (inner = 1)."""
    shape = t.shape
    if t.is_contiguous():  # (so is a tensor without elements)
        dim = shape[-1]
        return (shape[-2] * dim, dim) if inner == 2 else (dim, dim)
    stride = t.stride()
    _need(shape[-1] == 1 or stride[-1] == 1, f"{name}: the last axis must be contiguous")
    lead, step, span = None, 0, 1  # span: tokens covered by the axes seen so far
    for n, s in zip(reversed(shape[:-inner]), reversed(stride[:-inner])):
        if n == 1:
            continue
        if lead is None:
            lead = step = s
        else:
            _need(s == lead * span, f"{name}: the axes before the {'heads' if inner == 2 else 'channels'} must lie at one "
                                    "distance (view them as one axis)")
        span *= n
    return step, (stride[-2] if inner == 2 else 0)


def _result(x: torch.Tensor) -> torch.Tensor:
    """An uninitialised contiguous tensor like x."""
    if x.is_contiguous():
        return torch.empty_like(x)
    return torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _ptr(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.data_ptr()


def _code(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else _DT[t.dtype]


# ---------------------------------------------------------------- norm after a block
def _gated_check(x, z, weight, activation):
    index = _cuda(x, "x")
    _need(x.dim() >= 2, "x must be [..., heads, D]")
    if z is not None:
        _like(z, "z", index, x.shape, x.dtype)
    _vector(weight, "weight", index, x.shape[-1])
    if activation not in _ACT:
        raise ValueError(f"activation must be one of {sorted(_ACT)}")
    return index


def gated_norm_fwd(x, z, weight, *, eps=1e-6, activation="silu", stream=None) -> torch.Tensor:
    """y = weight * x / sqrt(mean(x^2) + eps) * act(z) over the last axis.

    x, z [..., heads, D] of one type (fp32, bf16 or fp16), the last axis contiguous and the axes before the heads at
    one distance; z None: no gate; weight [D] of any of the types, or None (1).  ``activation``: "silu" or "sigmoid".
    Returns y like x, contiguous."""
    if stream is not None:
        with _on(stream, (x, z, weight)):
            return gated_norm_fwd(x, z, weight, eps=eps, activation=activation)
    index = _gated_check(x, z, weight, activation)
    heads, dim = x.shape[-2:]
    y = _result(x)
    n = x.numel()
    if n == 0:
        return y
    xs = _strides(x, "x", 2)
    zs = (0, 0) if z is None else _strides(z, "z", 2)
    _queue("gdr_gated_norm_fwd",
           _pack_gated_fwd(x.data_ptr(), _ptr(z), _ptr(weight), y.data_ptr(), n // (heads * dim), heads, dim, *xs, *zs,
                           _DT[x.dtype], _code(weight), _ACT[activation], eps), index)
    return y


def gated_norm_bwd(dy, x, z, weight, *, eps=1e-6, activation="silu", stream=None) -> dict:
    """Gradients of :func:`gated_norm_fwd`: dict(dx, dz, dweight), each like its input (None where that is None)."""
    if stream is not None:
        with _on(stream, (dy, x, z, weight)):
            return gated_norm_bwd(dy, x, z, weight, eps=eps, activation=activation)
    index = _gated_check(x, z, weight, activation)
    _like(dy, "dy", index, x.shape, x.dtype)
    heads, dim = x.shape[-2:]
    dev = x.device
    dx = _result(x)
    dz = None if z is None else _result(x)
    dw = None if weight is None else torch.empty(dim, dtype=weight.dtype, device=dev)
    n = x.numel()
    if n == 0:
        return dict(dx=dx, dz=dz, dweight=None if dw is None else dw.zero_())
    tokens = n // (heads * dim)
    nbytes = 0 if dw is None else _entry("gdr_norm_workspace_bytes")(tokens * heads, dim, 1)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    zs = (0, 0) if z is None else _strides(z, "z", 2)
    _queue("gdr_gated_norm_bwd",
           _pack_gated_bwd(dy.data_ptr(), x.data_ptr(), _ptr(z), _ptr(weight), dx.data_ptr(), _ptr(dz), _ptr(dw), _ptr(ws),
                           tokens, heads, dim, *_strides(dy, "dy", 2), *_strides(x, "x", 2), *zs, nbytes, _DT[x.dtype],
                           _code(weight), _ACT[activation], eps), index)
    return dict(dx=dx, dz=dz, dweight=dw)


class GatedNorm(torch.autograd.Function):
    """:func:`gated_norm_fwd` with its exact backward; x, z and weight are saved."""

    @staticmethod
    def forward(ctx, x, z, weight, eps, activation):
        ctx.save_for_backward(x, z, weight)
        ctx.how = dict(eps=eps, activation=activation)
        return gated_norm_fwd(x, z, weight, **ctx.how)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, z, weight = ctx.saved_tensors
        d = gated_norm_bwd(_rows(dy, 2), x, z, weight, **ctx.how)
        return d["dx"], d["dz"], d["dweight"], None, None


def _rows(t: torch.Tensor, inner: int) -> torch.Tensor:
    """An incoming gradient in a layout that the kernels take (autograd may hand over expanded or permuted ones)."""
    try:
        _strides(t, "", inner)
        return t
    except ValueError:
        return t.contiguous()


def gated_norm(x, z, weight, *, eps=1e-6, activation="silu") -> torch.Tensor:
    """Differentiable :func:`gated_norm_fwd`."""
    _gated_check(x, z, weight, activation)
    return GatedNorm.apply(x, z, weight, eps, activation)


# ---------------------------------------------------------------- norm before a block
def _scale_of(scale, index, dim):
    """(the vector or None, the number)"""
    if isinstance(scale, torch.Tensor):
        _vector(scale, "scale", index, dim)
        return scale, 1.0
    return None, float(scale)


def _residual_type(t, name, index, x):
    _like(t, name, index, x.shape, x.dtype, _F32)


def add_norm_fwd(x, residual, weight, scale=1.0, *, eps=1e-6, stream=None):
    """r' = residual + scale * x and y = weight * r' / sqrt(mean(r'^2) + eps) over the last axis; returns (y, r').

    x [..., D] (fp32, bf16 or fp16); residual like x, of x's type or fp32, or None (the stream starts here: r' = scale x
    in x's type); weight [D] of any of the types, or None (1); scale a number, or a tensor [D] (one for each channel).
    The last axis is contiguous and the others at one distance.  y is formed from r' before r' is rounded."""
    if stream is not None:
        with _on(stream, (x, residual, weight, scale if isinstance(scale, torch.Tensor) else None)):
            return add_norm_fwd(x, residual, weight, scale, eps=eps)
    index = _cuda(x, "x")
    _need(x.dim() >= 1, "x must be [..., D]")
    dim = x.shape[-1]
    if residual is not None:
        _residual_type(residual, "residual", index, x)
    _vector(weight, "weight", index, dim)
    vec, num = _scale_of(scale, index, dim)
    y = _result(x)
    out = _result(x if residual is None else residual)
    n = x.numel()
    if n == 0:
        return y, out
    _queue("gdr_add_norm_fwd",
           _pack_add_fwd(x.data_ptr(), _ptr(residual), _ptr(weight), _ptr(vec), y.data_ptr(), out.data_ptr(), n // dim, dim,
                         _token_stride(x, "x"), 0 if residual is None else _token_stride(residual, "residual"), dim,
                         _DT[x.dtype], _DT[out.dtype], _code(weight), _code(vec), num, eps), index)
    return y, out


def add_norm_bwd(dy, dres, residual_out, weight, scale=1.0, *, x=None, eps=1e-6, stream=None) -> dict:
    """Gradients of :func:`add_norm_fwd` at the r' that it returned: dict(dx, dresidual, dweight, dscale).

    dy like y; dres, the gradient of r', like r' or None (zero).  dresidual is like r', dx like y; they are one and the
    same tensor when scale is the number 1 and their types agree.  dscale needs x and a tensor for scale, and is None
    without x; dweight is None when weight is."""
    if stream is not None:
        with _on(stream, (dy, dres, residual_out, weight, x, scale if isinstance(scale, torch.Tensor) else None)):
            return add_norm_bwd(dy, dres, residual_out, weight, scale, x=x, eps=eps)
    index = _cuda(dy, "dy")
    _need(dy.dim() >= 1, "dy must be [..., D]")
    dim = dy.shape[-1]
    _residual_type(residual_out, "residual_out", index, dy)
    if dres is not None:
        _like(dres, "dres", index, dy.shape, residual_out.dtype)
    _vector(weight, "weight", index, dim)
    vec, num = _scale_of(scale, index, dim)
    if x is not None:
        _need(vec is not None, "x is for dscale: scale must be a tensor")
        _like(x, "x", index, dy.shape, dy.dtype)
    dev = dy.device
    dr = _result(residual_out)
    same = vec is None and num == 1.0 and dr.dtype == dy.dtype
    dx = dr if same else _result(dy)
    dw = None if weight is None else torch.empty(dim, dtype=weight.dtype, device=dev)
    ds = None if x is None else torch.empty(dim, dtype=vec.dtype, device=dev)
    out = dict(dx=dx, dresidual=dr, dweight=dw, dscale=ds)
    n = dy.numel()
    if n == 0:
        for t in (dw, ds):
            if t is not None:
                t.zero_()
        return out
    sums = (dw is not None) + (ds is not None)
    nbytes = _entry("gdr_norm_workspace_bytes")(n // dim, dim, sums) if sums else 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None
    _queue("gdr_add_norm_bwd",
           _pack_add_bwd(dy.data_ptr(), _ptr(dres), residual_out.data_ptr(), _ptr(x), _ptr(weight), _ptr(vec),
                         0 if same else dx.data_ptr(), dr.data_ptr(), _ptr(dw), _ptr(ds), _ptr(ws), n // dim, dim,
                         _token_stride(dy, "dy"), 0 if dres is None else _token_stride(dres, "dres"),
                         _token_stride(residual_out, "residual_out"), 0 if x is None else _token_stride(x, "x"), nbytes,
                         _DT[dy.dtype], _DT[dr.dtype], _code(weight), _code(vec), num, eps), index)
    return out


class AddNorm(torch.autograd.Function):
    """:func:`add_norm_fwd` with its exact backward; r', weight and, when scale is a tensor, x are saved."""

    @staticmethod
    def forward(ctx, x, residual, weight, scale, eps):
        y, out = add_norm_fwd(x, residual, weight, scale, eps=eps)
        vec = scale if isinstance(scale, torch.Tensor) else None
        ctx.save_for_backward(out, weight, vec, None if vec is None else x)
        ctx.scale, ctx.eps, ctx.stream_in = scale if vec is None else None, eps, residual is not None
        return y, out

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dres):
        out, weight, vec, x = ctx.saved_tensors
        d = add_norm_bwd(_rows(dy, 1), _rows(dres, 1), out, weight, ctx.scale if vec is None else vec, x=x, eps=ctx.eps)
        return d["dx"], d["dresidual"] if ctx.stream_in else None, d["dweight"], d["dscale"], None


def add_norm(x, residual, weight, scale=1.0, *, eps=1e-6):
    """Differentiable :func:`add_norm_fwd`: returns (y, r')."""
    return AddNorm.apply(x, residual, weight, scale, eps)


# ---------------------------------------------------------------- gated linear recurrence
def _linrec_check(x, g, h0, cu_seqlens):
    index = _cuda(x, "x")
    _need(x.dim() == 3, "x must be [B, T, D]")
    _like(g, "g", index, x.shape, x.dtype, _F32)
    B, T, D = x.shape
    _need(B >= 1 and D >= 1, "x must be [B, T, D] with B and D at least 1")
    N = B
    if cu_seqlens is not None:
        _need(B == 1, "packed sequences (cu_seqlens) need B = 1")
        _need(cu_seqlens.dim() == 1 and cu_seqlens.shape[0] >= 2, "cu_seqlens must be [N + 1] with N at least 1")
        N = cu_seqlens.shape[0] - 1
        _like(cu_seqlens, "cu_seqlens", index, (N + 1,), torch.int32)
        _need(cu_seqlens.is_contiguous(), "cu_seqlens must be contiguous")
    if h0 is not None:
        _like(h0, "h0", index, (N, D), _F32)
        _need(h0.is_contiguous(), "h0 must be contiguous")
    return index, B, T, D, N


def _linrec_done(workspaces, check_status, index):
    """Waits for a call's passes, of which each has its own workspace (an address), and raises what they reported."""
    if check_status:
        with torch.cuda.device(index):
            for ws in workspaces:
                st = _entry("gdr_linrec_get_status")(ws, _raw_stream(index))
                if st:
                    raise GdrError(st, "gdr_linrec_get_status")


def linrec_fwd(x, g, h0=None, cu_seqlens=None, *, complement=False, return_states=False, stream=None,
               check_status=False):
    """h_t = a_t h_{t-1} + b_t for every channel, a = exp(g), b = x, or (1 - a) x with ``complement``.

    x [B, T, D] (fp32, bf16 or fp16); g [B, T, D] the raw log-gate, of x's type or fp32; h0 fp32 [N, D] or None (zero);
    cu_seqlens int32 [N + 1] (packed sequences, B == 1) or None (N = B).  The last axis of x and g is contiguous and the
    others at one distance.  Returns (h like x, ht fp32 [N, D]), and with ``return_states`` the states fp32
    [ceil(B T / 16), D] that :func:`linrec_bwd` takes.  ``check_status`` waits for the call and raises on malformed
    cu_seqlens."""
    if stream is not None:
        with _on(stream, (x, g, h0, cu_seqlens)):
            return linrec_fwd(x, g, h0, cu_seqlens, complement=complement, return_states=return_states,
                              check_status=check_status)
    index, B, T, D, N = _linrec_check(x, g, h0, cu_seqlens)
    dev = x.device
    h = _result(x)
    ht = torch.empty(N, D, dtype=_F32, device=dev)
    tiles = -(-B * T // _lib.LINREC_SAVE)
    states = torch.empty(tiles, D, dtype=_F32, device=dev) if return_states else None
    nbytes = _entry("gdr_linrec_workspace_bytes")(B * T, D)
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    _queue("gdr_linrec_fwd",
           _pack_linrec_fwd(x.data_ptr(), g.data_ptr(), _ptr(h0), _ptr(cu_seqlens), h.data_ptr(), ht.data_ptr(),
                            _ptr(states), ws.data_ptr(), B, T, D, 0 if cu_seqlens is None else N, _token_stride(x, "x"),
                            _token_stride(g, "g"), nbytes, _DT[x.dtype], _DT[g.dtype], int(complement), 0), index)
    _linrec_done([ws.data_ptr()], check_status, index)
    return (h, ht, states) if return_states else (h, ht)


def linrec_bwd(x, g, dh, h0=None, dht=None, cu_seqlens=None, states=None, *, complement=False, stream=None,
               check_status=False) -> dict:
    """Gradients of :func:`linrec_fwd`: dict(dx like x, dg like g, dh0 fp32 [N, D]).

    dh like x; dht fp32 [N, D], the gradient of ht, or None (zero); states as ``return_states`` gave them on the same
    x, g and h0, or None: they are computed first, by one more pass over x and g."""
    if stream is not None:
        with _on(stream, (x, g, dh, h0, dht, cu_seqlens, states)):
            return linrec_bwd(x, g, dh, h0, dht, cu_seqlens, states, complement=complement, check_status=check_status)
    index, B, T, D, N = _linrec_check(x, g, h0, cu_seqlens)
    _like(dh, "dh", index, x.shape, x.dtype)
    if dht is not None:
        _like(dht, "dht", index, (N, D), _F32)
        _need(dht.is_contiguous(), "dht must be contiguous")
    dev = x.device
    nbytes = _entry("gdr_linrec_workspace_bytes")(B * T, D)
    # (a pass starts by clearing its workspace's status: two passes in one would lose the first one's)
    ws = torch.empty(nbytes if states is not None else 2 * nbytes, dtype=torch.uint8, device=dev)
    passes = [ws.data_ptr()]
    tiles = -(-B * T // _lib.LINREC_SAVE)
    strides = _token_stride(x, "x"), _token_stride(g, "g")
    seqs = 0 if cu_seqlens is None else N
    if states is None:
        states = torch.empty(tiles, D, dtype=_F32, device=dev)
        passes.append(passes[0] + nbytes)
        _queue("gdr_linrec_fwd",
               _pack_linrec_fwd(x.data_ptr(), g.data_ptr(), _ptr(h0), _ptr(cu_seqlens), 0, 0, states.data_ptr(),
                                passes[1], B, T, D, seqs, *strides, nbytes, _DT[x.dtype], _DT[g.dtype],
                                int(complement), 0), index)
    else:
        _like(states, "states", index, (tiles, D), _F32)
        _need(states.is_contiguous(), "states must be contiguous")
    dx = _result(x)
    dg = _result(g)
    dh0 = torch.empty(N, D, dtype=_F32, device=dev)
    _queue("gdr_linrec_bwd",
           _pack_linrec_bwd(x.data_ptr(), g.data_ptr(), dh.data_ptr(), _ptr(h0), _ptr(dht), states.data_ptr(),
                            _ptr(cu_seqlens), dx.data_ptr(), dg.data_ptr(), dh0.data_ptr(), passes[0], B, T, D, seqs,
                            *strides, _token_stride(dh, "dh"), nbytes, _DT[x.dtype], _DT[g.dtype], int(complement), 0),
           index)
    _linrec_done(passes, check_status, index)
    return dict(dx=dx, dg=dg, dh0=dh0)


class LinearRecurrence(torch.autograd.Function):
    """h, ht = forward(x, g, h0, cu_seqlens, complement) with its exact backward.  The inputs and one fp32 state for
    every 16 tokens are saved."""

    @staticmethod
    def forward(ctx, x, g, h0, cu_seqlens, complement):
        h, ht, states = linrec_fwd(x, g, h0, cu_seqlens, complement=complement, return_states=True)
        ctx.save_for_backward(x, g, h0, cu_seqlens, states)
        ctx.complement = complement
        return h, ht

    @staticmethod
    @once_differentiable
    def backward(ctx, dh, dht):
        x, g, h0, cu_seqlens, states = ctx.saved_tensors
        d = linrec_bwd(x, g, _rows(dh, 1), h0, dht.contiguous(), cu_seqlens, states, complement=ctx.complement)
        return d["dx"], d["dg"], None if h0 is None else d["dh0"], None, None


def linear_recurrence(x, g, h0=None, cu_seqlens=None, *, complement=False):
    """Differentiable :func:`linrec_fwd`: returns (h, ht)."""
    return LinearRecurrence.apply(x, g, h0, cu_seqlens, complement)


def linrec_step(x, g, state, slots=None, *, complement=False, stream=None) -> torch.Tensor:
    """One token for each sequence: state = a state + b in place; returns y = state in x's type.

    x [B, D] (fp32, bf16 or fp16), g [B, D] of x's type or fp32, state fp32 [num_slots, D] contiguous.  Sequence i owns
    state[slots[i]] (slots int32 [B], distinct; None: state[i]).  A slot outside [0, num_slots), for example -1 for a
    row that only pads the batch, is skipped and its y row is zero."""
    if stream is not None:
        with _on(stream, (x, g, state, slots)):
            return linrec_step(x, g, state, slots, complement=complement)
    index = _cuda(x, "x")
    _need(x.dim() == 2, "x must be [B, D]")
    B, D = x.shape
    _like(g, "g", index, x.shape, x.dtype, _F32)
    _need(state.dim() == 2 and state.is_contiguous(), "state must be a contiguous [num_slots, D]")
    _like(state, "state", index, (state.shape[0], D), _F32)
    if slots is not None:
        _like(slots, "slots", index, (B,), torch.int32)
        _need(slots.is_contiguous(), "slots must be contiguous")
    else:
        _need(state.shape[0] >= B, "state must have a row for each sequence")
    y = _result(x)
    if B == 0 or D == 0:
        return y
    _queue("gdr_linrec_step",
           _pack_linrec_step(x.data_ptr(), g.data_ptr(), _ptr(slots), state.data_ptr(), y.data_ptr(), B, D, state.shape[0],
                             _token_stride(x, "x"), _token_stride(g, "g"), _DT[x.dtype], _DT[g.dtype], int(complement), 0),
           index)
    increment_version(state)  # (as torch's own in-place operations do: a backward that saved it notices)
    return y


# ---------------------------------------------------------------- gradient norm and clip
def _layout(t: torch.Tensor):
    """(size, distance) of the axes that have more than one element."""
    return [(n, s) for n, s in zip(t.shape, t.stride()) if n != 1]


def _dense(t: torch.Tensor) -> bool:
    """Whether the elements fill a stretch of memory, in whatever order of the axes."""
    span = 1
    for s, n in sorted((s, n) for n, s in _layout(t)):
        if s != span:
            return False
        span *= n
    return True


def _listed(tensors, name, index):
    """Addresses, sizes and types of a list of tensors as arrays for the C entry, and whether all are contiguous."""
    # (attribute by attribute: a list is checked in a fraction of the time that a loop over its tensors takes)
    flat = all([t.is_contiguous() for t in tensors])
    if [t.get_device() for t in tensors].count(index) != len(tensors) or not (
            flat or all([t.is_contiguous() or _dense(t) for t in tensors])):
        raise ValueError(f"{name} must be tensors on cuda:{index} without gaps (contiguous, or with their axes permuted)")
    try:
        types = array("i", [_DT[t.dtype] for t in tensors])
    except KeyError:
        raise ValueError(f"{name} must be float32, bfloat16 or float16 tensors") from None
    return array("Q", [t.data_ptr() for t in tensors]), array("q", [t.numel() for t in tensors]), types, flat


def _clip(entry, grads: Sequence[torch.Tensor], max_norm, out, eps):
    grads, out = list(grads), None if out is None else list(out)
    _need(out is None or len(out) == len(grads), "out must have one tensor for each gradient, of its size")
    _need(len(grads) > 0, "no gradients were given")
    try:
        index = _cuda(grads[0], "grads[0]")
        ptrs, sizes, types, flat = _listed(grads, "grads", index)
    except AttributeError:  # (None has no device; looking for it first would cost every call)
        kept = [i for i, t in enumerate(grads) if t is not None]
        if len(kept) == len(grads):
            raise
        return _clip(entry, [grads[i] for i in kept], max_norm, None if out is None else [out[i] for i in kept], eps)
    outs, out_types = None, None
    if out is not None:
        try:
            outs, out_sizes, out_types, out_flat = _listed(out, "out", index)
        except AttributeError:
            raise ValueError("out must have one tensor for each gradient, of its size") from None
        _need(out_sizes == sizes, "out must have one tensor for each gradient, of its size")
        if not (flat and out_flat):  # (element by element in the order of memory)
            _need(all([_layout(o) == _layout(g) or (o.is_contiguous() and g.is_contiguous()) for g, o in zip(grads, out)]),
                  "out must have its axes in the gradients' order in memory")
    dev = grads[0].device
    nbytes = _entry("gdr_clip_workspace_bytes")(len(grads), sum(sizes))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    norm = torch.empty((), dtype=_F32, device=dev)

    def addr(a):
        return 0 if a is None else a.buffer_info()[0]

    _queue(entry, _pack_clip(addr(ptrs), addr(outs), addr(sizes), addr(types), addr(out_types), norm.data_ptr(),
                             ws.data_ptr(), len(grads), nbytes, max_norm, eps), index)
    if out is not None or entry == "gdr_clip_grad_norm":
        increment_version(grads if out is None else out)
    return norm


def grad_norm(grads, *, stream=None) -> torch.Tensor:
    """sqrt of the sum of all squares over a list of tensors (fp32, bf16, fp16 in any mixture, any of them empty, without
    gaps in memory: contiguous or with their axes permuted), as a 0-dim fp32 tensor.  An entry may be None, as the
    gradient of a weight that took no part is, but not all of them."""
    if stream is not None:
        grads = list(grads)
        with _on(stream, grads):
            return grad_norm(grads)
    return _clip("gdr_grad_norm", grads, 0.0, None, 0.0)


def clip_grad_norm(grads, max_norm, out=None, *, eps=1e-6, stream=None) -> torch.Tensor:
    """Scale the gradients by min(1, max_norm / (norm + eps)), in place or into ``out`` (a tensor for each, of any of the
    types, with its axes in the same order in memory), and return their norm before that, as :func:`grad_norm` does.
    Nothing is read back to the host."""
    if stream is not None:
        grads, out = list(grads), None if out is None else list(out)
        with _on(stream, grads + (out or [])):
            return clip_grad_norm(grads, max_norm, out, eps=eps)
    _need(max_norm >= 0, "max_norm must not be negative")
    return _clip("gdr_clip_grad_norm", grads, float(max_norm), out, eps)
