"""Torch-facing calls of the gated feed-forward (include/gdr_block.h): h = act(x w_gate^T) * (x w_up^T) in one kernel, and its
backward.

As in :mod:`block`, everything is computed by libgdrbwd.so's kernels; ``*_fwd`` and ``*_bwd`` are the plain calls,
``gated_ffn`` is differentiable, once.  ``stream`` (default: torch's current stream) queues a call there.  The projection
that follows a gated feed-forward is one plain matrix product: ``gated_ffn(x, w_gate, w_up) @ w_down.t()``.
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _lib
from ._lib import GdrError
from .block import _DT, _F32, _cuda, _entry, _like, _need, _on, _ptr, _queue, _raw_stream, _result, _rows, _token_stride

_pack_fwd = _lib.packer(_lib.GdrFfnFwdArgs)
_pack_bwd = _lib.packer(_lib.GdrFfnBwdArgs)
_ACT = {"silu": 0, "sigmoid": 1, "gelu_tanh": 2}


def _check(x, w_gate, w_up, activation):
    """(device, tokens, width, inner width, distances of the weights' rows, code of the activation)"""
    index = _cuda(x, "x")
    dtype, dim = x.dtype, x.shape[-1] if x.dim() else 0
    _need(dtype != _F32, "x must be bfloat16 or float16 (the products run on 16-bit operands)")
    _need(dim >= 1 and w_gate.dim() == 2 and w_gate.shape[0] >= 1, "x must be [..., D] and w_gate [inner, D]")
    inner = w_gate.shape[0]
    _like(w_gate, "w_gate", index, (inner, dim), dtype)
    _like(w_up, "w_up", index, (inner, dim), dtype)
    (gs, g1), (us, u1) = w_gate.stride(), w_up.stride()
    _need(dim == 1 or g1 == u1 == 1, "the weights' last axis must be contiguous")
    code = _ACT.get(activation)
    if code is None:
        raise ValueError(f"activation must be one of {sorted(_ACT)}")
    return index, x.numel() // dim, dim, inner, (gs, us), code


def _workspace(x, xs, w_gate, w_up, strides, tokens, dim, inner, backward, status):
    """(tensor or None, bytes) of a call's workspace, and whether it is to have a status by all means."""
    gs, us = strides
    copies = ((x.data_ptr() | w_gate.data_ptr() | w_up.data_ptr()) % 16 or (xs | gs | us) % 8
              or xs < dim or gs < dim or us < dim)
    nbytes = _entry("gdr_ffn_workspace_bytes")(tokens, dim, inner, 1 if copies else 0, backward)
    if nbytes == 0 or (nbytes == _lib.FFN_STATUS_BYTES and not status):  # nothing but the status
        return None, 0
    return x.new_empty(nbytes, dtype=torch.uint8), nbytes


def _finish(ws, check_status, index):
    if check_status and ws is not None:
        with torch.cuda.device(index):
            st = _entry("gdr_ffn_get_status")(ws.data_ptr(), _raw_stream(index))
        if st:
            raise GdrError(st, "gdr_ffn_get_status")


def gated_ffn_fwd(x, w_gate, w_up, *, activation="silu", return_saved=False, stream=None, check_status=False):
    """h = act(x w_gate^T) * (x w_up^T) over the last axis.

    x [..., D], w_gate and w_up [inner, D] (as a Linear has them), all bf16 or all fp16, the last axis contiguous and the
    axes of x before it at one distance; ``activation``: "silu", "sigmoid" or "gelu_tanh".  Products are summed in fp32 and
    h [..., inner] is rounded once.  With ``return_saved``: (h, saved), what :func:`gated_ffn_bwd` takes: both projections,
    fp32 [2, ..., inner].  Widths that are multiples of 8 are read where they are, others are copied first.
    ``check_status`` waits for the call and raises if a wait inside it ran out."""
    if stream is not None:
        with _on(stream, (x, w_gate, w_up)):
            return gated_ffn_fwd(x, w_gate, w_up, activation=activation, return_saved=return_saved, check_status=check_status)
    index, tokens, dim, inner, strides, code = _check(x, w_gate, w_up, activation)
    shape = (*x.shape[:-1], inner)
    h = x.new_empty(shape)
    saved = x.new_empty((2, *shape), dtype=_F32) if return_saved else None
    if tokens:
        xs = _token_stride(x, "x")
        ws, nbytes = _workspace(x, xs, w_gate, w_up, strides, tokens, dim, inner, 0, check_status)
        gate = _ptr(saved)
        up = gate + tokens * inner * 4 if gate else 0
        _queue("gdr_ffn_fwd", _pack_fwd(x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), h.data_ptr(), gate, up, _ptr(ws), tokens, dim, inner, xs, *strides, nbytes, _DT[x.dtype], code), index)
        _finish(ws, check_status, index)
    return (h, saved) if return_saved else h


def gated_ffn_bwd(dh, x, w_gate, w_up, saved=None, *, activation="silu", need_dx=True, need_dw=True, stream=None,
                  check_status=False) -> dict:
    """Gradients of :func:`gated_ffn_fwd`: dict(dx like x, dw_gate, dw_up [inner, D]), all in x's type, None for what
    ``need_dx`` and ``need_dw`` leave out.

    dh like h; saved as ``return_saved`` gave it on the same x and weights, or None: the projections are computed first, by
    one more forward pass, which ``check_status`` covers too.  The gradients of the two projections are rounded to x's type
    before the products with them: in fp16 they have its range (infinite past 65504, 0 below 2^-25), so scale the loss for it."""
    if stream is not None:
        with _on(stream, (dh, x, w_gate, w_up, saved)):
            return gated_ffn_bwd(dh, x, w_gate, w_up, saved, activation=activation, need_dx=need_dx, need_dw=need_dw,
                                 check_status=check_status)
    index, tokens, dim, inner, strides, code = _check(x, w_gate, w_up, activation)
    shape = (*x.shape[:-1], inner)
    _like(dh, "dh", index, shape, x.dtype)
    if saved is None:
        _, saved = gated_ffn_fwd(x, w_gate, w_up, activation=activation, return_saved=True, check_status=check_status)
    _like(saved, "saved", index, (2, *shape), _F32)
    _need(saved.is_contiguous(), "saved must be contiguous")
    gate = saved.data_ptr()
    dx = _result(x) if need_dx else None
    dwg, dwu = (_result(w_gate), _result(w_up)) if need_dw else (None, None)
    if tokens or need_dw:
        xs, ds = (_token_stride(x, "x"), _token_stride(dh, "dh")) if tokens else (dim, inner)
        ws, nbytes = _workspace(x, xs, w_gate, w_up, strides, tokens, dim, inner, 1, check_status)
        _queue("gdr_ffn_bwd",
               _pack_bwd(dh.data_ptr(), x.data_ptr(), w_gate.data_ptr(), w_up.data_ptr(), gate, gate + tokens * inner * 4,
                         _ptr(dx), _ptr(dwg), _ptr(dwu), _ptr(ws), tokens, dim, inner, ds, xs, *strides, nbytes,
                         _DT[x.dtype], code), index)
        _finish(ws, check_status, index)
    return dict(dx=dx, dw_gate=dwg, dw_up=dwu)


class GatedFfn(torch.autograd.Function):
    """:func:`gated_ffn_fwd` with its backward; x, the weights and both projections are saved."""

    @staticmethod
    def forward(ctx, x, w_gate, w_up, activation):
        h, saved = gated_ffn_fwd(x, w_gate, w_up, activation=activation, return_saved=True)
        ctx.save_for_backward(x, w_gate, w_up, saved)
        ctx.activation = activation
        return h

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, w_gate, w_up, saved = ctx.saved_tensors
        d = gated_ffn_bwd(_rows(dh, 1), x, w_gate, w_up, saved, activation=ctx.activation,
                          need_dx=ctx.needs_input_grad[0], need_dw=any(ctx.needs_input_grad[1:3]))
        return d["dx"], d["dw_gate"], d["dw_up"], None


def _dual(*tensors) -> bool:
    """Whether any has a tangent of forward-mode differentiation (which no tensor has outside a level of it)."""
    return getattr(forward_ad, "_current_level", 0) >= 0 and any(forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def gated_ffn(x, w_gate, w_up, *, activation="silu") -> torch.Tensor:
    """Differentiable :func:`gated_ffn_fwd`; nothing is kept where no gradient is wanted.  Tangents of forward-mode
    differentiation are refused.

    A backward pass captured into a CUDA graph: as for every differentiable function, torch adds a leaf's gradients on the
    stream of that leaf's first use that is still alive.  Nothing that an earlier, eager pass over the same leaves gave may
    live then (losses and outputs with their graph dropped, as torch's own captures want it); ``gated_ffn_fwd`` and
    ``gated_ffn_bwd`` know no leaves and can be captured at any time."""
    if torch.is_grad_enabled() and (x.requires_grad or w_gate.requires_grad or w_up.requires_grad) or _dual(x, w_gate, w_up):
        return GatedFfn.apply(x, w_gate, w_up, activation)
    return gated_ffn_fwd(x, w_gate, w_up, activation=activation)
