"""The C entries of include/gdr_block.h on the GPU with any of their outputs absent, rows at distances wider than they are
and widths that are no whole number of 16-byte pieces: right values, and nothing written beside an output."""
import ctypes
import itertools

import pytest
import torch

import block_util as U
from chunked_gated_delta_09_gb300 import _lib

pytestmark = pytest.mark.gpu

EPS = 1e-5
CODE = {torch.float32: _lib.GDR_F32, torch.bfloat16: _lib.GDR_BF16, torch.float16: _lib.GDR_F16}
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
GUARD = 256  # elements on each side


class Guarded:
    """An output of n elements between guard values."""

    def __init__(self, n, dtype):
        self.all = torch.full((n + 2 * GUARD,), 77.0, dtype=dtype, device="cuda")
        self.n = n

    def ptr(self):
        return self.all.data_ptr() + GUARD * self.all.element_size()

    def value(self, *shape):
        assert (self.all[:GUARD] == 77.0).all() and (self.all[GUARD + self.n:] == 77.0).all(), "written beside the output"
        return self.all[GUARD:GUARD + self.n].view(*shape)


def padded(gen, rows, dim, stride, dtype, times=1.0):
    """Rows at a distance of `stride`, nans between them."""
    wide = torch.full((rows * stride,), float("nan"), dtype=dtype, device="cuda")
    view = torch.as_strided(wide, (rows, dim), (stride, 1))
    view.copy_(U.randn(gen, rows, dim, dtype=dtype, times=times))
    return view


def call(name, kind, **args):
    a = kind(**args)
    status = getattr(_lib.load(), name)(ctypes.addressof(a), torch.cuda.current_stream().cuda_stream)
    assert status == _lib.GDR_OK, status


def wide(dim):
    """A distance of whole 16-byte pieces in every type."""
    return (dim + 7) // 8 * 8 + 8


@pytest.mark.parametrize("dtype,rtype", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,dim", [(1, 4), (5, 12), (3, 13), (37, 20), (300, 260), (7, 2052), (3, 4102)])
def test_add_norm_backward(rows, dim, dtype, rtype):
    gen, dt, rt, ts = U.seeded(rows + dim), TYPES[dtype], TYPES[rtype], wide(dim)
    dy, x = (padded(gen, rows, dim, ts, dt) for _ in range(2))
    dres, r = (padded(gen, rows, dim, ts, rt, 2.0) for _ in range(2))
    w, s = (1.0 + U.randn(gen, dim, times=0.2) for _ in range(2))
    ref = U.add_norm_bwd(dy, dres, r, w, s, x, EPS)
    lib = _lib.load()
    for parts in itertools.product((False, True), repeat=4):
        names = [n for n, on in zip(("dx", "dresidual", "dweight", "dscale"), parts) if on]
        out = {n: Guarded(rows * dim if n in ("dx", "dresidual") else dim,
                          {"dx": dt, "dresidual": rt}.get(n, torch.float32)) for n in names}
        sums = sum(n in out for n in ("dweight", "dscale"))
        nbytes = lib.gdr_norm_workspace_bytes(rows, dim, sums) if sums else 0
        ws = Guarded(nbytes // 4, torch.float32)
        call("gdr_add_norm_bwd", _lib.GdrAddNormBwdArgs, dy=dy.data_ptr(), dres=dres.data_ptr(), residual_out=r.data_ptr(),
             x=x.data_ptr(), weight=w.data_ptr(), scale_vec=s.data_ptr(), workspace=ws.ptr() if sums else None,
             tokens=rows, dim=dim, dy_token_stride=ts, dres_token_stride=ts, residual_out_token_stride=ts, x_token_stride=ts,
             workspace_bytes=nbytes, dtype=CODE[dt], residual_dtype=CODE[rt], weight_dtype=0, scale_dtype=0, scale=1.0, eps=EPS,
             **{n: g.ptr() for n, g in out.items()})
        ws.value(-1)
        U.check({n: g.value(*ref[n].shape) for n, g in out.items()}, {n: ref[n] for n in names})


@pytest.mark.parametrize("dtype,rtype", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("rows,dim", [(1, 4), (5, 12), (3, 13), (300, 260), (7, 2052)])
def test_add_norm_forward(rows, dim, dtype, rtype):
    """residual_out absent, or at a distance of its own."""
    gen, dt, rt, ts = U.seeded(rows + dim), TYPES[dtype], TYPES[rtype], wide(dim)
    x, res = padded(gen, rows, dim, ts, dt), padded(gen, rows, dim, ts, rt, 2.0)
    w = 1.0 + U.randn(gen, dim, times=0.2)
    ref = U.add_norm_fwd(x, res, w, 0.5, EPS)
    for stride in (None, dim, ts):
        y, out = Guarded(rows * dim, dt), Guarded(rows * (stride or dim), rt)
        call("gdr_add_norm_fwd", _lib.GdrAddNormFwdArgs, x=x.data_ptr(), residual=res.data_ptr(), weight=w.data_ptr(),
             y=y.ptr(), residual_out=None if stride is None else out.ptr(), tokens=rows, dim=dim, x_token_stride=ts,
             residual_token_stride=ts, residual_out_token_stride=stride or 0, dtype=CODE[dt], residual_dtype=CODE[rt],
             weight_dtype=0, scale_dtype=0, scale=0.5, eps=EPS)
        U.check(dict(y=y.value(rows, dim)), dict(y=ref["y"]))
        got = out.value(rows, stride or dim)
        if stride is None:
            assert (got == 77.0).all()
        else:
            U.check(dict(r=got[:, :dim]), dict(r=ref["r"]))
            assert (got[:, dim:] == 77.0).all()


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("tokens,heads,dim", [(1, 1, 4), (5, 3, 12), (3, 2, 13), (70, 3, 68), (7, 1, 2052)])
def test_gated_norm(tokens, heads, dim, dtype):
    """Forward, and backward with dweight and the gate absent or not."""
    gen, dt, hs = U.seeded(tokens + dim), TYPES[dtype], wide(dim)
    x, z, dy = (padded(gen, tokens * heads, dim, hs, dt) for _ in range(3))
    w = 1.0 + U.randn(gen, dim, times=0.2)
    shape, at = (tokens, heads, dim), dict(tokens=tokens, heads=heads, dim=dim, dtype=CODE[dt], weight_dtype=0, activation=0,
                                           eps=EPS)
    places = dict(x_token_stride=heads * hs, x_head_stride=hs, z_token_stride=heads * hs, z_head_stride=hs)
    lib = _lib.load()
    for gate, weight in itertools.product((False, True), repeat=2):
        ref = U.gated_norm(x.view(shape), z.view(shape) if gate else None, w, EPS, "silu", dy.view(shape))
        y, dx, dz = (Guarded(tokens * heads * dim, dt) for _ in range(3))
        call("gdr_gated_norm_fwd", _lib.GdrGatedNormFwdArgs, x=x.data_ptr(), z=z.data_ptr() if gate else None,
             weight=w.data_ptr(), y=y.ptr(), **at, **places)
        nbytes = lib.gdr_norm_workspace_bytes(tokens * heads, dim, 1) if weight else 0
        ws, dw = Guarded(nbytes // 4, torch.float32), Guarded(dim, torch.float32)
        call("gdr_gated_norm_bwd", _lib.GdrGatedNormBwdArgs, dy=dy.data_ptr(), x=x.data_ptr(),
             z=z.data_ptr() if gate else None, weight=w.data_ptr(), dx=dx.ptr(), dz=dz.ptr() if gate else None,
             dweight=dw.ptr() if weight else None, workspace=ws.ptr() if weight else None, workspace_bytes=nbytes,
             dy_token_stride=heads * hs, dy_head_stride=hs, **at, **places)
        ws.value(-1)
        got = dict(y=y.value(shape), dx=dx.value(shape), dz=dz.value(shape), dweight=dw.value(dim))
        for name, on in (("dz", gate), ("dweight", weight)):
            if not on:
                assert (got[name] == 77.0).all()
                ref.pop(name)
        U.check(got, ref)


@pytest.mark.parametrize("dtype,gtype", [("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
@pytest.mark.parametrize("T,D", [(1, 4), (1, 12), (1, 7), (2, 4), (17, 20), (300, 36), (300, 33)])
def test_recurrence_forward(T, D, dtype, gtype):
    """h, ht and states absent or not."""
    gen, dt, gt, ts = U.seeded(T + D), TYPES[dtype], TYPES[gtype], wide(D)
    x, g = padded(gen, T, D, ts, dt), padded(gen, T, D, ts, gt)
    g.copy_(-g.abs())
    ref = U.linrec(x[None], g[None], None, None, False)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    saved = torch.cat([torch.zeros(1, D, dtype=torch.float64), ref["h"][0, 15::16]])[:-(-T // 16)]
    for parts in itertools.product((False, True), repeat=3):
        h, ht, states = Guarded(T * D, dt), Guarded(D, torch.float32), Guarded(-(-T // 16) * D, torch.float32)
        call("gdr_linrec_fwd", _lib.GdrLinrecFwdArgs, x=x.data_ptr(), g=g.data_ptr(), h=h.ptr() if parts[0] else None,
             ht=ht.ptr() if parts[1] else None, states=states.ptr() if parts[2] else None, workspace=ws.data_ptr(), batch=1,
             tokens=T, dim=D, x_token_stride=ts, g_token_stride=ts, workspace_bytes=256, dtype=CODE[dt], gate_dtype=CODE[gt])
        want = dict(h=ref["h"][0], ht=ref["ht"][0], states=saved[1:])
        got = dict(h=h.value(T, D), ht=ht.value(D), states=states.value(-1, D)[1:])
        for on, name in zip(parts, ("h", "ht", "states")):
            if not on:
                assert (got.pop(name) == 77.0).all()
                want.pop(name)
        U.check(got, want)
