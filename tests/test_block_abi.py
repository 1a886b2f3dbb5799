"""include/gdr_block.h: every declared function is exported, the structures agree with the header's, and bad arguments
are refused on the host, by the C entries and by the torch calls.  Nothing is launched here."""
import ctypes
import os
import re

import pytest
import torch

import chunked_gated_delta_09_gb300 as pkg
from chunked_gated_delta_09_gb300 import _lib
from chunked_gated_delta_09_gb300.build import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TEXT = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "gdr_block.h")).read(), flags=re.S)
P = 0x10000
BAD, UNSUPPORTED, OK = _lib.GDR_ERR_INVALID_ARG, _lib.GDR_ERR_UNSUPPORTED, _lib.GDR_OK


@pytest.fixture(scope="module")
def lib():
    build()
    return _lib.load()


def test_every_declared_symbol_is_exported(lib):
    names = sorted(set(re.findall(r"\b(gdr_[a-z_]+)\s*\(", TEXT)))
    assert names == sorted(_lib.BLOCK_EXPORTS)
    for n in names:
        assert hasattr(lib, n), n


@pytest.mark.parametrize("kind,name", [
    (_lib.GdrGatedNormFwdArgs, "gdr_gated_norm_fwd_args"), (_lib.GdrGatedNormBwdArgs, "gdr_gated_norm_bwd_args"),
    (_lib.GdrAddNormFwdArgs, "gdr_add_norm_fwd_args"), (_lib.GdrAddNormBwdArgs, "gdr_add_norm_bwd_args"),
    (_lib.GdrLinrecFwdArgs, "gdr_linrec_fwd_args"), (_lib.GdrLinrecBwdArgs, "gdr_linrec_bwd_args"),
    (_lib.GdrLinrecStepArgs, "gdr_linrec_step_args"), (_lib.GdrClipArgs, "gdr_clip_args")])
def test_structures_follow_the_header(kind, name):
    body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", TEXT).group(1)
    fields = []
    for line in body.split(";"):
        words = line.split(",")
        if not line.strip():
            continue
        head = words[0].split()
        ctype = " ".join(head[:-1])
        for w in [head[-1]] + words[1:]:
            pointer = "*" in ctype or "*" in w or "*" in head[-1]
            fields.append((w.replace("*", "").split()[-1],
                           ctypes.c_void_p if pointer else {"int64_t": ctypes.c_int64, "uint64_t": ctypes.c_uint64,
                                                            "int32_t": ctypes.c_int32, "float": ctypes.c_float}[ctype]))
    assert fields == [tuple(f) for f in kind._fields_]


def call(lib, name, kind, base, **over):
    unknown = set(over) - {f for f, _ in kind._fields_}
    assert not unknown
    a = kind(**{**base, **over})
    return getattr(lib, name)(ctypes.addressof(a), None)


def refused(lib, name, kind, base, bad, status=BAD):
    for over in bad:
        assert call(lib, name, kind, base, **over) == status, over
    assert getattr(lib, name)(None, None) == BAD


def test_gated_norm_refusals(lib):
    base = dict(x=P, z=P, weight=P, y=P, tokens=4, heads=2, dim=64, x_token_stride=128, x_head_stride=64,
                z_token_stride=128, z_head_stride=64, dtype=1, weight_dtype=0, activation=0, eps=1e-6)
    bad = [dict(x=0), dict(y=0), dict(tokens=-1), dict(heads=0), dict(dim=0), dict(dtype=3), dict(weight_dtype=-1),
           dict(activation=2), dict(x=P + 1), dict(y=P + 1), dict(weight=P + 2), dict(x_token_stride=-1)]
    refused(lib, "gdr_gated_norm_fwd", _lib.GdrGatedNormFwdArgs, base, bad)
    large = [dict(dim=16385), dict(tokens=1 << 31), dict(tokens=1 << 25, heads=64)]
    refused(lib, "gdr_gated_norm_fwd", _lib.GdrGatedNormFwdArgs, base, large, UNSUPPORTED)
    assert call(lib, "gdr_gated_norm_fwd", _lib.GdrGatedNormFwdArgs, base, tokens=0, x=0, y=0) == OK
    need = lib.gdr_norm_workspace_bytes(8, 64, 1)
    assert need > 0
    del base["y"]
    base.update(dy=P, dx=P, dz=P, dweight=P, workspace=P, workspace_bytes=need, dy_token_stride=128, dy_head_stride=64)
    bad = [dict(x=0), dict(dy=0), dict(dx=0), dict(dz=0), dict(weight=0), dict(z=0), dict(workspace=0),
           dict(workspace=P + 8), dict(workspace_bytes=need - 1), dict(dx=P + 1), dict(dweight=P + 2), dict(dim=-1),
           dict(dy_token_stride=-8)]
    refused(lib, "gdr_gated_norm_bwd", _lib.GdrGatedNormBwdArgs, base, bad)


def test_add_norm_refusals(lib):
    base = dict(x=P, residual=P, weight=P, scale_vec=P, y=P, residual_out=P, tokens=4, dim=64, x_token_stride=64,
                residual_token_stride=64, residual_out_token_stride=64, dtype=1, residual_dtype=0, weight_dtype=0,
                scale_dtype=0, scale=1.0, eps=1e-6)
    bad = [dict(x=0), dict(y=0), dict(tokens=-1), dict(dim=0), dict(dtype=9), dict(residual_dtype=2), dict(scale_dtype=4),
           dict(residual=P + 2), dict(residual_out_token_stride=63), dict(scale_vec=P + 1)]
    refused(lib, "gdr_add_norm_fwd", _lib.GdrAddNormFwdArgs, base, bad)
    refused(lib, "gdr_add_norm_fwd", _lib.GdrAddNormFwdArgs, base, [dict(dim=20000)], UNSUPPORTED)
    need = lib.gdr_norm_workspace_bytes(4, 64, 2)
    base = dict(dy=P, dres=P, residual_out=P, x=P, weight=P, scale_vec=P, dx=P, dresidual=P, dweight=P, dscale=P,
                workspace=P, tokens=4, dim=64, dy_token_stride=64, dres_token_stride=64, residual_out_token_stride=64,
                x_token_stride=64, workspace_bytes=need, dtype=1, residual_dtype=0, weight_dtype=0, scale_dtype=0,
                scale=1.0, eps=1e-6)
    bad = [dict(dy=0), dict(residual_out=0), dict(x=0), dict(weight=0), dict(scale_vec=0), dict(workspace=0),
           dict(workspace_bytes=need - 4), dict(dresidual=P + 2), dict(dweight=P + 1), dict(dscale=P + 2)]
    refused(lib, "gdr_add_norm_bwd", _lib.GdrAddNormBwdArgs, base, bad)


def test_linrec_refusals(lib):
    need = lib.gdr_linrec_workspace_bytes(200, 64)
    base = dict(x=P, g=P, h0=P, cu_seqlens=0, h=P, ht=P, states=P, workspace=P, batch=2, tokens=100, dim=64, num_seqs=0,
                x_token_stride=64, g_token_stride=64, workspace_bytes=need, dtype=1, gate_dtype=0, complement=0)
    bad = [dict(x=0), dict(g=0), dict(batch=0), dict(tokens=-1), dict(dim=0), dict(num_seqs=-1),
           dict(num_seqs=3, cu_seqlens=P), dict(batch=1, num_seqs=3), dict(dtype=5), dict(gate_dtype=2), dict(complement=2),
           dict(workspace=0), dict(workspace=P + 16), dict(workspace_bytes=need - 1), dict(h0=P + 2), dict(x=P + 1),
           dict(g_token_stride=-64)]
    refused(lib, "gdr_linrec_fwd", _lib.GdrLinrecFwdArgs, base, bad)
    refused(lib, "gdr_linrec_fwd", _lib.GdrLinrecFwdArgs, base, [dict(tokens=1 << 30)], UNSUPPORTED)
    for k in ("h", "ht"):
        del base[k]
    base.update(dh=P, dht=P, dx=P, dg=P, dh0=P, dh_token_stride=64)
    bad = [dict(x=0), dict(g=0), dict(dh=0), dict(dx=0), dict(dg=0), dict(states=0), dict(dht=P + 1),
           dict(workspace_bytes=need - 1), dict(dh_token_stride=-1)]
    refused(lib, "gdr_linrec_bwd", _lib.GdrLinrecBwdArgs, base, bad)
    assert lib.gdr_linrec_get_status(None, None) == BAD
    assert lib.gdr_linrec_get_status(P + 4, None) == BAD
    base = dict(x=P, g=P, slots=0, state=P, y=P, batch=4, dim=64, num_slots=4, x_token_stride=64, g_token_stride=64,
                dtype=1, gate_dtype=1, complement=0)
    bad = [dict(x=0), dict(g=0), dict(state=0), dict(y=0), dict(batch=-1), dict(dim=0), dict(num_slots=3), dict(dtype=3),
           dict(gate_dtype=2), dict(complement=-1), dict(slots=P + 2), dict(state=P + 2), dict(x_token_stride=-1)]
    refused(lib, "gdr_linrec_step", _lib.GdrLinrecStepArgs, base, bad)


def test_clip_refusals(lib):
    ptrs, sizes, types = (ctypes.c_uint64 * 2)(P, P), (ctypes.c_int64 * 2)(10, 20), (ctypes.c_int32 * 2)(0, 1)
    need = lib.gdr_clip_workspace_bytes(2, 30)
    base = dict(grads=ctypes.addressof(ptrs), outs=0, sizes=ctypes.addressof(sizes), dtypes=ctypes.addressof(types),
                out_dtypes=0, norm=P, workspace=P, count=2, workspace_bytes=need, max_norm=1.0, eps=1e-6)
    null, odd = (ctypes.c_uint64 * 2)(P, 0), (ctypes.c_uint64 * 2)(P + 2, P)
    neg, kinds = (ctypes.c_int64 * 2)(10, -1), (ctypes.c_int32 * 2)(0, 3)
    other = (ctypes.c_int32 * 2)(1, 1)
    bad = [dict(grads=0), dict(sizes=0), dict(dtypes=0), dict(norm=0), dict(norm=P + 2), dict(workspace=0), dict(count=-1),
           dict(workspace_bytes=need - 1), dict(grads=ctypes.addressof(null)), dict(grads=ctypes.addressof(odd)),
           dict(sizes=ctypes.addressof(neg)), dict(dtypes=ctypes.addressof(kinds))]
    refused(lib, "gdr_clip_grad_norm", _lib.GdrClipArgs, base, bad + [
        dict(max_norm=-1.0), dict(max_norm=float("nan")), dict(eps=-1.0), dict(outs=ctypes.addressof(ptrs)),
        dict(outs=ctypes.addressof(ptrs), out_dtypes=ctypes.addressof(other)),  # in place, into another type
        dict(outs=ctypes.addressof(null), out_dtypes=ctypes.addressof(types))])
    refused(lib, "gdr_grad_norm", _lib.GdrClipArgs, base, bad)


def test_torch_calls_refuse_cpu_tensors():
    x, w = torch.ones(2, 3, 8), torch.ones(8)
    for call_ in (lambda: pkg.gated_norm_fwd(x, x, w), lambda: pkg.gated_norm_bwd(x, x, x, w),
                  lambda: pkg.gated_norm(x, x, w), lambda: pkg.add_norm_fwd(x, x, w), lambda: pkg.add_norm(x, x, w),
                  lambda: pkg.add_norm_bwd(x, x, x, w), lambda: pkg.linrec_fwd(x, x), lambda: pkg.linrec_bwd(x, x, x),
                  lambda: pkg.linear_recurrence(x, x), lambda: pkg.linrec_step(x[0], x[0], x[0]),
                  lambda: pkg.clip_grad_norm([x], 1.0), lambda: pkg.grad_norm([x]), lambda: pkg.grad_norm([])):
        with pytest.raises(ValueError):
            call_()
