"""The norms around a block (gated_norm, add_norm) on the GPU against their 64-bit forms, their gradients against the
formulas and against differences, odd sizes, strides, and bit-identical repeats."""
import pytest
import torch

import block_util as U
from chunked_gated_delta_09_gb300 import (add_norm, add_norm_bwd, add_norm_fwd, gated_norm, gated_norm_bwd,
                                          gated_norm_fwd)

pytestmark = pytest.mark.gpu

EPS = 1e-5
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def check_gated(x, z, w, dy, act):
    got = dict(y=gated_norm_fwd(x, z, w, eps=EPS, activation=act))
    got.update(gated_norm_bwd(dy, x, z, w, eps=EPS, activation=act))
    U.check(got, U.gated_norm(x, z, w, EPS, act, dy))
    return got


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("shape", [(1, 1, 1), (1, 3, 7), (5, 3, 8), (33, 2, 40), (7, 16, 128), (301, 3, 64), (19, 2, 129),
                                   (3, 1, 512), (9, 1, 1000), (3, 2, 2048), (2, 1, 4100), (3, 1, 6152), (2, 1, 16384)])
def test_gated_norm_sizes(shape, dtype):
    dt, gen = TYPES[dtype], U.seeded(sum(shape))
    x, z, dy = (U.randn(gen, *shape, dtype=dt) for _ in range(3))
    w = (1.0 + U.randn(gen, shape[-1], times=0.2)).to(dt)
    check_gated(x, z, w, dy, "silu")


@pytest.mark.parametrize("act", ["silu", "sigmoid"])
@pytest.mark.parametrize("gate,weight", [(True, None), (False, torch.float32), (False, None), (True, torch.float16)])
def test_gated_norm_parts_may_be_absent(act, gate, weight):
    gen = U.seeded(3)
    x, z, dy = (U.randn(gen, 2, 37, 3, 96, dtype=torch.bfloat16) for _ in range(3))
    w = None if weight is None else (1.0 + U.randn(gen, 96, times=0.2)).to(weight)
    check_gated(x, z if gate else None, w, dy, act)


@pytest.mark.parametrize("dim,pad", [(64, 0), (64, 8), (64, 3), (63, 1)])
def test_gated_norm_takes_slices_of_a_projection(dim, pad):
    """x, z and dy as columns of wider rows, at aligned and odd distances."""
    gen = U.seeded(dim + pad)
    heads, n = 3, 45
    wide = U.randn(gen, 2, n, 3 * heads * dim + pad, dtype=torch.bfloat16)
    x, z, dy = (wide[..., i * heads * dim:(i + 1) * heads * dim].unflatten(-1, (heads, dim)) for i in range(3))
    assert not x.is_contiguous()
    check_gated(x, z, (1.0 + U.randn(gen, dim, times=0.2)), dy, "silu")


def test_gated_norm_heads_may_be_strided():
    gen = U.seeded(9)
    x = U.randn(gen, 21, 4, 2, 32)[:, :, 1]
    z = U.randn(gen, 4, 21, 32).transpose(0, 1)
    dy = U.randn(gen, 1, 1, 32).expand(21, 4, 32)
    check_gated(x, z, U.randn(gen, 32), dy, "sigmoid")


def test_gated_norm_extreme_values():
    """A row of zeros (rms 0), gates far out on both sides, and a nan that stays in its row."""
    gen = U.seeded(4)
    x, z, dy = (U.randn(gen, 6, 2, 64) for _ in range(3))
    x[1] = 0.0
    z[2], z[3] = -200.0, 200.0
    x[4] *= 1e-18
    w = U.randn(gen, 64)
    check_gated(x, z, w, dy, "silu")
    x[5, 0, 3] = float("nan")
    y = gated_norm_fwd(x, z, w, eps=EPS)
    assert torch.isnan(y[5, 0]).all() and torch.isfinite(y[:5]).all() and torch.isfinite(y[5, 1]).all()


def test_norms_of_no_tokens():
    x = torch.empty(0, 2, 64, device="cuda")
    w = torch.ones(64, device="cuda")
    assert gated_norm_fwd(x, x, w).shape == x.shape
    d = gated_norm_bwd(x, x, x, w)
    assert d["dx"].shape == x.shape and torch.equal(d["dweight"], torch.zeros_like(w))
    x = torch.empty(2, 0, 64, device="cuda")
    y, r = add_norm_fwd(x, x, w, w)
    assert y.shape == r.shape == x.shape
    d = add_norm_bwd(x, x, x, w, w, x=x)
    assert torch.equal(d["dweight"], torch.zeros_like(w)) and torch.equal(d["dscale"], torch.zeros_like(w))


def check_add(x, res, w, scale, dy, dres):
    y, r = add_norm_fwd(x, res, w, scale, eps=EPS)
    U.check(dict(y=y, r=r), U.add_norm_fwd(x, res, w, scale, EPS))
    xs = x if isinstance(scale, torch.Tensor) else None
    got = add_norm_bwd(dy, dres, r, w, scale, x=xs, eps=EPS)
    U.check(got, U.add_norm_bwd(dy, dres, r, w, scale, xs, EPS))
    return y, r, got


@pytest.mark.parametrize("scale", ["one", "number", "channel"])
@pytest.mark.parametrize("dtype,rtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("shape", [(1, 1), (3, 7), (1, 2048), (70, 64), (9, 1000), (33, 200), (5, 515), (4, 4096), (3, 8200),
                                   (2, 16384), (2, 16383)])
def test_add_norm_sizes(shape, dtype, rtype, scale):
    gen = U.seeded(sum(shape))
    dt, rt = TYPES[dtype], TYPES[rtype]
    x, dy = (U.randn(gen, *shape, dtype=dt) for _ in range(2))
    res, dres = (U.randn(gen, *shape, dtype=rt, times=2.0) for _ in range(2))
    w = (1.0 + U.randn(gen, shape[-1], times=0.2)).to(dt)
    s = {"one": 1.0, "number": -0.3}.get(scale)
    check_add(x, res, w, (0.5 + U.randn(gen, shape[-1], times=0.2)) if s is None else s, dy, dres)


def test_add_norm_many_rows():
    """More rows than the grid holds at a time, so that the column sums run over several rows and CTAs."""
    gen = U.seeded(12)
    x, dy = (U.randn(gen, 5003, 72, dtype=torch.bfloat16) for _ in range(2))
    res, dres = (U.randn(gen, 5003, 72) for _ in range(2))
    check_add(x, res, 1.0 + U.randn(gen, 72, times=0.2), 0.5 + U.randn(gen, 72, times=0.2), dy, dres)
    x, dy, res, dres = (U.randn(gen, 1301, 4096, dtype=torch.bfloat16) for _ in range(4))
    check_add(x, res, 1.0 + U.randn(gen, 4096, times=0.2), 0.5 + U.randn(gen, 4096, times=0.2), dy, dres)
    x, z, dy = (U.randn(gen, 4001, 5, 48, dtype=torch.bfloat16) for _ in range(3))
    check_gated(x, z, 1.0 + U.randn(gen, 48, times=0.2), dy, "silu")


@pytest.mark.parametrize("dtype,rtype", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("dim", [4104, 8200, 12288, 16376])
def test_rows_that_several_ctas_share(dim, dtype, rtype):
    """More rows than the device holds clusters, whose last CTAs have fewer columns."""
    gen = U.seeded(dim)
    dt, rt = TYPES[dtype], TYPES[rtype]
    x, dy = (U.randn(gen, 331, dim, dtype=dt) for _ in range(2))
    res, dres = (U.randn(gen, 331, dim, dtype=rt, times=2.0) for _ in range(2))
    w, s = (1.0 + U.randn(gen, dim, times=0.2) for _ in range(2))
    check_add(x, res, w, s, dy, dres)
    check_gated(x.view(331, 1, dim), res.to(dt).view(331, 1, dim), w, dy.view(331, 1, dim), "silu")


def test_add_norm_parts_may_be_absent():
    gen = U.seeded(13)
    x, dy = (U.randn(gen, 2, 11, 80, dtype=torch.bfloat16) for _ in range(2))
    y, r, got = check_add(x, None, None, 1.0, dy, None)
    assert torch.equal(r, x) and got["dweight"] is None and got["dscale"] is None
    assert got["dx"] is got["dresidual"]
    check_add(x, None, U.randn(gen, 80), U.randn(gen, 80), dy, None)


def test_add_norm_strided_rows():
    gen = U.seeded(14)
    for pad in (8, 3):
        wide = U.randn(gen, 3, 17, 4 * 64 + pad, dtype=torch.float16)
        x, res, dy, dres = (wide[..., i * 64:(i + 1) * 64] for i in range(4))
        check_add(x, res, U.randn(gen, 64), 0.5, dy, dres)
    check_add(U.randn(gen, 1, 64).expand(9, 64), U.randn(gen, 9, 64), U.randn(gen, 64), 0.5, U.randn(gen, 9, 64),
              U.randn(gen, 9, 64))


def test_results_repeat_bit_for_bit():
    gen = U.seeded(15)
    x, dy = (U.randn(gen, 3000, 256, dtype=torch.bfloat16) for _ in range(2))
    res, dres = (U.randn(gen, 3000, 256) for _ in range(2))
    w, s = U.randn(gen, 256), U.randn(gen, 256)
    _, r = add_norm_fwd(x, res, w, s)
    a, b = (add_norm_bwd(dy, dres, r, w, s, x=x) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)
    x, z, dy = (U.randn(gen, 3000, 2, 128, dtype=torch.bfloat16) for _ in range(3))
    a, b = (gated_norm_bwd(dy, x, z, w[:128]) for _ in range(2))
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_autograd_and_differences():
    """The Functions' gradients against central differences of the 64-bit forward, and with expanded incoming ones."""
    gen = U.seeded(16)
    x, z = (U.randn(gen, 4, 2, 24).requires_grad_() for _ in range(2))
    w = U.randn(gen, 24).requires_grad_()
    gated_norm(x, z, w, eps=EPS).sum().backward()  # the incoming gradient is an expanded 1
    leaves = dict(x=x, z=z, w=w)

    def loss(**at):
        v = {k: at.get(k, U.f64(t)) for k, t in leaves.items()}
        return float(U.gated_norm(v["x"], v["z"], v["w"], EPS, "silu")["y"].sum())

    _differences(loss, leaves, gen)
    x, res = (U.randn(gen, 5, 24).requires_grad_() for _ in range(2))
    w, s = (U.randn(gen, 24).requires_grad_() for _ in range(2))
    cy, cr = (U.randn(gen, 5, 24) for _ in range(2))
    y, r = add_norm(x, res, w, s, eps=EPS)
    ((y * cy).sum() + (r * cr).sum()).backward()
    leaves = dict(x=x, res=res, w=w, s=s)

    def loss(**at):
        v = {k: at.get(k, U.f64(t)) for k, t in leaves.items()}
        o = U.add_norm_fwd(v["x"], v["res"], v["w"], v["s"], EPS)
        return float((o["y"] * U.f64(cy)).sum() + (o["r"] * U.f64(cr)).sum())

    _differences(loss, leaves, gen)


def _differences(loss, leaves, gen):
    """Along a random direction of each leaf; h = 1e-5: truncation 1e-10 and cancellation 1e-11 of order-1 values, so the
    fp32 gradient's own bar decides."""
    for name, leaf in leaves.items():
        d = torch.randn(leaf.shape, generator=gen, dtype=torch.float64)
        at = U.f64(leaf)
        diff = (loss(**{name: at + 1e-5 * d}) - loss(**{name: at - 1e-5 * d})) / 2e-5
        grad = U.f64(leaf.grad)
        assert abs(float((grad * d).sum()) - diff) <= U.FP32_BAR * float(grad.norm() * d.norm()) + 1e-8, name


def test_another_stream():
    gen = U.seeded(17)
    x, z = (U.randn(gen, 500, 4, 128, dtype=torch.bfloat16) for _ in range(2))
    w = U.randn(gen, 128)
    ref = gated_norm_fwd(x, z, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y = gated_norm_fwd(x, z, w, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, ref)


def test_rows_beyond_32_bits():
    """More than 2^31 elements: the last rows are those of a call on them alone."""
    n, dim, tail = 140000, 16384, 9
    gen = torch.Generator("cuda").manual_seed(18)
    x = torch.empty(n, dim, device="cuda", dtype=torch.bfloat16)
    x[-tail:] = torch.randn(tail, dim, generator=gen, device="cuda").bfloat16()
    x[:-tail] = 1.0
    w = torch.ones(dim, device="cuda")
    y, r = add_norm_fwd(x, x, w, 0.5)
    ref_y, ref_r = add_norm_fwd(x[-tail:], x[-tail:], w, 0.5)
    assert torch.equal(y[-tail:], ref_y) and torch.equal(r[-tail:], ref_r)
    assert torch.equal(gated_norm_fwd(x[:, None], x[:, None], w)[-tail:, 0], gated_norm_fwd(x[-tail:, None], x[-tail:, None], w)[:, 0])


@pytest.mark.parametrize("rows", [1, 4, 5, 64, 65, 130])
def test_column_sums_of_few_rows(rows):
    """Around the numbers of rows up to which one CTA writes the sums itself."""
    gen = U.seeded(rows)
    for dim in (64, 128, 700, 2048):
        x, res, dy, dres = (U.randn(gen, rows, dim, dtype=torch.bfloat16) for _ in range(4))
        check_add(x, res, 1.0 + U.randn(gen, dim, times=0.2), 0.5 + U.randn(gen, dim, times=0.2), dy, dres)
        check_gated(x[:, None], res[:, None], 1.0 + U.randn(gen, dim, times=0.2), dy[:, None], "silu")


def test_capture_in_a_graph():
    gen = U.seeded(19)
    x, z, dy = (U.randn(gen, 2000, 4, 64, dtype=torch.bfloat16) for _ in range(3))
    w = U.randn(gen, 64)
    ref = gated_norm_bwd(dy, x, z, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = gated_norm_bwd(dy, x, z, w)
    graph.replay()
    assert all(torch.equal(got[k], ref[k]) for k in ref)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows", [1, 3, 37, 300])
@pytest.mark.parametrize("dim", [5, 64, 100, 128, 200, 256, 700])
def test_eps_of_zero(dim, rows, dtype):
    """No row here is zero, so nothing divides by zero: rows past the end, of which a CTA has some, must not either."""
    dt, gen = TYPES[dtype], U.seeded(dim + rows)
    x, z, dy = (U.randn(gen, rows, 1, dim, dtype=dt) for _ in range(3))
    w, s = (1.0 + U.randn(gen, dim, times=0.2) for _ in range(2))
    got = dict(y=gated_norm_fwd(x, z, w, eps=0.0))
    got.update(gated_norm_bwd(dy, x, z, w, eps=0.0))
    U.check(got, U.gated_norm(x, z, w, 0.0, "silu", dy))
    x, res, dy, dres = x[:, 0], z[:, 0].float(), dy[:, 0], U.randn(gen, rows, dim)
    y, r = add_norm_fwd(x, res, w, s, eps=0.0)
    U.check(dict(y=y, r=r), U.add_norm_fwd(x, res, w, s, 0.0))
    got = add_norm_bwd(dy, dres, r, w, s, x=x, eps=0.0)
    U.check(got, U.add_norm_bwd(dy, dres, r, w, s, x, 0.0))
