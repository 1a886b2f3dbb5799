"""The gated feed-forward against its formulas in 64 bits (ffn_util has the bars)."""
import pytest
import torch

import block_util as U
import ffn_util as F
from chunked_gated_delta_09_gb300 import GdrError, _lib, ffn, gated_ffn, gated_ffn_bwd, gated_ffn_fwd
from chunked_gated_delta_09_gb300.ffn import _pack_bwd, _pack_fwd

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16

# tokens, dim, inner: few tokens (up to 32) and more; widths below, at and past the tiles' edges, odd ones; long summed axes
# of few tiles (cut in parts), more tiles than processors
SIZES = [(1, 8, 8), (1, 64, 16), (8, 64, 48), (9, 40, 17), (17, 1001, 100), (31, 33, 7), (32, 2048, 512),
         (33, 64, 128), (64, 4096, 128), (65, 1001, 131), (128, 64, 128), (129, 72, 136), (200, 8, 8), (257, 33, 7),
         (300, 256, 640), (1000, 520, 264), (2048, 64, 64), (2048, 256, 4096), (2500, 1000, 1024), (4100, 2048, 520),
         (9000, 1300, 200), (9001, 1299, 201), (300, 2500, 2600), (301, 2499, 2601), (2500, 257, 2049),
         (2500, 4096, 1024), (2048, 2816, 2048)]  # (these: a last round that is cut; two jobs of several rounds)


@pytest.mark.parametrize("tokens,dim,inner", SIZES)
@pytest.mark.parametrize("dtype", [BF16, F16], ids=["bf16", "f16"])
def test_against_64_bits(tokens, dim, inner, dtype):
    act = ["silu", "sigmoid", "gelu_tanh"][(tokens + inner) % 3]
    x, wg, wu, dh = F.inputs(tokens, tokens, dim, inner, dtype)
    h, saved = gated_ffn_fwd(x, wg, wu, activation=act, return_saved=True, check_status=True)
    g, u = saved
    F.check(dict(h=h, gate=g, up=u), F.forward(x, wg, wu, act))
    d = gated_ffn_bwd(dh, x, wg, wu, saved, activation=act, check_status=True)
    F.check(d, F.backward(dh, x, wg, wu, g, u, act), times=2)
    # the same bits again, without what is kept and from projections that are computed again
    assert torch.equal(gated_ffn_fwd(x, wg, wu, activation=act), h)
    again = gated_ffn_bwd(dh, x, wg, wu, activation=act)
    assert all(torch.equal(again[n], d[n]) for n in d)


@pytest.mark.parametrize("act", ["silu", "sigmoid", "gelu_tanh"])
@pytest.mark.parametrize("tokens", [5, 150])
def test_activations_far_out(act, tokens):
    # projections up to some hundreds: slopes that vanish, exponentials that overflow
    x, wg, wu, dh = F.inputs(7, tokens, 64, 96, BF16)
    x = x * 60
    h, saved = gated_ffn_fwd(x, wg, wu, activation=act, return_saved=True)
    g, u = saved
    F.check(dict(h=h, gate=g, up=u), F.forward(x, wg, wu, act))
    F.check(gated_ffn_bwd(dh, x, wg, wu, saved, activation=act), F.backward(dh, x, wg, wu, g, u, act), times=2)


@pytest.mark.parametrize("lead,dim,inner", [((2, 5), 64, 40), ((3, 4, 30), 136, 72), ((2, 100), 250, 36)])
def test_autograd(lead, dim, inner):
    x, wg, wu, dh = F.inputs(8, None, dim, inner, BF16, lead)
    for t in (x, wg, wu):
        t.requires_grad_()
    h = gated_ffn(x, wg, wu)
    assert h.shape == (*lead, inner)
    f = F.forward(x, wg, wu, "silu")
    F.check(dict(h=h), dict(h=f["h"]))
    grads = torch.autograd.grad(h, (x, wg, wu), dh)
    assert [t.shape for t in grads] == [x.shape, wg.shape, wu.shape]
    F.check(dict(zip(("dx", "dw_gate", "dw_up"), grads)), F.backward(dh, x, wg, wu, f["gate"], f["up"], "silu"), times=2)
    # some of the gradients alone: the same bits
    for wanted in ([0], [1], [2], [0, 2]):
        xs = [t.detach().requires_grad_(i in wanted) for i, t in enumerate((x, wg, wu))]
        got = torch.autograd.grad(gated_ffn(*xs), [xs[i] for i in wanted], dh)
        assert all(torch.equal(a, grads[i]) for a, i in zip(got, wanted))
    (first,) = torch.autograd.grad(gated_ffn(x, wg, wu).float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        first.float().square().sum().backward()
    with torch.no_grad():
        assert torch.equal(gated_ffn(x, wg, wu), h) and not gated_ffn(x, wg, wu).requires_grad
    expanded = torch.autograd.grad(gated_ffn(x, wg, wu).sum(), x)[0]  # a gradient of stride 0
    assert torch.isfinite(expanded).all()


@pytest.mark.parametrize("tokens", [6, 140])
@pytest.mark.parametrize("shift", [0, 1, 8])
def test_parts_of_larger_tensors(tokens, shift):
    dim, inner = 72, 56
    gen = U.seeded(9)
    wide = U.randn(gen, tokens, 2 * dim + 16, dtype=BF16)
    both = U.randn(gen, 2 * inner, dim + 16, dtype=BF16, times=dim ** -0.5)
    dwide = U.randn(gen, tokens, inner + 9, dtype=BF16)
    x, w, dh = wide[:, shift:shift + dim], both[:, shift:shift + dim], dwide[:, shift:shift + inner]
    wg, wu = w[:inner], w[inner:]
    h, saved = gated_ffn_fwd(x, wg, wu, return_saved=True)
    F.check(dict(h=h), dict(h=F.forward(x, wg, wu, "silu")["h"]))
    d = gated_ffn_bwd(dh, x, wg, wu, saved)
    F.check(d, F.backward(dh, x, wg, wu, *saved, "silu"), times=2)
    if shift == 0:  # rows that all are one
        one = x[:1].expand(tokens, dim)
        F.check(dict(h=gated_ffn_fwd(one, wg, wu)), dict(h=F.forward(one, wg, wu, "silu")["h"]))


@pytest.mark.parametrize("tokens", [20, 200])
def test_what_is_not_finite_stays_in_its_row(tokens):
    x, wg, wu, dh = F.inputs(10, tokens, 64, 64, BF16)
    want = gated_ffn_fwd(x, wg, wu)
    x[3, 5], x[7, 60] = float("nan"), float("inf")
    h = gated_ffn_fwd(x, wg, wu)
    rows = [i for i in range(tokens) if i not in (3, 7)]
    assert torch.equal(h[rows], want[rows]) and h[3].isnan().all() and not h[7].isfinite().all()


def test_nothing():
    x, wg, wu, dh = F.inputs(11, 4, 16, 24, BF16)
    h, saved = gated_ffn_fwd(x[:0], wg, wu, return_saved=True)
    assert h.shape == (0, 24)
    d = gated_ffn_bwd(dh[:0], x[:0], wg, wu, saved)
    assert d["dx"].shape == (0, 16) and not d["dw_gate"].any() and not d["dw_up"].any()
    d = gated_ffn_bwd(dh, x, wg, wu, need_dx=False)
    assert d["dx"] is None and d["dw_gate"].any()
    d = gated_ffn_bwd(dh, x, wg, wu, need_dw=False)
    assert d["dw_gate"] is None and d["dw_up"] is None and d["dx"].any()


@pytest.mark.parametrize("tokens,dim,inner", [(7, 24, 40), (7, 25, 41), (190, 72, 200), (190, 73, 199), (700, 64, 64)])
def test_nothing_else_is_written(tokens, dim, inner):
    x, wg, wu, dh = F.inputs(12, tokens, dim, inner, BF16)
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    guard = 4096

    def out(n, dtype=BF16):
        t = torch.full((n + 2 * guard,), 3.0, dtype=dtype, device="cuda")
        return t, t.data_ptr() + t.element_size() * guard

    def kept(t):
        return bool((t[:guard] == 3).all() and (t[-guard:] == 3).all())

    ptrs = [t.data_ptr() for t in (x, wg, wu)]
    (h, hp), (g, gp), (u, up) = (out(tokens * inner, d) for d in (BF16, F32, F32))
    n = lib.gdr_ffn_workspace_bytes(tokens, dim, inner, 1, 0)
    ws = torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda")
    assert lib.gdr_ffn_fwd(_pack_fwd(*ptrs, hp, gp, up, ws.data_ptr(), tokens, dim, inner, dim, dim, dim, n, 1, 0), stream) == 0
    assert kept(h) and kept(g) and kept(u) and (ws[n:] == 7).all()
    (dx, dxp), (dg, dgp), (du, dup) = out(tokens * dim), out(inner * dim), out(inner * dim)
    n = lib.gdr_ffn_workspace_bytes(tokens, dim, inner, 1, 1)
    ws = torch.full((n + 4096,), 7, dtype=torch.uint8, device="cuda")
    assert lib.gdr_ffn_bwd(_pack_bwd(dh.data_ptr(), *ptrs, gp, up, dxp, dgp, dup, ws.data_ptr(), tokens, dim, inner, inner, dim,
                                     dim, dim, n, 1, 0), stream) == 0
    assert kept(dx) and kept(dg) and kept(du) and (ws[n:] == 7).all()
    f = F.forward(x, wg, wu, "silu")
    part = slice(guard, -guard)
    F.check(dict(h=h[part].view(tokens, inner)), dict(h=f["h"]))
    want = F.backward(dh, x, wg, wu, g[part].view(tokens, inner), u[part].view(tokens, inner), "silu")
    F.check(dict(dx=dx[part].view(tokens, dim), dw_gate=dg[part].view(inner, dim), dw_up=du[part].view(inner, dim)), want, times=2)


@pytest.mark.parametrize("tokens", [12, 500])
def test_streams_and_graphs(tokens):
    x, wg, wu, dh = F.inputs(13, tokens, 128, 192, F16)
    h, saved = gated_ffn_fwd(x, wg, wu, return_saved=True)
    d = gated_ffn_bwd(dh, x, wg, wu, saved)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h2, saved2 = gated_ffn_fwd(x, wg, wu, return_saved=True, stream=side)
    d2 = gated_ffn_bwd(dh, x, wg, wu, saved2, stream=side)
    side.synchronize()
    assert torch.equal(h, h2) and all(torch.equal(d[n], d2[n]) for n in d)
    graph = torch.cuda.CUDAGraph()
    keep = x.clone()
    with torch.cuda.graph(graph):
        h3, saved3 = gated_ffn_fwd(x, wg, wu, return_saved=True)
        d3 = gated_ffn_bwd(dh, x, wg, wu, saved3)
    x.zero_()
    graph.replay()
    assert not h3.any()
    x.copy_(keep)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(h, h3) and all(torch.equal(d[n], d3[n]) for n in d)


def test_two_calls_at_once():
    parts = [F.inputs(14 + i, 700, 256, 512, BF16) for i in range(2)]
    want = [gated_ffn_fwd(x, wg, wu) for x, wg, wu, _ in parts]
    streams = [torch.cuda.Stream() for _ in parts]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    got = [[gated_ffn_fwd(x, wg, wu, stream=s) for (x, wg, wu, _), s in zip(parts, streams)] for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))


@pytest.mark.parametrize("tokens,dim,inner", [(600, 512, 512), (5000, 256, 1024), (5000, 2048, 64), (640, 2560, 2560)])
def test_waits_that_run_out_are_reported(monkeypatch, tokens, dim, inner):
    x, wg, wu, dh = F.inputs(16, tokens, dim, inner, BF16)
    want, saved = gated_ffn_fwd(x, wg, wu, return_saved=True, check_status=True)
    monkeypatch.setenv("GDR_SPIN_LIMIT", "1")
    for call in (lambda: gated_ffn_fwd(x, wg, wu, check_status=True),
                 lambda: gated_ffn_bwd(dh, x, wg, wu, saved, check_status=True)):
        with pytest.raises(GdrError) as e:
            call()
        assert e.value.status == _lib.GDR_ERR_TIMEOUT
    monkeypatch.delenv("GDR_SPIN_LIMIT")
    assert torch.equal(gated_ffn_fwd(x, wg, wu, check_status=True), want)


def z(*shape, dtype=BF16):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


REFUSED = {
    "fp32": lambda: gated_ffn_fwd(z(4, 8, dtype=torch.float32), z(16, 8, dtype=torch.float32), z(16, 8, dtype=torch.float32)),
    "types": lambda: gated_ffn_fwd(z(4, 8), z(16, 8, dtype=F16), z(16, 8)),
    "widths": lambda: gated_ffn_fwd(z(4, 8), z(16, 9), z(16, 9)),
    "two widths": lambda: gated_ffn_fwd(z(4, 8), z(16, 8), z(15, 8)),
    "weight layout": lambda: gated_ffn_fwd(z(4, 8), z(8, 16).t(), z(16, 8)),
    "rows": lambda: gated_ffn_fwd(z(4, 3, 8)[:, :2], z(16, 8), z(16, 8)),
    "columns": lambda: gated_ffn_fwd(z(4, 16)[:, ::2], z(16, 8), z(16, 8)),
    "activation": lambda: gated_ffn_fwd(z(4, 8), z(16, 8), z(16, 8), activation="relu"),
    "one axis of weights": lambda: gated_ffn_fwd(z(4, 8), z(8), z(8)),
    "dh": lambda: gated_ffn_bwd(z(4, 8), z(4, 8), z(16, 8), z(16, 8)),
    "saved": lambda: gated_ffn_bwd(z(4, 16), z(4, 8), z(16, 8), z(16, 8), z(2, 4, 8, dtype=F32)),
    "saved type": lambda: gated_ffn_bwd(z(4, 16), z(4, 8), z(16, 8), z(16, 8), z(2, 4, 16)),
    "saved layout": lambda: gated_ffn_bwd(z(4, 16), z(4, 8), z(16, 8), z(16, 8), z(2, 16, 4, dtype=F32).transpose(1, 2)),
    "empty width": lambda: gated_ffn_fwd(z(4, 0), z(16, 0), z(16, 0)),
}


@pytest.mark.parametrize("name", REFUSED)
def test_refused(name):
    with pytest.raises(ValueError):
        REFUSED[name]()


def test_offsets_beyond_32_bits():
    tokens, dim, inner = 270000, 64, 8192  # 2.2e9 values of h
    _, wg, wu, _ = F.inputs(17, 1, dim, inner, BF16)
    x = torch.randn(tokens, dim, dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    dh = torch.randn(tokens, inner, dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    h, saved = gated_ffn_fwd(x, wg, wu, return_saved=True, check_status=True)
    rows = torch.tensor([0, 1, 131071, 262143, 262144, tokens - 1], device="cuda")
    f = F.forward(x[rows], wg, wu, "silu")
    F.check(dict(h=h[rows], gate=saved[0][rows], up=saved[1][rows]), f)
    d = gated_ffn_bwd(dh, x, wg, wu, saved, check_status=True)
    F.check(dict(dx=d["dx"][rows]), dict(dx=F.backward(dh[rows], x[rows], wg, wu, f["gate"], f["up"], "silu")["dx"]), times=2)
    part = slice(inner - 16, inner)
    f = F.forward(x, wg[part], wu[part], "silu")
    want = F.backward(dh[:, part], x, wg[part], wu[part], f["gate"], f["up"], "silu")
    F.check({n: d[n][part] for n in ("dw_gate", "dw_up")}, {n: want[n] for n in ("dw_gate", "dw_up")}, times=2)


# Rows that are copied to 16-byte boundaries, of more than 2^32 elements in all: the first row past it, its neighbours, and the rows
# that an offset of 32 bits would take for those.
LONG, ODD = 1048000, 4097
PAST = -(-2 ** 32 // 4104)
AROUND = [0, 1, PAST - 1, PAST, PAST + 1, LONG - PAST - 1, LONG - PAST, LONG - 1]


def test_copied_tokens_beyond_32_bits():
    inner = 24
    _, wg, wu, _ = F.inputs(18, 1, ODD, inner, BF16)
    x = torch.randn(LONG, ODD, dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(3))
    dh = torch.randn(LONG, inner, dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    h, saved = gated_ffn_fwd(x, wg, wu, return_saved=True, check_status=True)
    rows = torch.tensor(AROUND, device="cuda")
    for some in (rows, slice(0, 256), slice(PAST - 128, PAST + 128), slice(LONG - 256, LONG)):
        F.check(dict(h=h[some], gate=saved[0][some], up=saved[1][some]), F.forward(x[some], wg, wu, "silu"))
    d = gated_ffn_bwd(dh, x, wg, wu, saved, check_status=True)
    want = F.backward(dh[rows], x[rows], wg, wu, saved[0][rows], saved[1][rows], "silu")
    F.check(dict(dx=d["dx"][rows]), dict(dx=want["dx"]), times=2)
    sums = {n: torch.zeros(inner, ODD, dtype=torch.float64, device="cuda") for n in ("dw_gate", "dw_up")}
    for i in range(0, LONG, 1 << 17):
        some = slice(i, i + (1 << 17))
        part = F.backward(dh[some], x[some], wg, wu, saved[0][some], saved[1][some], "silu")
        for n in sums:
            sums[n] += part[n]
    F.check({n: d[n] for n in sums}, sums, times=2)


def test_copied_weights_beyond_32_bits():
    tokens = 40
    x, _, _, _ = F.inputs(19, tokens, ODD, 1, BF16)
    wg, wu = (torch.randn(LONG, ODD, dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(s)).mul_(ODD ** -0.5)
              for s in (5, 6))
    dh = torch.randn(tokens, LONG, dtype=BF16, device="cuda", generator=torch.Generator("cuda").manual_seed(7))
    h, saved = gated_ffn_fwd(x, wg, wu, return_saved=True, check_status=True)
    for some in (torch.tensor(AROUND, device="cuda"), slice(0, 256), slice(PAST - 128, PAST + 128), slice(LONG - 256, LONG)):
        F.check(dict(h=h[:, some], gate=saved[0][:, some], up=saved[1][:, some]), F.forward(x, wg[some], wu[some], "silu"))
    d = gated_ffn_bwd(dh, x, wg, wu, saved, need_dw=False, check_status=True)
    want = torch.zeros(tokens, ODD, dtype=torch.float64, device="cuda")
    for i in range(0, LONG, 1 << 17):
        some = slice(i, i + (1 << 17))
        want += F.backward(dh[:, some], x, wg[some], wu[some], saved[0][:, some], saved[1][:, some], "silu")["dx"]
    F.check(dict(dx=d["dx"]), dict(dx=want), times=2)


def test_projections_computed_again_report_their_waits(monkeypatch):
    x, wg, wu, dh = F.inputs(20, 600, 512, 512, BF16)
    want = gated_ffn_bwd(dh, x, wg, wu, check_status=True)

    def short(*args, **kwargs):  # the limit holds for the forward pass inside the call alone
        monkeypatch.setenv("GDR_SPIN_LIMIT", "1")
        try:
            return gated_ffn_fwd(*args, **kwargs)
        finally:
            monkeypatch.delenv("GDR_SPIN_LIMIT")

    with monkeypatch.context() as m:
        m.setattr(ffn, "gated_ffn_fwd", short)
        with pytest.raises(GdrError) as e:
            gated_ffn_bwd(dh, x, wg, wu, check_status=True)
        assert e.value.status == _lib.GDR_ERR_TIMEOUT
    again = gated_ffn_bwd(dh, x, wg, wu, check_status=True)
    assert all(torch.equal(again[n], want[n]) for n in want)


@pytest.mark.parametrize("which", [0, 1, 2])
@pytest.mark.parametrize("grad", [True, False])
def test_forward_mode_is_refused(which, grad):
    parts = list(F.inputs(21, 5, 16, 24, BF16)[:3])
    with torch.set_grad_enabled(grad), torch.autograd.forward_ad.dual_level():
        want = gated_ffn(*parts)  # no tangents: as without the level
        dual = list(parts)
        dual[which] = torch.autograd.forward_ad.make_dual(parts[which], torch.ones_like(parts[which]))
        with pytest.raises(NotImplementedError):
            gated_ffn(*dual)
    assert torch.equal(gated_ffn(*parts), want)


def test_every_cta_has_a_report_of_its_own(monkeypatch):
    tokens, dim, inner = 640, 512, 512
    x, wg, wu, _ = F.inputs(23, tokens, dim, inner, BF16)
    h = torch.empty(tokens, inner, dtype=BF16, device="cuda")
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    n = lib.gdr_ffn_workspace_bytes(tokens, dim, inner, 0, 0)
    ws = torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    packed = _pack_fwd(x.data_ptr(), wg.data_ptr(), wu.data_ptr(), h.data_ptr(), 0, 0, ws.data_ptr(), tokens, dim, inner, dim, dim,
                       dim, n, 1, 0)
    status = ws[:_lib.FFN_STATUS_BYTES]
    assert lib.gdr_ffn_fwd(packed, stream) == 0
    assert not status.any()  # also what an earlier call of more CTAs would have left
    monkeypatch.setenv("GDR_SPIN_LIMIT", "1")
    assert lib.gdr_ffn_fwd(packed, stream) == 0
    monkeypatch.delenv("GDR_SPIN_LIMIT")
    assert int((status != 0).sum()) > 1
    assert lib.gdr_ffn_get_status(ws.data_ptr(), stream) == _lib.GDR_ERR_TIMEOUT
    assert lib.gdr_ffn_get_status(ws.data_ptr(), stream) == 0


@pytest.mark.parametrize("call", ["few tokens", "no tokens", "no tokens backward", "nothing wanted"])
def test_calls_that_wait_for_nothing_clear_the_status(monkeypatch, call):
    tokens, dim, inner = 600, 64, 96
    x, wg, wu, dh = F.inputs(22, tokens, dim, inner, BF16)
    h = torch.empty_like(dh)
    g, u = torch.zeros(2, tokens, inner, device="cuda")
    lib, stream = _lib.load(), torch.cuda.current_stream().cuda_stream
    n = lib.gdr_ffn_workspace_bytes(tokens, dim, inner, 0, 1)
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ptrs = [t.data_ptr() for t in (x, wg, wu)]

    def fwd(count):
        return lib.gdr_ffn_fwd(_pack_fwd(*ptrs, h.data_ptr(), 0, 0, ws.data_ptr(), count, dim, inner, dim, dim, dim, n, 1, 0), stream)

    def bwd(count):
        return lib.gdr_ffn_bwd(_pack_bwd(dh.data_ptr(), *ptrs, g.data_ptr(), u.data_ptr(), 0, 0, 0, ws.data_ptr(), count, dim,
                                         inner, inner, dim, dim, dim, n, 1, 0), stream)

    calls = {"few tokens": lambda: fwd(8), "no tokens": lambda: fwd(0), "no tokens backward": lambda: bwd(0),
             "nothing wanted": lambda: bwd(tokens)}
    monkeypatch.setenv("GDR_SPIN_LIMIT", "1")
    assert fwd(tokens) == 0
    assert lib.gdr_ffn_get_status(ws.data_ptr(), stream) == _lib.GDR_ERR_TIMEOUT
    assert fwd(tokens) == 0
    monkeypatch.delenv("GDR_SPIN_LIMIT")
    assert calls[call]() == 0
    assert lib.gdr_ffn_get_status(ws.data_ptr(), stream) == 0
