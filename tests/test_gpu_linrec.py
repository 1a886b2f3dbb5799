"""The gated linear recurrence on the GPU against the token-by-token 64-bit form: dense and packed sequences, lengths of
zero and one, odd sizes and strides, its backward with and without saved states, its single-token step."""
import pytest
import torch

import block_util as U
from chunked_gated_delta_09_gb300 import GdrError, _lib, block, linear_recurrence, linrec_bwd, linrec_fwd, linrec_step

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def problem(B, T, D, dtype, gtype, seed, lens=None):
    gen = U.seeded(seed)
    dt, gt = TYPES[dtype], TYPES[gtype]
    N = B if lens is None else len(lens)
    cu = None
    if lens is not None:
        cu = torch.tensor([sum(lens[:i]) for i in range(N + 1)], dtype=torch.int32, device="cuda")
    return dict(x=U.randn(gen, B, T, D, dtype=dt), g=U.gates(gen, B, T, D, dtype=gt), h0=U.randn(gen, N, D),
                cu_seqlens=cu), dict(dh=U.randn(gen, B, T, D, dtype=dt), dht=U.randn(gen, N, D))


def check(p, d, lens, complement):
    h, ht, states = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"], complement=complement, return_states=True,
                               check_status=True)
    got = dict(h=h, ht=ht)
    got.update(linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], p["cu_seqlens"], states, complement=complement,
                          check_status=True))
    U.check(got, U.linrec(p["x"], p["g"], p["h0"], lens, complement, d["dh"], d["dht"]))
    return got


@pytest.mark.parametrize("complement", [False, True], ids=["plain", "complement"])
@pytest.mark.parametrize("dtype,gtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("B,T,D", [(1, 1, 1), (3, 1, 40), (2, 7, 33), (1, 64, 128), (2, 65, 130), (3, 200, 8),
                                   (1, 300, 256), (5, 63, 31)])
def test_dense(B, T, D, dtype, gtype, complement):
    p, d = problem(B, T, D, dtype, gtype, seed=B + T + D)
    check(p, d, None, complement)


@pytest.mark.parametrize("D", [64, 37])
@pytest.mark.parametrize("lens", [[5], [0, 3, 0, 0, 130, 1, 1, 64, 0], [64, 64, 64], [1] * 70, [63, 65, 1, 127, 200],
                                  [0, 0, 9], [2000, 3, 900]], ids=str)
def test_packed(lens, D):
    p, d = problem(1, sum(lens), D, "bf16", "f32", seed=len(lens) + D, lens=lens)
    check(p, d, lens, True)


@pytest.mark.parametrize("T,D", [(20000, 32), (5000, 200)])
def test_long_sequences(T, D):
    """Enough rows that a state passes through many tiles."""
    p, d = problem(1, T, D, "f32", "f32", seed=T)
    check(p, d, None, False)


def test_no_tokens():
    p, d = problem(2, 0, 8, "f32", "f32", seed=1)
    h, ht = linrec_fwd(p["x"], p["g"], p["h0"])
    assert h.shape == (2, 0, 8) and torch.equal(ht, p["h0"])
    got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"])
    assert torch.equal(got["dh0"], d["dht"])
    p, d = problem(1, 0, 8, "f32", "f32", seed=1, lens=[0, 0])
    h, ht = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"], check_status=True)
    assert torch.equal(ht, p["h0"])


def test_absent_states_and_backward_without_saved_states():
    p, d = problem(1, 400, 48, "bf16", "f32", seed=2, lens=[150, 0, 250])
    p["h0"] = None
    d["dht"] = None
    got = check(p, d, [150, 0, 250], True)
    again = linrec_bwd(p["x"], p["g"], d["dh"], None, None, p["cu_seqlens"], complement=True)
    assert all(torch.equal(got[k], again[k]) for k in again)


def test_strided_rows():
    gen = U.seeded(5)
    for pad in (8, 3):
        wide = U.randn(gen, 2, 90, 3 * 64 + pad, dtype=torch.bfloat16)
        x, dh = wide[..., :64], wide[..., 64:128]
        g = U.gates(gen, 2, 90, 128, dtype=torch.bfloat16)[..., 5:69]
        p = dict(x=x, g=g, h0=U.randn(gen, 2, 64), cu_seqlens=None)
        check(p, dict(dh=dh, dht=U.randn(gen, 2, 64)), None, True)


def test_a_gate_of_zero_and_a_nan_stay_in_their_place():
    """a = 0 (g = -inf) forgets the past; a nan reaches the rest of its own sequence and no other one."""
    lens = [100, 90, 80]
    p, d = problem(1, 270, 36, "f32", "f32", seed=6, lens=lens)
    p["g"][0, 50] = float("-inf")
    p["g"][0, 129, 3] = float("-inf")
    p["g"][0, 200] = 0.0
    check(p, d, lens, True)
    clean, _ = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"])
    p["x"][0, 110, 7] = float("nan")
    h, ht, states = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"], return_states=True)
    bad = torch.isnan(h)
    assert bad[0, 110:190, 7].all() and bad.sum() == 80
    assert torch.equal(h[~bad], clean[~bad]) and torch.isnan(ht).sum() == 1
    d["dh"][0, 195, 2] = float("inf")
    got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], p["cu_seqlens"], states)
    assert torch.isfinite(got["dx"][0, :190]).all() and torch.isfinite(got["dx"][0, 196:]).all()


def test_results_repeat_bit_for_bit():
    p, d = problem(1, 9000, 96, "bf16", "f32", seed=7)
    first = None
    for _ in range(5):
        h, ht, states = linrec_fwd(p["x"], p["g"], p["h0"], return_states=True)
        got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], None, states)
        now = [h, ht, *got.values()]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


@pytest.mark.parametrize("cu", [[0, 100, 60, 201], [1, 50, 100, 201], [0, 50, 100, 200], [0, 50, 300, 201],
                                [0, -5, 100, 201]], ids=str)
def test_malformed_cu_seqlens_are_reported(cu):
    p, d = problem(1, 201, 40, "f32", "f32", seed=8, lens=[100, 50, 51])
    _, _, states = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"], return_states=True, check_status=True)
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    with pytest.raises(GdrError) as e:
        linrec_fwd(p["x"], p["g"], p["h0"], bad, check_status=True)
    assert e.value.status == _lib.GDR_ERR_DEVICE
    with pytest.raises(GdrError) as e:
        linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], bad, states, check_status=True)
    assert e.value.status == _lib.GDR_ERR_DEVICE


def test_autograd_and_differences():
    p, _ = problem(1, 150, 20, "f32", "f32", seed=9, lens=[70, 1, 79])
    leaves = {k: p[k].requires_grad_() for k in ("x", "g", "h0")}
    h, ht = linear_recurrence(p["x"], p["g"], p["h0"], p["cu_seqlens"], complement=True)
    (h.sum() + 2.0 * ht.sum()).backward()
    gen = U.seeded(10)
    for name, leaf in leaves.items():
        d = torch.randn(leaf.shape, generator=gen, dtype=torch.float64)

        def loss(step):
            v = {k: U.f64(t) + (step * d if k == name else 0.0) for k, t in leaves.items()}
            o = U.linrec(v["x"], v["g"], v["h0"], [70, 1, 79], True)
            return float(o["h"].sum() + 2.0 * o["ht"].sum())

        diff = (loss(1e-5) - loss(-1e-5)) / 2e-5
        grad = U.f64(leaf.grad)
        # truncation h^2 f''' / 6 with sums over up to 79 tokens: below 1e-6 of the gradient's size
        assert abs(float((grad * d).sum()) - diff) <= 2 * U.FP32_BAR * float(grad.norm() * d.norm()), name


# ---------------------------------------------------------------- single tokens
@pytest.mark.parametrize("complement", [False, True], ids=["plain", "complement"])
@pytest.mark.parametrize("dtype,gtype", [("f32", "f32"), ("bf16", "f32"), ("f16", "f16")])
@pytest.mark.parametrize("B,D,pad", [(1, 1, 0), (3, 33, 0), (64, 2048, 0), (5, 64, 8), (7, 64, 3)])
def test_step(B, D, pad, dtype, gtype, complement):
    gen = U.seeded(B + D + pad)
    x = U.randn(gen, B, D + pad, dtype=TYPES[dtype])[:, :D]
    g = U.gates(gen, B, D + pad, dtype=TYPES[gtype])[:, :D]
    state = U.randn(gen, B + 9, D)
    slots = torch.randperm(B + 9, generator=gen)[:B].to(torch.int32).cuda()
    if B > 2:
        slots[1] = -1
    if B > 4:
        slots[3] = B + 9
    ref, y_ref = U.f64(state), torch.zeros(B, D, dtype=torch.float64)
    for i, s in enumerate(slots.tolist()):
        if 0 <= s < B + 9:
            a, rest = torch.exp(U.f64(g[i])), -torch.expm1(U.f64(g[i]))
            ref[s] = y_ref[i] = a * ref[s] + (rest if complement else 1.0) * U.f64(x[i])
    y = linrec_step(x, g, state, slots, complement=complement)
    U.check(dict(y=y, state=state), dict(y=y_ref, state=ref))


def test_steps_continue_a_prefill():
    p, _ = problem(3, 40, 72, "bf16", "bf16", seed=11)
    h, ht = linrec_fwd(p["x"], p["g"], p["h0"], complement=True)
    _, state = linrec_fwd(p["x"][:, :30].contiguous(), p["g"][:, :30].contiguous(), p["h0"], complement=True)
    for t in range(30, 40):
        y = linrec_step(p["x"][:, t], p["g"][:, t], state, complement=True)
        assert U.rel(y, U.f64(h[:, t])) <= 2 * U.BAR[torch.bfloat16]
    assert U.rel(state, U.f64(ht)) <= U.FP32_BAR


def test_step_of_nothing():
    state = torch.ones(4, 16, device="cuda")
    x = torch.empty(0, 16, device="cuda")
    assert linrec_step(x, x, state).shape == (0, 16)
    x = torch.ones(2, 16, device="cuda")
    y = linrec_step(x, x, state, torch.tensor([-1, -1], dtype=torch.int32, device="cuda"))
    assert not y.any() and torch.equal(state, torch.ones_like(state))


# ---------------------------------------------------------------- many channels, many sequences, long rows
@pytest.mark.parametrize("T,D", [(3000, 1000), (700, 4100), (257, 10008), (5000, 520), (1025, 96)])
def test_blocks_of_channels(T, D):
    """Widths whose blocks of 32 channels fill several waves of clusters, or end inside a block."""
    p, d = problem(1, T, D, "bf16", "f32", seed=T)
    check(p, d, None, True)


@pytest.mark.parametrize("dtype,gtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f16", "f16")])
@pytest.mark.parametrize("T,D", [(3000, 100), (900, 1002), (700, 2049), (4000, 35), (129, 70)])
def test_rows_that_are_no_multiple_of_16_bytes(T, D, dtype, gtype):
    """Rows that start on words, and rows that do not, through many tiles and ends of sequences in them."""
    lens = [T // 3, 1, 0, T // 2 - 1, T - T // 3 - T // 2]
    p, d = problem(1, T, D, dtype, gtype, seed=T + D, lens=lens)
    check(p, d, lens, True)


@pytest.mark.parametrize("D", [64, 66])
def test_rows_that_start_beside_a_word(D):
    p, d = problem(1, 500, D, "bf16", "bf16", seed=D)
    want = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"])
    for name, where in (("x", p), ("g", p), ("dh", d)):
        wide = torch.zeros(1, 500, D + 2, dtype=torch.bfloat16, device="cuda")
        wide[..., 1:-1] = where[name]
        where[name] = wide[..., 1:-1]
    check(p, d, None, False)
    got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"])
    for key in want:
        assert torch.equal(want[key], got[key])


@pytest.mark.parametrize("dtype,T,D", [("bf16", 40, 35), ("bf16", 700, 66), ("f32", 40, 37), ("f16", 300, 35)])
def test_rows_whose_stride_is_wider_than_they_are(dtype, T, D):
    """The columns between the rows hold nans, of which nothing is read."""
    p, d = problem(1, T, D, dtype, dtype, seed=T + D)
    for name, where in (("x", p), ("g", p), ("dh", d)):
        wide = torch.full((T * 72,), float("nan"), dtype=TYPES[dtype], device="cuda")
        view = torch.as_strided(wide, (1, T, D), (T * 72, 72, 1))
        view.copy_(where[name])
        where[name] = view
    check(p, d, None, True)
    got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], complement=True)
    assert all(torch.isfinite(v.float()).all() for v in got.values())


def test_many_sequences():
    gen = torch.Generator().manual_seed(21)
    lens = torch.randint(0, 4, (2500,), generator=gen).tolist()
    p, d = problem(1, sum(lens), 40, "f32", "f32", seed=22, lens=lens)
    check(p, d, lens, False)


def test_rows_beyond_32_bits():
    """More than 2^31 elements: the last rows, whose sequence starts late, against the same sequence by itself."""
    T, D, tail = (1 << 20) + 5000, 2056, 700
    gen = torch.Generator("cuda").manual_seed(23)
    x = torch.randn(1, T, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    g = torch.full((1, T, D), -0.05, device="cuda", dtype=torch.bfloat16)
    g[:, -tail:] = -torch.rand(1, tail, D, generator=gen, device="cuda").bfloat16()
    cu = torch.tensor([0, T - tail, T], dtype=torch.int32, device="cuda")
    h, ht, states = linrec_fwd(x, g, None, cu, return_states=True, check_status=True)
    ref, ref_ht = linrec_fwd(x[:, -tail:].contiguous(), g[:, -tail:].contiguous())
    assert U.rel(h[:, -tail:], U.f64(ref)) <= 1e-3 and U.rel(ht[1:], U.f64(ref_ht)) <= U.FP32_BAR
    dh = x
    got = linrec_bwd(x, g, dh, None, None, cu, states)
    alone = linrec_bwd(x[:, -tail:].contiguous(), g[:, -tail:].contiguous(), dh[:, -tail:].contiguous())
    assert U.rel(got["dx"][:, -tail:], U.f64(alone["dx"])) <= 1e-3
    assert U.rel(got["dg"][:, -tail:], U.f64(alone["dg"])) <= 1e-3
    assert U.rel(got["dh0"][1:], U.f64(alone["dh0"])) <= U.FP32_BAR


def test_large_and_small_gates():
    """Decays that underflow, that are 1, and that grow."""
    g = torch.tensor([0.0, -1e-6, -87.0, -88.5, -200.0, float("-inf"), 0.5, 3.0, -0.35, -0.34], device="cuda")
    g = g.repeat(8, 4)[None].contiguous()
    x = U.randn(U.seeded(24), *g.shape)
    p = dict(x=x, g=g, h0=U.randn(U.seeded(25), 1, 40), cu_seqlens=None)
    check(p, dict(dh=U.randn(U.seeded(26), *g.shape), dht=U.randn(U.seeded(27), 1, 40)), None, True)


def test_waits_that_run_out_are_reported(monkeypatch):
    """With a limit of one poll real waits run out: the call reports it, ends in order, and the next call is right."""
    p, _ = problem(1, 6000, 256, "bf16", "f32", seed=28)
    ref = linrec_fwd(p["x"], p["g"], p["h0"])
    monkeypatch.setenv("GDR_SPIN_LIMIT", "1")
    statuses = []
    for _ in range(3):
        try:
            h, ht = linrec_fwd(p["x"], p["g"], p["h0"], check_status=True)
            statuses.append(_lib.GDR_OK)
        except GdrError as e:
            statuses.append(e.status)
    assert _lib.GDR_ERR_TIMEOUT in statuses and set(statuses) <= {_lib.GDR_OK, _lib.GDR_ERR_TIMEOUT}, statuses
    monkeypatch.delenv("GDR_SPIN_LIMIT")
    again = linrec_fwd(p["x"], p["g"], p["h0"], check_status=True)
    assert all(torch.equal(a, b) for a, b in zip(ref, again))


def test_capture_in_a_graph_and_other_streams():
    p, d = problem(1, 900, 96, "bf16", "bf16", seed=29, lens=[300, 600])
    ref = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"])
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))


def test_the_status_is_read_on_the_calls_own_stream():
    """Work on the default stream is not waited for, and nothing is left to be done to the workspace on return."""
    p, _ = problem(1, 500, 64, "bf16", "f32", seed=30)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ref = linrec_fwd(p["x"], p["g"], p["h0"], stream=side, check_status=True)  # (loads and allocates what the call needs)
    torch.cuda.synchronize()
    torch.cuda._sleep(1_000_000_000)
    busy = torch.cuda.Event()
    busy.record()
    out = linrec_fwd(p["x"], p["g"], p["h0"], stream=side, check_status=True)
    assert not busy.query()
    with torch.cuda.stream(side):
        again = torch.full((256,), 255, dtype=torch.uint8, device="cuda")  # the workspace's block, as a rule
    torch.cuda.synchronize()
    assert (again == 255).all() and all(torch.equal(a, b) for a, b in zip(ref, out))


@pytest.mark.parametrize("short", ["gdr_linrec_fwd", "gdr_linrec_bwd"])
def test_waits_that_run_out_in_either_pass_of_a_backward_are_reported(short, monkeypatch):
    """A backward without saved states runs the forward first; a limit of one poll for one of the two passes alone."""
    p, d = problem(1, 6000, 256, "bf16", "f32", seed=31)
    _, _, states = linrec_fwd(p["x"], p["g"], p["h0"], return_states=True)
    ref = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], states=states, check_status=True)
    queue = block._queue

    def limited(name, packed, index):
        with monkeypatch.context() as m:
            if name == short:
                m.setenv("GDR_SPIN_LIMIT", "1")
            queue(name, packed, index)

    with monkeypatch.context() as m:
        m.setattr(block, "_queue", limited)
        for kept in (None, states):
            statuses = []
            for _ in range(3):
                try:
                    linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], states=kept, check_status=True)
                    statuses.append(_lib.GDR_OK)
                except GdrError as e:
                    statuses.append(e.status)
            expected = short == "gdr_linrec_bwd" or kept is None
            assert (_lib.GDR_ERR_TIMEOUT in statuses) == expected, statuses
            assert set(statuses) <= {_lib.GDR_OK, _lib.GDR_ERR_TIMEOUT}, statuses
    again = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], check_status=True)
    assert all(torch.equal(ref[k], again[k]) for k in ref)


def test_malformed_lists_of_many_sequences_are_reported():
    """More sequences than one CTA checks; no lengths but the list is out of order, or ends early."""
    lens = [3] * 2000
    p, d = problem(1, 6000, 40, "f32", "f32", seed=32, lens=lens)
    _, _, states = linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"], return_states=True, check_status=True)
    for at, value in ((1999, 5000), (700, 6001), (0, 1), (2000, 5999)):
        bad = p["cu_seqlens"].clone()
        bad[at] = value
        for call in (lambda: linrec_fwd(p["x"], p["g"], p["h0"], bad, check_status=True),
                     lambda: linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], bad, states, check_status=True),
                     lambda: linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], bad, check_status=True)):
            with pytest.raises(GdrError) as e:
                call()
            assert e.value.status == _lib.GDR_ERR_DEVICE
    linrec_fwd(p["x"], p["g"], p["h0"], p["cu_seqlens"], check_status=True)


@pytest.mark.parametrize("lo,hi", [(-1, 0), (-10, -1), (-40, -10), (-87, -40), (0, 1), (1, 10), (10, 88)])
def test_decays_by_themselves(lo, hi):
    """exp(g) and 1 - exp(g) as a step on a state of 1 and on an input of 1 shows them.

    In units of 2^-24 of a: its own rounding 1, those before it 0.25 each for p, r and 1 + p's share, the polynomial 0.2: below
    2; and n times the constant's 1.9e-9, which is 0.033 for each n = g / ln 2.  Near 1 both signs are as frequent: the
    mean of a million is below 0.1.  1 - a for decays: its rounding 1 and what a has, times a / (1 - a) <= 2.4 outside the
    polynomial's own range: below 4 plus the same n, of which a / (1 - a) leaves less than half a unit."""
    g = (torch.rand(1024, 1024, generator=U.seeded(33), dtype=torch.float64) * (hi - lo) + lo).float().cuda()
    state = torch.ones_like(g)
    linrec_step(torch.zeros_like(g), g, state)
    a = torch.exp(g.double())
    off = (state.double() - a) / a * 2.0 ** 24
    assert float(off.abs().max()) <= 2.0 + 0.033 * max(abs(lo), abs(hi)) / 0.693
    if abs(lo) <= 1 and abs(hi) <= 1:
        assert abs(float(off.mean())) <= 0.1
    if hi <= 0:
        rest = torch.zeros_like(g)
        linrec_step(torch.ones_like(g), g, rest, complement=True)
        want = -torch.expm1(g.double())
        seen = want > 0  # (a gate of exactly 0 leaves nothing)
        assert float(((rest.double() - want)[seen] / want[seen]).abs().max()) <= 4.5 * 2.0 ** -24
