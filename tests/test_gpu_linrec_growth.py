"""The recurrence where gates are above 0 and states grow: products of such decays over some rows pass what fp32 holds, while
the states themselves do not.

Bars, relative, row by row: each token adds at most 6 units of 2^-24 to a state (the decay's, one rounding of the
sum), and these states remember every token, so 8 T 2^-24 bounds T tokens; a gradient has two such factors and the
difference of two values, 3 times that.  bf16 results carry their own rounding, 2^-8."""
import math

import pytest
import torch

import block_util as U
from chunked_gated_delta_09_gb300 import linrec_bwd, linrec_fwd, linrec_step

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}
UP = 120.0   # what the gates of a rise add up to: e^120 = 2^173; states go from about e^-60 to e^60 and back


def rise_and_fall(rows, down, periods, D, dtype, gtype, seed):
    """Gates of `periods` rises in `rows` tokens, each taken back in `down`, and values of the states' size."""
    gen = U.seeded(seed)

    def steps(n):
        w = 0.8 + 0.4 * torch.rand(periods, n, D, generator=gen)
        return w * (UP / w.sum(1, keepdim=True))

    g = torch.cat([steps(rows), -steps(down)], 1).to(gtype).reshape(1, -1, D)
    log = torch.cumsum(g.double(), 1)  # of a state that starts at 1
    T = g.shape[1]
    low = torch.minimum(log, torch.cat([torch.zeros(1, 1, D, dtype=torch.float64), log[:, :-1]], 1))
    half = math.exp(-UP / 2)
    x = 0.1 * torch.randn(1, T, D, generator=gen).double() * torch.exp(low) * half
    dh = 0.1 * torch.randn(1, T, D, generator=gen).double() * torch.exp(-log) / half
    h0, dht = torch.randn(1, D, generator=gen) * half, torch.randn(1, D, generator=gen) / half
    return dict(x=x.to(dtype).cuda(), g=g.cuda(), h0=h0.cuda()), dict(dh=dh.to(dtype).cuda(), dht=dht.cuda())


def close(got, ref, bar):
    if got.dtype == torch.bfloat16:
        bar += 2.0 ** -8
    got, ref = U.f64(got), ref.reshape(got.shape)
    assert torch.isfinite(got).all()
    off = (got - ref).norm(dim=-1) / ref.norm(dim=-1)
    assert float(off.max()) <= bar, (float(off.max()), int(off.argmax()), bar)


@pytest.mark.parametrize("complement", [False, True], ids=["plain", "complement"])
@pytest.mark.parametrize("dtype,gtype", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
@pytest.mark.parametrize("rows,down,periods,D", [(2, 700, 2, 40), (7, 700, 2, 40), (7, 700, 1, 35), (70, 700, 2, 40),
                                                 (140, 700, 1, 64), (140, 700, 2, 33), (140, 700, 5, 64), (600, 700, 3, 96),
                                                 (2, 2, 60, 40), (7, 7, 40, 40), (7, 7, 20, 35), (70, 70, 4, 40),
                                                 (140, 140, 2, 64), (140, 140, 2, 33), (140, 140, 10, 64), (600, 600, 4, 96),
                                                 (500, 3, 6, 40)])
def test_states_that_rise_and_fall(rows, down, periods, D, dtype, gtype, complement):
    p, d = rise_and_fall(rows, down, periods, D, TYPES[dtype], TYPES[gtype], seed=rows + D)
    bar = 8 * p["x"].shape[1] * 2.0 ** -24
    h, ht, states = linrec_fwd(p["x"], p["g"], p["h0"], complement=complement, return_states=True, check_status=True)
    got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], states=states, complement=complement, check_status=True)
    ref = U.linrec(p["x"], p["g"], p["h0"], None, complement, d["dh"], d["dht"])
    close(h, ref["h"], bar)
    close(ht, ref["ht"], bar)
    for name in ("dx", "dg", "dh0"):
        close(got[name], ref[name], 3 * bar)


@pytest.mark.parametrize("D", [40, 35])
@pytest.mark.parametrize("gate", [0.01, 0.7, 2.0, 88.0, float("inf")])
def test_zeros_do_not_grow(gate, D):
    """States, inputs and gradients of zero stay zero, whatever multiplies them; in packed sequences too."""
    lens = [300, 0, 1, 699]
    cu = torch.tensor([0, 300, 300, 301, 1000], dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.float16):
        x = torch.zeros(1, 1000, D, dtype=dtype, device="cuda")
        g = torch.full((1, 1000, D), gate, device="cuda")
        for list_, n in ((None, 1), (cu, len(lens))):
            zero = torch.zeros(n, D, device="cuda")
            h, ht, states = linrec_fwd(x, g, zero, list_, return_states=True)
            got = linrec_bwd(x, g, x, zero, zero, list_, states)
            for t in (h, ht, *got.values()):
                assert not t.any()


def test_sequences_that_grow_end_inside_a_tile():
    """Rises and falls in packed sequences: what one sequence's growth makes of its maps does not reach the next one."""
    lens, parts = [], []
    for i, rows in enumerate((9, 50, 70, 3, 150)):
        parts.append(rise_and_fall(rows, 20 + rows, 1, 40, torch.float32, torch.float32, seed=50 + i))
        lens.append(20 + 2 * rows)
    p = {k: torch.cat([a[k] for a, _ in parts], 0 if k == "h0" else 1) for k in ("x", "g", "h0")}
    d = {k: torch.cat([b[k] for _, b in parts], 0 if k == "dht" else 1) for k in ("dh", "dht")}
    cu = torch.tensor([sum(lens[:i]) for i in range(6)], dtype=torch.int32, device="cuda")
    bar = 8 * max(lens) * 2.0 ** -24
    h, ht, states = linrec_fwd(p["x"], p["g"], p["h0"], cu, return_states=True, check_status=True)
    got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], cu, states, check_status=True)
    ref = U.linrec(p["x"], p["g"], p["h0"], lens, False, d["dh"], d["dht"])
    close(h, ref["h"], bar)
    close(ht, ref["ht"], bar)
    for name in ("dx", "dg", "dh0"):
        close(got[name], ref[name], 3 * bar)


def test_channels_that_do_not_grow_keep_their_bits():
    gen = U.seeded(60)
    x, dh, g = U.randn(gen, 1, 900, 64), U.randn(gen, 1, 900, 64), U.gates(gen, 1, 900, 64)
    h, ht, states = linrec_fwd(x, g, return_states=True)
    ref = linrec_bwd(x, g, dh, states=states)
    grown = g.clone()
    grown[..., ::2] = 3.0
    h2, ht2, states = linrec_fwd(x, grown, return_states=True)
    got = linrec_bwd(x, grown, dh, states=states)
    assert torch.equal(h[..., 1::2], h2[..., 1::2]) and torch.equal(ht[..., 1::2], ht2[..., 1::2])
    for name in ref:
        assert torch.equal(ref[name][..., 1::2], got[name][..., 1::2]), name


def test_steps_give_what_the_whole_gives():
    p, _ = rise_and_fall(70, 70, 1, 40, torch.float32, torch.float32, seed=61)
    h, _ = linrec_fwd(p["x"], p["g"], p["h0"])
    state = p["h0"].clone()
    for t in range(140):
        y = linrec_step(p["x"][:, t], p["g"][:, t], state)
        close(h[:, t], U.f64(y), 2 * 8 * 140 * 2.0 ** -24)


@pytest.mark.parametrize("rows", [2, 3, 40, 150, 600])
def test_what_decays_leave_below_the_smallest_number(rows):
    """A state of 1e28 alone (no input) that falls by e^-130: what the decays of a tile leave of it below 2^-126 may count as
    zero, anything above is right to its own rounding."""
    g = torch.full((1, rows, 40), -130.0 / rows, device="cuda")
    h0 = 1e28 * (1.0 + torch.rand(1, 40, generator=U.seeded(62))).cuda()
    h, _ = linrec_fwd(torch.zeros_like(g), g, h0, check_status=True)
    ref = U.linrec(torch.zeros_like(g), g, h0, None, False)["h"]
    assert ((U.f64(h) - ref).abs() <= 8 * rows * 2.0 ** -24 * ref + 2.0 ** -126 * U.f64(h0)[:, None]).all()


@pytest.mark.parametrize("D", [64, 33])
def test_an_infinite_state_stays_infinite(D):
    """An infinity goes through decays whose products underflow, and leaves the channels beside it as they were; a decay of 0
    makes it a nan, as the formula does."""
    gen = U.seeded(63)
    x, dh, g = U.randn(gen, 1, 1500, D), U.randn(gen, 1, 1500, D), -torch.ones(1, 1500, D, device="cuda")
    h, _, states = linrec_fwd(x, g, return_states=True)
    ref = linrec_bwd(x, g, dh, states=states)
    bad = x.clone()
    bad[0, 100, 5], bad[0, 7, 6] = float("inf"), float("-inf")
    g[0, 900, 6] = float("-inf")
    got, ht = linrec_fwd(bad, g)
    assert (got[0, 100:, 5] == float("inf")).all() and ht[0, 5] == float("inf")
    assert (got[0, 7:900, 6] == float("-inf")).all() and torch.isnan(got[0, 900:, 6]).all() and torch.isnan(ht[0, 6])
    others = [c for c in range(D) if c not in (5, 6)]
    assert torch.equal(got[..., others], h[..., others])
    g[0, 900, 6] = -1.0
    dh[0, 1400, 9] = float("inf")
    back = linrec_bwd(x, g, dh, states=states)
    assert (back["dx"][0, :1401, 9] == float("inf")).all()
    others = [c for c in range(D) if c != 9]
    assert all(torch.equal(back[k][..., others], ref[k][..., others]) for k in ref)


@pytest.mark.parametrize("B,rows,down,D", [(3, 2, 3, 40), (5, 2, 2, 33), (2, 70, 90, 64), (4, 150, 700, 40)])
@pytest.mark.parametrize("complement", [False, True], ids=["plain", "complement"])
def test_batches_and_rows_at_a_distance(B, rows, down, D, complement):
    """Sequences side by side, shorter than a range of rows or longer, x, g and dh as columns of wider rows."""
    parts = [rise_and_fall(rows, down, 1, D, torch.float32, torch.float32, seed=80 + b) for b in range(B)]
    p = {k: torch.cat([a[k] for a, _ in parts]) for k in ("x", "g", "h0")}
    d = {k: torch.cat([b[k] for _, b in parts]) for k in ("dh", "dht")}
    for name, where in (("x", p), ("g", p), ("dh", d)):
        wide = torch.full((*where[name].shape[:2], D + 5), float("nan"), device="cuda")
        wide[..., 2:2 + D] = where[name]
        where[name] = wide[..., 2:2 + D]
    bar = 8 * p["x"].shape[1] * 2.0 ** -24
    h, ht, states = linrec_fwd(p["x"], p["g"], p["h0"], complement=complement, return_states=True, check_status=True)
    got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], states=states, complement=complement, check_status=True)
    ref = U.linrec(p["x"], p["g"], p["h0"], None, complement, d["dh"], d["dht"])
    close(h, ref["h"], bar)
    close(ht, ref["ht"], bar)
    for name in ("dx", "dg", "dh0"):
        close(got[name], ref[name], 3 * bar)


def test_results_repeat_bit_for_bit():
    p, d = rise_and_fall(140, 140, 6, 96, torch.bfloat16, torch.float32, seed=90)
    first = None
    for _ in range(5):
        h, ht, states = linrec_fwd(p["x"], p["g"], p["h0"], return_states=True)
        got = linrec_bwd(p["x"], p["g"], d["dh"], p["h0"], d["dht"], None, states)
        now = [h, ht, states, *got.values()]
        first = first or now
        assert all(torch.equal(a, b) for a, b in zip(first, now))


def test_states_beside_the_largest_number():
    """States (forward) and their gradients (backward) of up to 3e38 that the decays of a range take down a little."""
    D, up, down = 40, 176, 500
    g = torch.cat([torch.full((up, D), 0.5), torch.full((down, D), -0.01)])[None].cuda()
    h0 = (1.6 + 0.4 * torch.rand(1, D, generator=U.seeded(91))).cuda()
    zero = torch.zeros_like(g)
    bar = 8 * (up + down) * 2.0 ** -24
    h, ht, states = linrec_fwd(zero, g, h0, return_states=True)
    ref = U.linrec(zero, g, h0, None, False)
    assert 2.5e38 < float(ref["h"].max()) < 3.4e38
    close(h, ref["h"], bar)
    close(ht, ref["ht"], bar)
    back = g.flip(1).contiguous()
    got = linrec_bwd(zero, back, zero, None, h0)
    ref = U.linrec(zero, back, None, None, False, zero, h0)
    close(got["dx"], ref["dx"], bar)
    close(got["dh0"], ref["dh0"], bar)
