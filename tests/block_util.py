"""Plain 64-bit forms of the operators around the delta rule, on the CPU, and the bars of their tests.

Bars, relative L2 for each output.  A result of a 16-bit type carries its own rounding, at most half a unit in the last
place of each value (bf16, 8 significant bits: 2^-8; fp16, 11 of them: 2^-11), and the fp32 arithmetic before it.  That arithmetic sums a row in a tree with
at most some 50 roundings on a path (50 x 2^-24 = 3e-6); a column sum's roundings are independent and add up as their
square root (100 on a path: 6e-7); a recurrence adds one rounding of the decay and one of the state at each of the tokens
that it remembers, up to 1000 here (sqrt(2000) x 2^-24 = 3e-6).  1e-5 covers each with a factor of three and more.
A value below fp16's smallest normal number is rounded to a multiple of 2^-24: off by up to 2^-25 whatever its size."""
import numpy as np
import torch

FP32_BAR = 1e-5
BAR = {torch.float32: FP32_BAR, torch.bfloat16: 2.0 ** -8 + FP32_BAR, torch.float16: 2.0 ** -11 + FP32_BAR}


def f64(t):
    return None if t is None else t.detach().double().cpu()


def rel(got, ref):
    got_type, got, ref = got.dtype, f64(got).numpy(), ref.numpy()
    assert got.shape == ref.shape, (got.shape, ref.shape)
    assert np.array_equal(np.isfinite(got), np.isfinite(ref))
    ok = np.isfinite(ref)
    norm = np.linalg.norm(ref[ok])
    diff = np.linalg.norm(got[ok] - ref[ok])
    if got_type == torch.float16 and diff <= 2.0 ** -25 * np.sqrt(ok.sum()):
        return 0.0
    return diff / norm if norm > 0 else diff


def check(got, ref):
    """Every named output within its type's bar."""
    bad = {}
    for name, r in ref.items():
        if r is None:
            assert got[name] is None, name
            continue
        e = rel(got[name], r)
        if not e <= BAR[got[name].dtype]:
            bad[name] = e
    assert not bad, bad


def gated_norm(x, z, w, eps, act, dy=None):
    x, z, w, dy = f64(x), f64(z), f64(w), f64(dy)
    rs = (x.square().mean(-1, keepdim=True) + eps) ** -0.5
    sg = None if z is None else 1.0 / (1.0 + torch.exp(-z))
    a = 1.0 if z is None else (z * sg if act == "silu" else sg)
    wv = 1.0 if w is None else w
    out = dict(y=wv * x * rs * a)
    if dy is not None:
        t = dy * a * wv
        out["dx"] = rs * t - x * rs ** 3 * (t * x).mean(-1, keepdim=True)
        out["dz"] = None if z is None else dy * wv * x * rs * (sg * (1 + z * (1 - sg)) if act == "silu" else sg * (1 - sg))
        out["dweight"] = None if w is None else (dy * a * x * rs).reshape(-1, x.shape[-1]).sum(0)
    return out


def add_norm_fwd(x, res, w, scale, eps):
    x, res, w = f64(x), f64(res), f64(w)
    s = f64(scale) if isinstance(scale, torch.Tensor) else scale
    r = s * x + (0.0 if res is None else res)
    rs = (r.square().mean(-1, keepdim=True) + eps) ** -0.5
    return dict(y=r * rs * (1.0 if w is None else w), r=r)


def add_norm_bwd(dy, dres, r, w, scale, x, eps):
    dy, dres, r, w, x = f64(dy), f64(dres), f64(r), f64(w), f64(x)
    s = f64(scale) if isinstance(scale, torch.Tensor) else scale
    rs = (r.square().mean(-1, keepdim=True) + eps) ** -0.5
    t = dy if w is None else dy * w
    dr = rs * t - r * rs ** 3 * (t * r).mean(-1, keepdim=True) + (0.0 if dres is None else dres)
    flat = (-1, r.shape[-1])
    return dict(dresidual=dr, dx=s * dr, dweight=None if w is None else (dy * r * rs).reshape(flat).sum(0),
                dscale=None if x is None else (dr * x).reshape(flat).sum(0))


def spans(B, T, lens):
    """(batch row, first token, end, sequence) of every sequence."""
    if lens is None:
        return [(b, 0, T, b) for b in range(B)]
    out, at = [], 0
    for i, n in enumerate(lens):
        out.append((0, at, at + n, i))
        at += n
    return out


def linrec(x, g, h0, lens, complement, dh=None, dht=None):
    """The recurrence token by token, and the adjoint token by token."""
    x, g, h0, dh, dht = f64(x), f64(g), f64(h0), f64(dh), f64(dht)
    B, T, D = x.shape
    seqs = spans(B, T, lens)
    a, rest = torch.exp(g), -torch.expm1(g)
    b = rest * x if complement else x
    h, ht = torch.zeros_like(x), torch.zeros(len(seqs), D, dtype=torch.float64)
    out = dict(h=h, ht=ht)
    if dh is not None:
        dx, dg, dh0 = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(ht)
        out.update(dx=dx, dg=dg, dh0=dh0)
    for row, lo, hi, s in seqs:
        now = torch.zeros(D, dtype=torch.float64) if h0 is None else h0[s].clone()
        first = now.clone()
        for t in range(lo, hi):
            now = a[row, t] * now + b[row, t]
            h[row, t] = now
        ht[s] = now
        if dh is None:
            continue
        mu = torch.zeros(D, dtype=torch.float64) if dht is None else dht[s].clone()
        for t in range(hi - 1, lo - 1, -1):
            lam = dh[row, t] + mu
            mu = a[row, t] * lam
            before = h[row, t - 1] if t > lo else first
            dx[row, t] = rest[row, t] * lam if complement else lam
            dg[row, t] = mu * (before - x[row, t] if complement else before)
        dh0[s] = mu
    return out


def seeded(seed):
    return torch.Generator().manual_seed(seed)


def randn(gen, *shape, dtype=torch.float32, times=1.0, device="cuda"):
    return (torch.randn(*shape, generator=gen) * times).to(dtype).to(device)


def gates(gen, *shape, dtype=torch.float32, device="cuda"):
    """Log-gates whose channels forget in a few tokens to about a thousand."""
    rate = torch.exp(torch.rand(shape[-1], generator=gen) * 6.2 - 6.9)
    return (-2.0 * rate * torch.sigmoid(torch.randn(*shape, generator=gen))).to(dtype).to(device)
