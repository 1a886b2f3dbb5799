"""Cases of the operators around the delta rule: the norms before and after a block, the gated linear recurrence and the
gradient clip.  ``run`` computes them as elementary torch operations in 32 bits, or, with ``own`` set, through this
package's calls; ``exact`` computes them in 64 bits from their definitions.

    gated norm   y = w x / rms(x) act(z) over each head          (after the block's rule, before its projection)
    add norm     r' = r + s x,  y = w r' / rms(r')               (the residual stream, before the next block)
    recurrence   h_t = a_t h_{t-1} + b_t, a = exp(g), b = x or (1 - a) x, per channel, sequences packed or dense
    clip         out_i = grad_i min(1, max_norm / (|grads| + eps)) over all gradients of a model

A "train" case is the forward call and then the backward call, as a training step makes them.
"""
import math

import torch

own = False

EPS = 1e-6
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


# ---------------------------------------------------------------- cases
def listed():
    return [
        # one decoding step of 8 sequences through the norm after a 16-head block: latency
        dict(name="gate_decode_8", op="gate", tokens=8, heads=16, dim=128, dtype="bf16", wtype="f32", act="silu",
             fused=False, train=False),
        # training at the 32-head per-channel workload's sizes, sigmoid gate
        dict(name="gate_train_2k_f16", op="gate", tokens=2048, heads=32, dim=128, dtype="f16", wtype="f16", act="sigmoid",
             fused=False, train=True),
        # training at the longest workload's sizes; z is a slice of a fused projection's rows
        dict(name="gate_train_32k_bf16", op="gate", tokens=32768, heads=16, dim=128, dtype="bf16", wtype="f32", act="silu",
             fused=True, train=True),
        # one token of one sequence into the residual stream: latency
        dict(name="add_norm_decode_1", op="addnorm", tokens=1, dim=2048, dtype="bf16", rtype="bf16", wtype="bf16",
             scale="one", train=False),
        # training: residual stream in fp32 and a learnt residual scale for each channel
        dict(name="add_norm_train_32k", op="addnorm", tokens=32768, dim=2048, dtype="bf16", rtype="f32", wtype="f32",
             scale="channel", train=True),
        # prefill of packed sequences of an odd total length, residual stream in bf16, one fixed residual scale
        dict(name="add_norm_prefill_48k", op="addnorm", tokens=48763, dim=4096, dtype="bf16", rtype="bf16", wtype="bf16",
             scale="number", train=False),
        # one decoding step of 64 sequences of a cache of 96 states: latency
        dict(name="linrec_step_64", op="step", batch=64, slots=96, dim=2048, dtype="bf16", gtype="f32", complement=True),
        # the tiny fp32 workload's sizes: 2 sequences of 128 tokens, 64 channels
        dict(name="linrec_train_tiny", op="linrec", batch=2, tokens=128, dim=64, packed=False, dtype="f32", gtype="f32",
             complement=True, train=True),
        # prefill of 8 packed ragged sequences, gates in bf16
        dict(name="linrec_prefill_48k", op="linrec", batch=8, tokens=48763, dim=4096, packed=True, dtype="bf16",
             gtype="bf16", complement=True, train=False),
        # training on one long sequence, gates in fp32
        dict(name="linrec_train_32k", op="linrec", batch=1, tokens=32768, dim=2048, packed=False, dtype="bf16", gtype="f32",
             complement=False, train=True),
        # the gradients of two tiny blocks: latency
        dict(name="clip_tiny_f32", op="clip", layers=2, dim=64, vocab=200, dtype="f32", otype="f32", clipped=True),
        # the bf16 gradients of six blocks and an embedding, clipped into the optimizer's fp32 gradients
        dict(name="clip_model_bf16", op="clip", layers=6, dim=2048, vocab=32000, dtype="bf16", otype="f32", clipped=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5))))))


def draw(rng):
    op = rng.choice(["gate", "gate", "addnorm", "addnorm", "step", "linrec", "linrec", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    most = 1 << 26 if dtype != "f32" else 1 << 25  # values of one input
    if op == "gate":
        dim = rng.choice([_log_int(rng, 8, 512), 8 * _log_int(rng, 2, 64), 64, 128])
        heads = _log_int(rng, 1, 48)
        return dict(op=op, tokens=_log_int(rng, 1, most // (dim * heads)), heads=heads, dim=dim, dtype=dtype,
                    wtype=rng.choice(["f32", dtype]), act=rng.choice(["silu", "sigmoid"]), fused=rng.random() < 0.4,
                    train=rng.random() < 0.6)
    if op == "addnorm":
        dim = rng.choice([_log_int(rng, 32, 8192), 8 * _log_int(rng, 8, 1024), 1 << rng.randint(6, 13)])
        return dict(op=op, tokens=_log_int(rng, 1, most // dim), dim=dim, dtype=dtype, rtype=rng.choice(["f32", dtype]),
                    wtype=rng.choice(["f32", dtype]), scale=rng.choice(["one", "number", "channel"]), train=rng.random() < 0.6)
    if op == "step":
        batch = _log_int(rng, 1, 2048)
        return dict(op=op, batch=batch, slots=batch + _log_int(rng, 1, 64), dim=rng.choice([_log_int(rng, 32, 8192), 2048]),
                    dtype=dtype, gtype=rng.choice(["f32", dtype]), complement=rng.random() < 0.5)
    if op == "linrec":
        dim = rng.choice([_log_int(rng, 16, 4096), 4 * _log_int(rng, 8, 1024), 1 << rng.randint(5, 12)])
        packed = rng.random() < 0.5
        batch = _log_int(rng, 1, 64)
        tokens = _log_int(rng, 1, min(65536, most // dim))
        return dict(op=op, batch=batch, tokens=tokens if packed else max(1, tokens // batch), dim=dim, packed=packed,
                    dtype=dtype, gtype=rng.choice(["f32", dtype]), complement=rng.random() < 0.5, train=rng.random() < 0.6)
    return dict(op=op, layers=rng.randint(1, 6), dim=_log_int(rng, 32, 1536), vocab=_log_int(rng, 100, 32000), dtype=dtype,
                otype=rng.choice(["f32", dtype]), clipped=rng.random() < 0.7)


def _clip_shapes(case):
    """Projections of a block (q, k, v, gate, out, two of its MLP) and its two norms, layer by layer, then the embedding
    and the last norm."""
    d = case["dim"]
    block = [(d, d)] * 5 + [(4 * d, d), (d, 4 * d)] + [(d,)] * 2
    return block * case["layers"] + [(case["vocab"], d), (d,)]


# ---------------------------------------------------------------- inputs
def _lengths(total, n, seed):
    """n sequence lengths that add up to total, some of them far longer than others, some possibly empty."""
    r = torch.rand(n, generator=torch.Generator().manual_seed(seed), dtype=torch.float64).square()
    cuts = [round(float(v)) for v in torch.cumsum(r, 0) / r.sum() * total]
    cuts[-1] = total
    return [b - a for a, b in zip([0] + cuts[:-1], cuts)]


def _gates(shape, dim, gen):
    """Log-gates: each channel has its own rate of forgetting, from a few tokens to about a thousand, moved by the input."""
    rate = torch.exp(torch.rand(dim, generator=gen, device="cuda") * math.log(500.0) + math.log(1e-3))
    return -rate * 2.0 * torch.sigmoid(torch.randn(*shape, generator=gen, device="cuda"))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.float32, times=1.0):
        return (torch.randn(*shape, generator=gen, device="cuda") * times).to(dtype)

    dt = DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "gate":
        n, h, d = case["tokens"], case["heads"], case["dim"]
        s["x"] = randn(1, n, h, d, dtype=dt)
        if case["fused"]:  # the gate's columns among those of the projection that makes it
            s["z"] = randn(1, n, 2, h, d, dtype=dt)[:, :, 1]
        else:
            s["z"] = randn(1, n, h, d, dtype=dt)
        s["w"] = (1.0 + randn(d, times=0.1)).to(DTYPES[case["wtype"]])
        s["dy"] = randn(1, n, h, d, dtype=dt) if case["train"] else None
    elif case["op"] == "addnorm":
        n, d = case["tokens"], case["dim"]
        rt = DTYPES[case["rtype"]]
        s["x"], s["r"] = randn(1, n, d, dtype=dt), randn(1, n, d, dtype=rt, times=2.0)
        s["w"] = (1.0 + randn(d, times=0.1)).to(DTYPES[case["wtype"]])
        s["scale"] = {"one": 1.0, "number": 0.5}.get(case["scale"])
        if s["scale"] is None:
            s["scale"] = (0.5 + randn(d, times=0.1)).to(DTYPES[case["wtype"]])
        s["dy"] = randn(1, n, d, dtype=dt) if case["train"] else None
        s["dr"] = randn(1, n, d, dtype=rt) if case["train"] else None
    elif case["op"] == "step":
        b, d = case["batch"], case["dim"]
        s["x"], s["g"] = randn(b, d, dtype=dt), _gates((b, d), d, gen).to(DTYPES[case["gtype"]])
        s["h"] = randn(case["slots"], d)
        s["slots"] = torch.randperm(case["slots"], generator=gen, device="cuda")[:b].to(torch.int32)
    elif case["op"] == "linrec":
        d = case["dim"]
        if case["packed"]:
            lens, lead = _lengths(case["tokens"], case["batch"], seed), (1, case["tokens"])
            cu = [0]
            for v in lens:
                cu.append(cu[-1] + v)
            s["cu"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
        else:
            lens, lead = [case["tokens"]] * case["batch"], (case["batch"], case["tokens"])
            s["cu"] = None
        s["lens"], n = lens, torch.tensor(lens)
        s["full"] = torch.nonzero(n).flatten()  # the sequences that have a token, and their first and last ones
        s["last"] = (torch.cumsum(n, 0)[s["full"]] - 1).cuda()
        s["full"] = s["full"].cuda()
        s["first"] = s["last"] + 1 - n.cuda()[s["full"]]
        s["x"] = randn(*lead, d, dtype=dt)
        s["g"] = _gates((*lead, d), d, gen).to(DTYPES[case["gtype"]])
        s["h0"] = randn(case["batch"], d, times=0.1)
        s["dh"] = randn(*lead, d, dtype=dt) if case["train"] else None
        s["dht"] = randn(case["batch"], d, times=0.1) if case["train"] else None
    else:
        s["grads"] = [randn(*shape, dtype=dt, times=0.01) for shape in _clip_shapes(case)]
        s["out"] = [torch.empty_like(t, dtype=DTYPES[case["otype"]]) for t in s["grads"]]
        norm = 0.01 * math.sqrt(sum(t.numel() for t in s["grads"]))
        s["max_norm"] = norm * (0.3 if case["clipped"] else 3.0)
    return s


# ---------------------------------------------------------------- plain forms, 32 bits
def _gate_values(z, act):
    s = torch.sigmoid(z)
    return (z * s, s * (1.0 + z * (1.0 - s))) if act == "silu" else (s, s * (1.0 - s))


def _plain_gate(s):
    c = s["case"]
    x, z, w = s["x"].float(), s["z"].float(), s["w"].float()
    rs = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    a, da = _gate_values(z, c["act"])
    out = dict(y=(x * rs * w * a).to(s["x"].dtype))
    if c["train"]:
        dy = s["dy"].float()
        xhat, dn = x * rs, dy * a
        t = dn * w
        out["dx"] = (rs * (t - xhat * (t * xhat).mean(-1, keepdim=True))).to(s["x"].dtype)
        out["dz"] = (dy * xhat * w * da).to(s["x"].dtype)
        out["dw"] = (dn * xhat).sum((0, 1, 2)).to(s["w"].dtype)
    return out


def _plain_addnorm(s):
    c = s["case"]
    channel = c["scale"] == "channel"
    x, w = s["x"].float(), s["w"].float()
    scale = s["scale"].float() if channel else s["scale"]
    r = s["r"].float() + scale * x
    rs = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    out = dict(y=(r * rs * w).to(s["x"].dtype), r=r.to(s["r"].dtype))
    if c["train"]:
        dy, r = s["dy"].float(), out["r"].float()  # the backward call is given the stream as it was stored
        rs = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
        t, xhat = dy * w, r * rs
        dr = rs * (t - xhat * (t * xhat).mean(-1, keepdim=True)) + s["dr"].float()
        out["dr"], out["dx"] = dr.to(s["r"].dtype), (scale * dr).to(s["x"].dtype)
        out["dw"] = (dy * xhat).sum((0, 1)).to(s["w"].dtype)
        if channel:
            out["dscale"] = (dr * x).sum((0, 1)).to(s["scale"].dtype)
    return out


def _decay(g):
    """exp(g) and 1 - exp(g).  Near 1 exp(g) is formed from expm1: a rounding that leans to one side, repeated for each
    of the hundreds of tokens that such a channel remembers, would add up."""
    e = torch.expm1(g)
    return torch.where(g > -0.5, 1.0 + e, torch.exp(g)), -e


def _plain_step(s):
    at = s["slots"].long()
    a, rest = _decay(s["g"].float())
    x = s["x"].float()
    h = a * s["h"][at] + (rest * x if s["case"]["complement"] else x)
    s["h"][at] = h
    return dict(y=h.to(s["x"].dtype), h=s["h"])


def _scan(a, b, longest):
    """h_t = a_t h_{t-1} + b_t over the rows, by doubling the distance that each row looks back."""
    k = 1
    while k < longest:
        b = torch.cat([b[:k], b[k:] + a[k:] * b[:-k]])
        a = torch.cat([a[:k], a[k:] * a[:-k]])
        k *= 2
    return b


def _plain_linrec(s):
    c = s["case"]
    n, d = sum(s["lens"]), c["dim"]
    first, full, last = s["first"], s["full"], s["last"]
    x, g = s["x"].reshape(n, d).float(), s["g"].reshape(n, d).float()
    a, rest = _decay(g)
    b = rest * x if c["complement"] else x
    a_in, b_in = a.clone(), b.clone()
    b_in[first] += a[first] * s["h0"][full]
    a_in[first] = 0.0
    h = _scan(a_in, b_in, max(s["lens"]))
    ht = s["h0"].clone()
    ht[full] = h[last]
    out = dict(h=h.reshape(s["x"].shape).to(s["x"].dtype), ht=ht)
    if c["train"]:
        before = torch.cat([h[:1], h[:-1]])
        before[first] = s["h0"][full]
        a_next = torch.cat([a[1:], a[:1]])
        a_next[last] = 0.0
        dh = s["dh"].reshape(n, d).float().clone()
        dh[last] += s["dht"][full]
        lam = _scan(a_next.flip(0), dh.flip(0), max(s["lens"])).flip(0)
        dg = a * before * lam - (a * x * lam if c["complement"] else 0.0)
        out["dx"] = (rest * lam if c["complement"] else lam).reshape(s["x"].shape).to(s["x"].dtype)
        out["dg"] = dg.reshape(s["g"].shape).to(s["g"].dtype)
        dh0 = s["dht"].clone()
        dh0[full] = a[first] * lam[first]
        out["dh0"] = dh0
    return out


def _plain_clip(s):
    norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
    factor = torch.clamp(s["max_norm"] / (norm + EPS), max=1.0)
    return dict(norm=norm, out=[(t.float() * factor).to(o.dtype) for t, o in zip(s["grads"], s["out"])])


PLAIN = dict(gate=_plain_gate, addnorm=_plain_addnorm, step=_plain_step, linrec=_plain_linrec, clip=_plain_clip)


# ---------------------------------------------------------------- the package's calls
def _own_gate(s):
    from chunked_gated_delta_09_gb300 import gated_norm_bwd, gated_norm_fwd
    c = s["case"]
    out = dict(y=gated_norm_fwd(s["x"], s["z"], s["w"], eps=EPS, activation=c["act"]))
    if c["train"]:
        d = gated_norm_bwd(s["dy"], s["x"], s["z"], s["w"], eps=EPS, activation=c["act"])
        out.update(dx=d["dx"], dz=d["dz"], dw=d["dweight"])
    return out


def _own_addnorm(s):
    from chunked_gated_delta_09_gb300 import add_norm_bwd, add_norm_fwd
    c = s["case"]
    y, r = add_norm_fwd(s["x"], s["r"], s["w"], s["scale"], eps=EPS)
    out = dict(y=y, r=r)
    if c["train"]:
        channel = c["scale"] == "channel"
        d = add_norm_bwd(s["dy"], s["dr"], r, s["w"], s["scale"], x=s["x"] if channel else None, eps=EPS)
        out.update(dr=d["dresidual"], dx=d["dx"], dw=d["dweight"])
        if channel:
            out["dscale"] = d["dscale"]
    return out


def _own_step(s):
    from chunked_gated_delta_09_gb300 import linrec_step
    y = linrec_step(s["x"], s["g"], s["h"], s["slots"], complement=s["case"]["complement"])
    return dict(y=y, h=s["h"])


def _own_linrec(s):
    from chunked_gated_delta_09_gb300 import linrec_bwd, linrec_fwd
    c = s["case"]
    if not c["train"]:
        h, ht = linrec_fwd(s["x"], s["g"], s["h0"], s["cu"], complement=c["complement"])
        return dict(h=h, ht=ht)
    h, ht, states = linrec_fwd(s["x"], s["g"], s["h0"], s["cu"], complement=c["complement"], return_states=True)
    d = linrec_bwd(s["x"], s["g"], s["dh"], s["h0"], s["dht"], s["cu"], states, complement=c["complement"])
    return dict(h=h, ht=ht, dx=d["dx"], dg=d["dg"], dh0=d["dh0"])


def _own_clip(s):
    from chunked_gated_delta_09_gb300 import clip_grad_norm
    norm = clip_grad_norm(s["grads"], s["max_norm"], out=s["out"], eps=EPS)
    return dict(norm=norm, out=s["out"])


OWN = dict(gate=_own_gate, addnorm=_own_addnorm, step=_own_step, linrec=_own_linrec, clip=_own_clip)


def run(state):
    return (OWN if own else PLAIN)[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without
def work(case):
    """Each input read once and each output written once, though a train case is two calls that both read x."""
    e = 4 if case["dtype"] == "f32" else 2
    if case["op"] == "gate":
        n = case["tokens"] * case["heads"] * case["dim"]
        return dict(bytes=n * e * (6 if case["train"] else 3), flops=n * (30 if case["train"] else 10))
    if case["op"] == "addnorm":
        n, er = case["tokens"] * case["dim"], 4 if case["rtype"] == "f32" else 2
        return dict(bytes=n * ((4 * e + 4 * er) if case["train"] else (2 * e + 2 * er)), flops=n * (20 if case["train"] else 6))
    if case["op"] == "step":
        n, eg = case["batch"] * case["dim"], 4 if case["gtype"] == "f32" else 2
        return dict(bytes=n * (2 * e + eg + 8), flops=n * 5)
    if case["op"] == "linrec":
        n = case["tokens"] * case["dim"] * (1 if case["packed"] else case["batch"])
        eg = 4 if case["gtype"] == "f32" else 2
        return dict(bytes=n * ((4 * e + 2 * eg) if case["train"] else (2 * e + eg)), flops=n * (16 if case["train"] else 5))
    n = sum(math.prod(shape) for shape in _clip_shapes(case))
    return dict(bytes=n * (e + (4 if case["otype"] == "f32" else 2)), flops=n * 3)


# ---------------------------------------------------------------- 64 bits
def _exact_gate(s):
    c = s["case"]
    x, z, w = s["x"].double(), s["z"].double(), s["w"].double()
    d = c["dim"]
    inv = ((x * x).sum(-1, keepdim=True) / d + EPS) ** -0.5
    sg = 1.0 / (1.0 + torch.exp(-z))
    a = z * sg if c["act"] == "silu" else sg
    out = dict(y=inv * x * w * a)
    if c["train"]:
        dy = s["dy"].double()
        out["dz"] = dy * (inv * x * w) * (sg + z * sg * (1.0 - sg) if c["act"] == "silu" else sg * (1.0 - sg))
        up = dy * a
        out["dw"] = (up * x * inv).sum((0, 1, 2))
        up = up * w
        out["dx"] = inv * up - x * inv ** 3 * (up * x).sum(-1, keepdim=True) / d
    return out


def _exact_addnorm(s):
    c = s["case"]
    d = c["dim"]
    scale = s["scale"].double() if c["scale"] == "channel" else s["scale"]
    x, w = s["x"].double(), s["w"].double()
    r = s["r"].double() + x * scale
    inv = ((r * r).sum(-1, keepdim=True) / d + EPS) ** -0.5
    out = dict(y=w * (r * inv), r=r)
    if c["train"]:
        dy = s["dy"].double()
        up = dy * w
        dr = s["dr"].double() + inv * up - r * inv ** 3 * (up * r).sum(-1, keepdim=True) / d
        out.update(dr=dr, dx=dr * scale, dw=(dy * r * inv).sum((0, 1)))
        if c["scale"] == "channel":
            out["dscale"] = (dr * x).sum((0, 1))
    return out


def _exact_step(s):
    at = s["slots"].long()
    a, x, h = torch.exp(s["g"].double()), s["x"].double(), s["h"].double()
    new = h[at] * a + (x - a * x if s["case"]["complement"] else x)
    h[at] = new
    return dict(y=new, h=h)


def _exact_linrec(s):
    """One token after the other, as the recurrence is written; dense sequences side by side."""
    c = s["case"]
    d = c["dim"]
    x, a = s["x"].double(), torch.exp(s["g"].double())
    b = x - a * x if c["complement"] else x
    h, ht, dh0 = torch.empty_like(x), s["h0"].double(), None
    lam = torch.empty_like(x) if c["train"] else None
    if c["train"]:
        dh, dh0 = s["dh"].double(), s["dht"].double()
    spans, at = [], 0
    for i, n in enumerate(s["lens"] if c["packed"] else s["lens"][:1]):
        spans.append((slice(i, i + 1) if c["packed"] else slice(None), at, at + n))
        at += n
    before = torch.empty_like(x)
    for who, lo, hi in spans:
        now = ht[who].clone()
        for t in range(lo, hi):
            before[:, t] = now
            now = torch.addcmul(b[:, t], a[:, t], now)
            h[:, t] = now
        ht[who] = now
        if c["train"]:
            now = dh0[who].clone()
            for t in range(hi - 1, lo - 1, -1):
                now = now + dh[:, t]
                lam[:, t] = now
                now = now * a[:, t]
            dh0[who] = now
    out = dict(h=h, ht=ht)
    if c["train"]:
        out["dx"] = lam - a * lam if c["complement"] else lam
        out["dg"] = lam * a * (before - x if c["complement"] else before)
        out["dh0"] = dh0
    return out


def _exact_clip(s):
    norm = sum(float(t.double().square().sum()) for t in s["grads"]) ** 0.5
    factor = min(1.0, s["max_norm"] / (norm + EPS))
    return dict(norm=norm, out=[t.double() * factor for t in s["grads"]])


EXACT = dict(gate=_exact_gate, addnorm=_exact_addnorm, step=_exact_step, linrec=_exact_linrec, clip=_exact_clip)


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))
