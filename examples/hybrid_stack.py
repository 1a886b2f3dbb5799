"""A small stack that alternates delta-rule blocks with blocks of the gated linear recurrence, trained for a few steps and
then run token by token: the operators around the delta rule as a model uses them.

    python examples/hybrid_stack.py [--steps 20] [--tokens 512] [--dim 256]

Each block reads the residual stream through ``add_norm`` (which adds the block before it, scaled per channel, and
normalises), mixes its tokens by ``chunk_gated_delta_rule`` or ``linear_recurrence``, normalises the result per head and
gates it by ``gated_norm``, and projects it back.  The gradients are clipped by ``clip_grad_norm``.  The projections are
plain matrix products of torch.  The task: of a sequence of random vectors, answer each with the one three tokens before.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunked_gated_delta_09_gb300 import (add_norm, add_norm_fwd, clip_grad_norm, gated_norm, gated_norm_fwd,  # noqa: E402
                                          linear_recurrence, linrec_step)
from chunked_gated_delta_09_gb300.ops import chunk_gated_delta_rule  # noqa: E402


def _weight(gen, rows, cols):
    w = torch.randn(rows, cols, generator=gen, device="cuda") * cols ** -0.5
    return w.to(torch.bfloat16).requires_grad_()


class Mixer:
    """What the two kinds of block share: the norm and the residual scale before, the gated norm and the projection after."""

    def __init__(self, dim, heads, gen, inner):
        self.heads, self.dim = heads, dim
        self.norm = torch.ones(dim, device="cuda").requires_grad_()
        self.scale = torch.full((dim,), 0.5, device="cuda").requires_grad_()
        self.head_norm = torch.ones(dim // heads, device="cuda").requires_grad_()
        self.inp = _weight(gen, inner, dim)
        self.out = _weight(gen, dim, dim)

    def parameters(self):
        return [self.norm, self.scale, self.head_norm, self.inp, self.out]

    def close(self, o, z):
        o, z = o.unflatten(-1, (self.heads, -1)), z.unflatten(-1, (self.heads, -1))
        return gated_norm(o, z, self.head_norm).flatten(-2) @ self.out.t()


class DeltaBlock(Mixer):
    """Queries, keys, values and the gate of width dim each, beta and the log-decay for each head."""

    def __init__(self, dim, heads, gen):
        super().__init__(dim, heads, gen, 4 * dim + 2 * heads)

    def __call__(self, x):
        q, k, v, z, b, g = (x @ self.inp.t()).split([self.dim] * 4 + [self.heads] * 2, -1)
        q, k, v = (t.unflatten(-1, (self.heads, -1)) for t in (q, k, v))
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype) for t in (q, k))
        o, _ = chunk_gated_delta_rule(q.contiguous(), k.contiguous(), v.contiguous(), torch.sigmoid(b.float()),
                                      torch.nn.functional.logsigmoid(g.float() + 4.0).contiguous())
        return self.close(o.flatten(-2), z)


class RecurrenceBlock(Mixer):
    """Input, log-decay and gate of width dim each; the projection's slices are used where they lie."""

    def __init__(self, dim, heads, gen):
        super().__init__(dim, heads, gen, 3 * dim)

    def __call__(self, x):
        u, g, z = (x @ self.inp.t()).chunk(3, -1)
        h, _ = linear_recurrence(u, torch.nn.functional.logsigmoid(g.float()), complement=True)
        return self.close(h, z)

    @torch.no_grad()
    def step(self, x, state):
        """One token for each sequence; state fp32 [B, dim] is updated in place."""
        u, g, z = (x @ self.inp.t()).chunk(3, -1)
        h = linrec_step(u, torch.nn.functional.logsigmoid(g.float()), state, complement=True)
        return gated_norm_fwd(h.unflatten(-1, (self.heads, -1)), z.unflatten(-1, (self.heads, -1)),
                              self.head_norm).flatten(-2) @ self.out.t()


class Stack:
    """The residual stream is fp32; each block's result is added, scaled, by the norm of the next."""

    def __init__(self, dim=256, heads=4, kinds="rdr", seed=0):
        gen = torch.Generator("cuda").manual_seed(seed)
        self.blocks = [DeltaBlock(dim, heads, gen) if k == "d" else RecurrenceBlock(dim, heads, gen) for k in kinds]
        self.last_norm = torch.ones(dim, device="cuda").requires_grad_()
        self.last_scale = torch.full((dim,), 0.5, device="cuda").requires_grad_()
        self.head = _weight(gen, dim, dim)

    def parameters(self):
        return [p for b in self.blocks for p in b.parameters()] + [self.last_norm, self.last_scale, self.head]

    def __call__(self, x):
        stream, out = x.float(), torch.zeros_like(x)
        for block in self.blocks:
            y, stream = add_norm(out, stream, block.norm, block.scale)
            out = block(y)
        y, _ = add_norm(out, stream, self.last_norm, self.last_scale)
        return y @ self.head.t()

    @torch.no_grad()
    def step(self, x, states):
        """One token for each sequence through a stack of recurrences alone: x [B, dim], a state for each block."""
        stream, out = x.float(), torch.zeros_like(x)
        for block, state in zip(self.blocks, states):
            y, stream = add_norm_fwd(out, stream, block.norm, block.scale)
            out = block.step(y, state)
        y, _ = add_norm_fwd(out, stream, self.last_norm, self.last_scale)
        return y @ self.head.t()


def train(steps=20, tokens=512, dim=256, batch=4, lr=3e-3, max_norm=1.0):
    """Adam on fp32 copies of the weights; returns the loss of each step."""
    model = Stack(dim)
    params = model.parameters()
    master = [p.detach().float().clone() for p in params]
    first, second = ([torch.zeros_like(m) for m in master] for _ in range(2))
    clipped = [torch.empty_like(m) for m in master]
    gen = torch.Generator("cuda").manual_seed(1)
    losses = []
    for i in range(1, steps + 1):
        x = torch.randn(batch, tokens, dim, generator=gen, device="cuda", dtype=torch.bfloat16)
        answer = model(x)
        loss = (answer[:, 3:].float() - x[:, :-3].float()).square().mean()
        grads = torch.autograd.grad(loss, params)
        clip_grad_norm(grads, max_norm, clipped)  # the bf16 and fp32 gradients into the optimizer's fp32 ones
        with torch.no_grad():
            for p, m, u, v, g in zip(params, master, first, second, clipped):
                u.lerp_(g, 0.1)
                v.lerp_(g * g, 0.01)
                m.sub_(lr * (u / (1 - 0.9 ** i)) / ((v / (1 - 0.99 ** i)).sqrt() + 1e-8))
                p.copy_(m)
        losses.append(loss.detach())
    return [float(v) for v in losses]


@torch.no_grad()
def decode_error(tokens=64, dim=256, batch=3):
    """A stack of recurrences run over whole sequences against the same, a token at a time: relative difference."""
    model = Stack(dim, kinds="rr", seed=2)
    x = torch.randn(batch, tokens, dim, generator=torch.Generator("cuda").manual_seed(3), device="cuda").bfloat16()
    whole = model(x)
    states = [torch.zeros(batch, dim, device="cuda") for _ in model.blocks]
    single = torch.stack([model.step(x[:, t], states) for t in range(tokens)], 1)
    return float((whole.float() - single.float()).norm() / whole.float().norm())


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--tokens", type=int, default=512)
    ap.add_argument("--dim", type=int, default=256)
    args = ap.parse_args()
    losses = train(args.steps, args.tokens, args.dim)
    print("loss " + " ".join(f"{v:.3f}" for v in losses))
    print(f"token by token against whole sequences: {decode_error(dim=args.dim):.2e}")


if __name__ == "__main__":
    main()
