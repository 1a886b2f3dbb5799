"""The backwards are kernels without a derivative of their own: a second derivative is an error, never a gradient that takes
the first one for a constant."""
import pytest
import torch

import block_util as U
from chunked_gated_delta_09_gb300 import add_norm, gated_norm, linear_recurrence
from chunked_gated_delta_09_gb300.ops import chunk_gated_delta_rule

pytestmark = pytest.mark.gpu


def ask_twice(x, *outputs):
    (first,) = torch.autograd.grad(sum(o.float().square().sum() for o in outputs), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        (x.square().sum() + first.square().sum()).backward()


def leaf(gen, *shape):
    return U.randn(gen, *shape).requires_grad_()


def test_gated_norm():
    gen = U.seeded(40)
    x, w = leaf(gen, 3, 2, 64), leaf(gen, 64)
    ask_twice(x, gated_norm(x, U.randn(gen, 3, 2, 64), w))


def test_add_norm():
    gen = U.seeded(41)
    x = leaf(gen, 3, 64)
    ask_twice(x, *add_norm(x, U.randn(gen, 3, 64), U.randn(gen, 64), 0.5))


def test_linear_recurrence():
    gen = U.seeded(42)
    x = leaf(gen, 1, 20, 32)
    ask_twice(x, *linear_recurrence(x, U.gates(gen, 1, 20, 32)))


def test_chunk_gated_delta_rule():
    gen = U.seeded(43)
    q, k, v = (leaf(gen, 1, 64, 2, 32) for _ in range(3))
    beta, g = (torch.rand(1, 64, 2, generator=gen).cuda() for _ in range(2))
    ask_twice(v, *chunk_gated_delta_rule(q, k, v, beta, -g))
