"""The example that runs the operators together: its loss falls, its gradients reach every weight, and a stack run token by
token gives what it gives on whole sequences."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


def test_training_lowers_the_loss():
    import hybrid_stack
    losses = hybrid_stack.train(steps=25, tokens=192, dim=128)
    # the answer's variance is 1, so a model that has learnt nothing stays above it
    assert losses[-1] < 0.9 * losses[0], losses


def test_gradients_reach_every_weight():
    import hybrid_stack
    model = hybrid_stack.Stack(128)
    x = torch.randn(2, 70, 128, device="cuda").bfloat16()
    grads = torch.autograd.grad(model(x).float().square().mean(), model.parameters())
    for g, p in zip(grads, model.parameters()):
        assert g.shape == p.shape and g.dtype == p.dtype and torch.isfinite(g).all()
    # (the first block's input is the stream alone: what it adds is zero, and so is its scale's gradient)
    assert all(float(g.float().norm()) > 0 for i, g in enumerate(grads) if i != 1)


def test_token_by_token():
    import hybrid_stack
    # two blocks of bf16 results, each rounded a few times on either way: 2^-8 for each of some ten roundings in a row
    assert hybrid_stack.decode_error(tokens=48, dim=128) < 10 * 2.0 ** -8
