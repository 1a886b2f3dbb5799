"""What the calls write in place counts as written: a backward that has saved it raises instead of using the new values."""
import pytest
import torch

import block_util as U
from chunked_gated_delta_09_gb300 import clip_grad_norm, grad_norm, linrec_step

pytestmark = pytest.mark.gpu


def saved_by_a_backward(t):
    """A loss whose backward needs t as it is now."""
    return (torch.ones_like(t).requires_grad_() * t).sum()


def overwritten(loss):
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()


def test_step():
    gen = U.seeded(70)
    state, x = U.randn(gen, 4, 32), U.randn(gen, 2, 32)
    loss, kept = saved_by_a_backward(state), saved_by_a_backward(x)
    linrec_step(x, -x.abs(), state, torch.tensor([2, 0], dtype=torch.int32, device="cuda"))
    overwritten(loss)
    kept.backward()


def test_clip():
    gen = U.seeded(71)
    grads = [U.randn(gen, 40), U.randn(gen, 7)]
    out = [torch.empty_like(t) for t in grads]
    kept, loss = [saved_by_a_backward(t) for t in grads], [saved_by_a_backward(t) for t in out]
    grad_norm(grads)
    clip_grad_norm(grads, 1.0, out)
    for a, b in zip(kept, loss):
        a.backward()
        overwritten(b)
    loss = [saved_by_a_backward(t) for t in grads]
    clip_grad_norm(grads, 1.0)
    for a in loss:
        overwritten(a)
    with torch.inference_mode():
        clip_grad_norm([torch.ones(5, device="cuda")], 1.0)
