"""The gradient norm and clip on the GPU against 64 bits: mixed types and sizes, empty tensors, odd alignment, more
tensors than one launch holds, norms that are zero or not finite, in place and into other types."""
import pytest
import torch

import block_util as U
from chunked_gated_delta_09_gb300 import clip_grad_norm, grad_norm

pytestmark = pytest.mark.gpu


def norm64(ts):
    return float(sum(U.f64(t).square().sum() for t in ts)) ** 0.5


def check(grads, max_norm, out=None, eps=1e-6):
    ref = [U.f64(t) for t in grads]
    n = norm64(grads)
    assert abs(float(grad_norm(grads)) - n) <= U.FP32_BAR * n
    got = clip_grad_norm(grads, max_norm, out, eps=eps)
    assert got.shape == () and got.dtype == torch.float32 and abs(float(got) - n) <= U.FP32_BAR * n
    f = min(1.0, max_norm / (n + eps))
    for t, r in zip(grads if out is None else out, ref):
        if t.numel():
            assert U.rel(t, f * r) <= U.BAR[t.dtype]
    if out is not None:
        assert all(torch.equal(U.f64(t), r) for t, r in zip(grads, ref))


SHAPES = [(64, 64), (1,), (0,), (7, 13), (33000,), (3, 0, 5), (16384,), (16385,), (128,)]


@pytest.mark.parametrize("max_norm", [0.5, 1e6])
@pytest.mark.parametrize("where", ["in place", "f32", "bf16"])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_clip(dtype, where, max_norm):
    gen = U.seeded(1)
    grads = [U.randn(gen, *s, dtype=dtype) for s in SHAPES]
    out = None
    if where != "in place":
        out = [torch.full_like(t, float("nan"), dtype=torch.float32 if where == "f32" else torch.bfloat16) for t in grads]
    check(grads, max_norm, out)


def test_mixed_types_and_odd_alignment():
    gen = U.seeded(2)
    grads = [U.randn(gen, 1001, dtype=torch.bfloat16)[1:], U.randn(gen, 70000)[3:], U.randn(gen, 9, dtype=torch.float16),
             U.randn(gen, 40000, dtype=torch.bfloat16)[8:]]
    check(grads, 1.0, [torch.empty(t.numel() + 1, device="cuda")[1:] for t in grads])
    check(grads, 1.0)


@pytest.mark.parametrize("count", [1, 639, 640, 641, 1500])
def test_many_tensors(count):
    gen = U.seeded(count)
    flat = U.randn(gen, count * 40)
    grads = [flat[40 * i:40 * i + 1 + i % 39] for i in range(count)]
    check(grads, 1.0)


def test_large_total():
    """More elements than the grid takes in one round."""
    gen = torch.Generator(device="cuda").manual_seed(3)
    grads = [torch.randn(n, generator=gen, device="cuda").bfloat16() for n in (30_000_001, 5, 12_000_000)]
    n = float(torch.stack([t.double().square().sum() for t in grads]).sum().sqrt())
    out = [torch.empty_like(t, dtype=torch.float32) for t in grads]
    got = clip_grad_norm(grads, 10.0, out)
    assert abs(float(got) - n) <= U.FP32_BAR * n
    for t, o in zip(grads, out):
        assert float((o.double() - t.double() * (10.0 / (n + 1e-6))).norm() / o.double().norm()) <= U.FP32_BAR


def test_norms_that_are_zero_or_not_finite():
    z = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    assert float(clip_grad_norm(z, 1.0)) == 0.0 and not z[0].any()
    assert float(grad_norm([torch.zeros(0, device="cuda")])) == 0.0
    assert float(clip_grad_norm([torch.zeros(0, device="cuda")], 1.0)) == 0.0
    g = [torch.tensor([1.0, float("inf"), -2.0], device="cuda"), torch.ones(5, device="cuda")]
    assert float(clip_grad_norm(g, 1.0)) == float("inf")
    assert torch.equal(g[1], torch.zeros_like(g[1])) and torch.isnan(g[0][1]) and g[0][0] == 0
    g = [torch.tensor([1.0, float("nan")], device="cuda"), torch.ones(5, device="cuda")]
    assert torch.isnan(clip_grad_norm(g, 1.0)) and torch.isnan(g[1]).all()
    g = [torch.ones(4, device="cuda")]
    assert float(clip_grad_norm(g, 0.0)) == 2.0 and not g[0].any()


def test_results_repeat_bit_for_bit_and_streams():
    gen = U.seeded(4)
    grads = [U.randn(gen, 200001), U.randn(gen, 77)]
    a = clip_grad_norm(grads, 1.0, [torch.empty_like(t) for t in grads])
    assert all(torch.equal(a, grad_norm(grads)) for _ in range(5))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = clip_grad_norm(grads, 1.0, [torch.empty_like(t) for t in grads], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)


def test_capture_in_a_graph():
    """The call copies nothing from the host, so a training step that ends with it can be captured."""
    gen = U.seeded(5)
    grads = [U.randn(gen, 5000), U.randn(gen, 300, dtype=torch.bfloat16)]
    out = [torch.empty_like(t, dtype=torch.float32) for t in grads]
    clip_grad_norm(grads, 1.0, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip_grad_norm(grads, 1.0, out)
    for t in grads:
        t.mul_(3.0)
    graph.replay()
    n = norm64(grads)
    assert abs(float(norm) - n) <= U.FP32_BAR * n
    assert all(U.rel(o, U.f64(t) / (n + 1e-6)) <= U.FP32_BAR for o, t in zip(out, grads))


@pytest.mark.parametrize("pieces", [31, 32, 33])
def test_around_the_largest_single_launch(pieces):
    gen = U.seeded(pieces)
    check([U.randn(gen, 16384 * (pieces - 3) + 5), U.randn(gen, 3, dtype=torch.bfloat16), U.randn(gen, 100)], 1.0)


def test_a_tensor_beyond_32_bits():
    n = (1 << 31) + 70000
    g = torch.full((n,), 0.5, device="cuda", dtype=torch.bfloat16)
    g[-3:] = torch.tensor([1.0, 2.0, -4.0], device="cuda").bfloat16()
    norm = clip_grad_norm([g], 1.0)
    ref = ((n - 3) * 0.25 + 21.0) ** 0.5
    assert abs(float(norm) - ref) <= U.FP32_BAR * ref
    assert U.rel(g[-3:], torch.tensor([1.0, 2.0, -4.0], dtype=torch.float64) / (ref + 1e-6)) <= U.BAR[torch.bfloat16]


def test_axes_may_be_permuted():
    """Gradients of transposed and channels-last weights, in place and into tensors of their layout."""
    gen = U.seeded(6)

    def lists(dtype):
        return [U.randn(gen, 30, 50, dtype=dtype).t(), U.randn(gen, 4, 6, 5, 3).to(dtype).to(memory_format=torch.channels_last),
                U.randn(gen, 9, dtype=dtype), U.randn(gen, 7, 1, 4).to(dtype).permute(2, 1, 0)]

    for dtype in (torch.float32, torch.bfloat16):
        grads = lists(dtype)
        assert not grads[0].is_contiguous() and not grads[3].is_contiguous()
        check(grads, 1.0, [torch.full_like(t, float("nan"), dtype=torch.float32) for t in grads])
        check(grads, 1.0)
    grads, out = lists(torch.float32), lists(torch.float32)
    for bad in (0, 1, 3):
        with pytest.raises(ValueError):
            clip_grad_norm(grads, 1.0, [t.contiguous() if i == bad else t for i, t in enumerate(out)])
    with pytest.raises(ValueError):
        grad_norm([U.randn(gen, 1, 8).expand(4, 8)])
    with pytest.raises(ValueError):
        grad_norm([U.randn(gen, 8, 8).t()[::2]])


def test_weights_that_took_no_part_have_no_gradient():
    gen = U.seeded(7)
    a, b = U.randn(gen, 40), U.randn(gen, 5, 5)
    n = norm64([a, b])
    assert abs(float(grad_norm([None, a, None, b])) - n) <= U.FP32_BAR * n
    out = [None, torch.empty_like(a), torch.full((3,), 7.0, device="cuda"), torch.empty_like(b)]
    for stream in (None, torch.cuda.current_stream()):
        clip_grad_norm([None, a, None, b], 1.0, out, stream=stream)
        assert U.rel(out[1], U.f64(a) / (n + 1e-6)) <= U.FP32_BAR and U.rel(out[3], U.f64(b) / (n + 1e-6)) <= U.FP32_BAR
        assert (out[2] == 7.0).all()
    for call in (lambda: grad_norm([None, None]), lambda: clip_grad_norm([None], 1.0),
                 lambda: clip_grad_norm([a, None], 1.0, [a]), lambda: clip_grad_norm([a], 1.0, [None])):
        with pytest.raises(ValueError):
            call()
    x, unused = U.randn(gen, 8).requires_grad_(), U.randn(gen, 8).requires_grad_()
    x.square().sum().backward()
    clip_grad_norm([p.grad for p in (x, unused)], 1.0)
    assert abs(float(x.grad.norm()) - 1.0) <= U.FP32_BAR
