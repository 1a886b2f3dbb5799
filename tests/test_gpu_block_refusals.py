"""The torch calls around the delta rule refuse wrong shapes, types, devices and layouts before anything is launched."""
import pytest
import torch

import chunked_gated_delta_09_gb300 as pkg

pytestmark = pytest.mark.gpu


def z(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


X = (4, 2, 16)
CASES = {
    "gate shape": lambda: pkg.gated_norm_fwd(z(*X), z(4, 2, 8), z(16)),
    "gate type": lambda: pkg.gated_norm_fwd(z(*X), z(*X, dtype=torch.bfloat16), z(16)),
    "weight size": lambda: pkg.gated_norm_fwd(z(*X), z(*X), z(8)),
    "weight on the CPU": lambda: pkg.gated_norm_fwd(z(*X), z(*X), torch.zeros(16)),
    "activation": lambda: pkg.gated_norm_fwd(z(*X), z(*X), z(16), activation="relu"),
    "double": lambda: pkg.gated_norm_fwd(z(*X, dtype=torch.float64), None, None),
    "last axis strided": lambda: pkg.gated_norm_fwd(z(4, 2, 32)[..., ::2], None, None),
    "one axis": lambda: pkg.gated_norm_fwd(z(16), None, None),
    "uneven rows": lambda: pkg.add_norm_fwd(z(4, 4, 16)[:, :3], None, None),
    "dy shape": lambda: pkg.gated_norm_bwd(z(4, 2, 8), z(*X), z(*X), z(16)),
    "residual type": lambda: pkg.add_norm_fwd(z(*X, dtype=torch.bfloat16), z(*X, dtype=torch.float16), None),
    "residual shape": lambda: pkg.add_norm_fwd(z(*X), z(4, 16), None),
    "scale size": lambda: pkg.add_norm_fwd(z(*X), z(*X), None, z(1)),
    "x without a scale": lambda: pkg.add_norm_bwd(z(*X), None, z(*X), None, 1.0, x=z(*X)),
    "dres type": lambda: pkg.add_norm_bwd(z(*X, dtype=torch.bfloat16), z(*X, dtype=torch.bfloat16), z(*X), None),
    "two axes": lambda: pkg.linrec_fwd(z(4, 16), z(4, 16)),
    "gate shape of the recurrence": lambda: pkg.linrec_fwd(z(*X), z(4, 2, 1)),
    "gate type of the recurrence": lambda: pkg.linrec_fwd(z(*X), z(*X, dtype=torch.bfloat16)),
    "h0 shape": lambda: pkg.linrec_fwd(z(*X), z(*X), z(3, 16)),
    "h0 type": lambda: pkg.linrec_fwd(z(*X), z(*X), z(4, 16, dtype=torch.bfloat16)),
    "cu_seqlens with a batch": lambda: pkg.linrec_fwd(z(*X), z(*X), None, z(3, dtype=torch.int32)),
    "cu_seqlens type": lambda: pkg.linrec_fwd(z(1, 4, 8), z(1, 4, 8), None, z(3, dtype=torch.int64)),
    "cu_seqlens of nothing": lambda: pkg.linrec_fwd(z(1, 4, 8), z(1, 4, 8), None, z(1, dtype=torch.int32)),
    "states shape": lambda: pkg.linrec_bwd(z(*X), z(*X), z(*X), states=z(2, 16)),
    "dht shape": lambda: pkg.linrec_bwd(z(*X), z(*X), z(*X), dht=z(2, 16)),
    "step without rows": lambda: pkg.linrec_step(z(4, 8), z(4, 8), z(3, 8)),
    "step slots type": lambda: pkg.linrec_step(z(4, 8), z(4, 8), z(5, 8), z(4, dtype=torch.int64)),
    "step state type": lambda: pkg.linrec_step(z(4, 8), z(4, 8), z(5, 8, dtype=torch.bfloat16)),
    "gradient layout": lambda: pkg.clip_grad_norm([z(8, 8).t()[:4]], 1.0),
    "gradient type": lambda: pkg.grad_norm([z(8, dtype=torch.int32)]),
    "out count": lambda: pkg.clip_grad_norm([z(8), z(8)], 1.0, [z(8)]),
    "out size": lambda: pkg.clip_grad_norm([z(8)], 1.0, [z(9)]),
    "max_norm": lambda: pkg.clip_grad_norm([z(8)], -1.0),
    "max_norm nan": lambda: pkg.clip_grad_norm([z(8)], float("nan")),
}


@pytest.mark.parametrize("name", CASES)
def test_refused(name):
    with pytest.raises(ValueError):
        CASES[name]()


def test_rows_beyond_the_longest_are_unsupported():
    x = z(2, 1, pkg._lib.NORM_MAX_DIM + 1)
    with pytest.raises(pkg.GdrError) as e:
        pkg.gated_norm_fwd(x, None, None)
    assert e.value.status == pkg._lib.GDR_ERR_UNSUPPORTED
