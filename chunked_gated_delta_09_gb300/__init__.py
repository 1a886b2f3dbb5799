"""GB300 chunked gated delta rule, and the operators around it.

The backward runs in libgdrbwd.so (hand-written sm_103a CUDA behind the C ABI of include/gdr_bwd.h);
this package builds it (``build``), loads it (``_lib``) and marshals torch tensors into it (``ops``).
``block`` has what surrounds the rule in a model (include/gdr_block.h): the norms before and after a block,
the gated linear recurrence, and the gradient clip.
``inputs`` holds the seeded synthetic workloads and ``counts`` the FLOP and byte conventions.
"""
from .ops import GdrBwdPlan, chunk_indices, gdr_bwd, plan_for, problem_to_device  # noqa: F401
from .block import (add_norm, add_norm_bwd, add_norm_fwd, clip_grad_norm, gated_norm, gated_norm_bwd,  # noqa: F401
                    gated_norm_fwd, grad_norm, linear_recurrence, linrec_bwd, linrec_fwd, linrec_step)
from ._lib import GdrError  # noqa: F401
