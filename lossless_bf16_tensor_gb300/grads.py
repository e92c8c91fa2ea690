"""The global norm of a list of gradients, and clipping by it, before the fused
optimizer steps that take them (``lct_sgd_momentum_step_fused``,
``lct_adamw_step_fused``).

    norm = clip_grads([p.grad for p in params], max_norm=1.0)

The sums and the scaling run in liblct's kernels (``lct_grad_norm``,
``lct_grad_clip``), on the current stream, and nothing synchronises.
"""
from __future__ import annotations

import torch

from .calls import calls


def grad_norm(grads) -> torch.Tensor:
    """sqrt(sum of g^2) over every value of `grads` (contiguous BF16 or float32
    CUDA tensors on one device), a float32 scalar there.  An empty list gives
    0."""
    return calls.grad_norm(grads)


def clip_grads(grads, max_norm: float, out=None) -> torch.Tensor:
    """Scale every gradient by min(1, max_norm / (norm + 1e-6)), in place or
    into `out` (tensors of the same sizes and types); returns the norm before
    clipping, a float32 scalar on the device."""
    return calls.clip_grads(grads, max_norm, out)
