"""The global norm of a list of gradients, and clipping by it, before the fused
optimizer steps that take them (``lct_sgd_momentum_step_fused``,
``lct_adamw_step_fused``).

    norm = clip_grads([p.grad for p in params], max_norm=1.0)

Only orchestration lives here: the sums and the scaling run in liblct's
kernels, on the current stream, and nothing synchronises.
"""
from __future__ import annotations

import torch

from . import binding as B


def _scratch(g: B.GradArrays, device) -> tuple[torch.Tensor, torch.Tensor]:
    if device is None:
        device = torch.device("cuda", next(iter(g.devices)) if g.devices else torch.cuda.current_device())
    work = torch.empty(B.LCT_GRAD_WORK_BYTES, dtype=torch.uint8, device=device)
    return torch.empty((), dtype=torch.float32, device=device), work


def grad_norm(grads, device=None) -> torch.Tensor:
    """sqrt(sum of g^2) over every value of `grads` (contiguous BF16 or float32
    CUDA tensors), a float32 scalar on the device.  An empty list gives 0."""
    g = B.GradArrays(grads)
    norm, work = _scratch(g, device)
    with torch.cuda.device(norm.device):
        B.lct_grad_norm(g, norm, work)
    return norm


def clip_grads(grads, max_norm: float, out=None) -> torch.Tensor:
    """Scale every gradient by min(1, max_norm / (norm + 1e-6)), in place or
    into `out` (tensors of the same sizes and types); returns the norm before
    clipping, a float32 scalar on the device."""
    g = B.GradArrays(grads)
    o = g if out is None else B.GradArrays(out, "out")
    if o.devices != g.devices:
        raise ValueError("out must be on the gradients' device")
    norm, work = _scratch(g, None)
    with torch.cuda.device(norm.device):
        B.lct_grad_clip(g, o, max_norm, norm, work)
    return norm
