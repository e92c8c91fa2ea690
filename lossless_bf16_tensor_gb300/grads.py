"""The global norm of a list of gradients, and clipping by it, before the fused
optimizer steps that take them (``lct_sgd_momentum_step_fused``,
``lct_adamw_step_fused``).

    norm = clip_grads([p.grad for p in params], max_norm=1.0)

Only orchestration lives here: the sums and the scaling run in liblct's
kernels, on the current stream, and nothing synchronises.  Gradients that stay
in the same buffers from step to step may be given as one ``GradArrays``, which
spares the collecting of their addresses.
"""
from __future__ import annotations

import torch

from . import binding as B

_SCRATCH = B.LCT_GRAD_WORK_BYTES // 4


def _arrays(tensors, what: str) -> B.GradArrays:
    return tensors if isinstance(tensors, B.GradArrays) else B.GradArrays(tensors, what)


def _buffers(g: B.GradArrays) -> tuple[torch.Tensor, torch.Tensor]:
    """The norm and the calls' scratch, from one allocation."""
    device = g.tensors[0].device if g.count else torch.device("cuda", g.device)
    buf = torch.empty(_SCRATCH + 4, dtype=torch.float32, device=device)
    return buf[_SCRATCH], buf


def grad_norm(grads) -> torch.Tensor:
    """sqrt(sum of g^2) over every value of `grads` (contiguous BF16 or float32
    CUDA tensors on one device), a float32 scalar there.  An empty list gives
    0."""
    g = _arrays(grads, "gradients")
    norm, work = _buffers(g)
    B.lct_grad_norm(g, norm, work)
    return norm


def clip_grads(grads, max_norm: float, out=None) -> torch.Tensor:
    """Scale every gradient by min(1, max_norm / (norm + 1e-6)), in place or
    into `out` (tensors of the same sizes and types); returns the norm before
    clipping, a float32 scalar on the device."""
    g = _arrays(grads, "gradients")
    o = g if out is None else _arrays(out, "out")
    norm, work = _buffers(g)
    B.lct_grad_clip(g, o, max_norm, norm, work)
    return norm
