"""Gradients that cannot be differentiated themselves."""
from __future__ import annotations

import torch


class _Once(torch.autograd.Function):
    @staticmethod
    def forward(ctx, name, *grads):
        ctx.name = name
        return tuple(g.data for g in grads)  # the same memory, and no view: it may be changed in place

    @staticmethod
    def backward(ctx, *dy):
        raise RuntimeError("%s is differentiable once" % ctx.name)


def once(name: str, *grads: torch.Tensor | None) -> tuple:
    """The gradients that a backward pass of ``name`` computed without autograd, as autograd has to see them where it
    records that pass (create_graph): whoever asks for gradients of these gets an error.  torch's once_differentiable
    does that only where the upstream itself requires a gradient, although the gradients depend on the operands in any
    case, and a penalty on them would lose its term in silence."""
    if not torch.is_grad_enabled():
        return grads
    some = iter(_Once.apply(name, *(g.detach().requires_grad_(True) for g in grads if g is not None)))
    return tuple(None if g is None else next(some) for g in grads)
