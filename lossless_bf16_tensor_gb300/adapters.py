"""Low-rank adapters of many requests beside a shared projection, whose weight
stays compressed (``compressed_linear``): serving many adapters at once, and
training them.

    plan = adapter_plan(index, bank.adapters)      # each token's adapter, -1 for none: once for a batch
    y = compressed_linear(x, w, cb, n, k)
    adapter_apply(x, bank, plan, y, out=y)         # y += s_a (x A_a^T) B_a^T

``adapter_linear`` is both in one call, with gradients for x and the bank.
Only orchestration lives here: the products run in liblct's kernels, on the
current stream, and nothing synchronises.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from .calls import calls
from .matmul import compressed_linear, compressed_linear_input_grad


class AdapterBank:
    """The adapters of one projection of k to n columns: a [adapters, R, k] and
    b [adapters, n, R] in BF16, scale [adapters] in float32, ranks [adapters]
    in int32 (the ranks that each adapter uses; None: all R).  All contiguous,
    on one CUDA device; the tensors stay the caller's, and their values may
    change between calls."""

    __slots__ = ("a", "b", "scale", "ranks", "adapters", "rank", "k", "n", "device")

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor, ranks: torch.Tensor | None = None):
        self.adapters, self.rank, self.k, self.n, self.device = calls.check_bank(a, b, scale, ranks)
        self.a, self.b, self.scale, self.ranks = a, b, scale, ranks


class AdapterPlan:
    """A batch's tokens grouped by adapter, as ``adapter_plan`` makes it:
    order [tokens], starts [adapters + 2] and tiles [rows, 4], all int32."""

    __slots__ = ("order", "starts", "tiles", "tokens", "adapters", "device")

    def __init__(self, order: torch.Tensor, starts: torch.Tensor, tiles: torch.Tensor):
        self.tokens, self.adapters, self.device = calls.check_plan(order, starts, tiles)
        self.order, self.starts, self.tiles = order, starts, tiles

    def status(self) -> int:
        """The plan's latched status (0 is fine); synchronises."""
        return int(self.tiles[0, 3].item())


def adapter_plan(index: torch.Tensor, adapters: int) -> AdapterPlan:
    """Group a batch's tokens by adapter; index is each token's adapter (int32,
    any shape, flattened), -1 for none."""
    return AdapterPlan(*calls.adapter_plan(index, adapters))


def adapter_apply(x: torch.Tensor, bank: AdapterBank, plan: AdapterPlan, y: torch.Tensor,
                  out: torch.Tensor | None = None, keep: bool = False):
    """out = y + s_a (x A_a^T) B_a^T for every token (out = y for tokens without
    an adapter); x [..., k], y and out [..., n], BF16, rows at any stride.  out
    may be y itself; by default it is a new tensor.  With `keep`, returns (out,
    xa): xa = x A_a^T, float32 [tokens, R], is what ``adapter_grads`` needs.
    Autograd does not see this call: it raises where an operand requires a
    gradient and gradients are enabled (``adapter_linear`` gives them)."""
    return calls.adapter_apply(bank.a, bank.b, bank.scale, bank.ranks, plan.order, plan.starts, plan.tiles, x, y, out,
                               bool(keep))


def adapter_grads(dy: torch.Tensor, x: torch.Tensor, xa: torch.Tensor, bank: AdapterBank, plan: AdapterPlan,
                  dx: torch.Tensor | None, out: torch.Tensor | None = None):
    """(dx', da, db): the gradients of ``adapter_apply`` for dy, the gradient of
    its out.  dx is the shared projection's gradient of x, to which the
    adapters' part is added, into `out` (may be dx itself) or a new tensor; None
    where no gradient of x is wanted, and dx' is then None."""
    return calls.adapter_grads(bank.a, bank.b, bank.scale, bank.ranks, plan.order, plan.starts, plan.tiles, dy, x, xa,
                               dx, out)


_OPERANDS = ("the bank's a", "the bank's b", "the bank's scale", "the bank's ranks", "the plan's order",
             "the plan's starts", "the plan's tiles")


def _rows(x, k):
    """x [..., k] as a matrix whose rows the kernels can read: a copy where its leading dimensions make no single row
    index, or a row's values do not lie side by side."""
    rows = x.reshape(-1, k)
    return rows if rows.stride(1) == 1 and rows.stride(0) >= k else rows.contiguous()


def _versions(tensors):
    return [None if t is None or t.is_inference() else t._version for t in tensors]


class _AdapterLinear(torch.autograd.Function):
    # The bank and the plan are long-lived operands, not activations: they stay out of save_for_backward, whose hooks
    # (compressed_activations) would copy a plain tensor and skip the check of a parameter's version.  Backward makes
    # that check itself.
    @staticmethod
    def forward(ctx, x, a, b, bank, plan, w, cb):
        y = compressed_linear(x, w, cb, bank.n, bank.k)
        operands = (a, b, bank.scale, bank.ranks, plan.order, plan.starts, plan.tiles)
        x = _rows(x, bank.k)
        out, xa = calls.adapter_apply(*operands, x, y, y, True)
        ctx.save_for_backward(x, xa)
        ctx.rest = (operands, _versions(operands), w, cb, bank.n, bank.k)
        return out

    @staticmethod
    @once_differentiable  # the gradients' own gradients are not there: asking for them raises
    def backward(ctx, dy):
        x, xa = ctx.saved_tensors
        operands, versions, w, cb, n, k = ctx.rest
        for name, then, now in zip(_OPERANDS, versions, _versions(operands)):
            if then != now:
                raise RuntimeError("adapter_linear: %s was modified in place between forward and backward "
                                   "(version %s, now %s)" % (name, then, now))
        dy = dy.contiguous()
        dx = compressed_linear_input_grad(dy, w, cb, n, k) if ctx.needs_input_grad[0] else None
        dx, da, db = calls.adapter_grads(*operands, dy, x, xa, dx, dx)
        return dx, da, db, None, None, None, None


def adapter_linear(x: torch.Tensor, w: B.CompressedTensor, cb: B.lct_codebook, bank: AdapterBank,
                   plan: AdapterPlan) -> torch.Tensor:
    """y = x W^T + s_a (x A_a^T) B_a^T for a compressed frozen W [n, k] and each
    token's own adapter; x [..., k] BF16 on CUDA, at any strides.  Differentiable (once) in x and in
    the bank's a and b (leaves such as ``torch.nn.Parameter``); the weight is
    decoded again for the gradient of x.  What it saves for backward goes
    through ``compressed_activations`` like any other saved tensor; the bank
    and the plan are used as they are, and backward raises if one of them was
    modified in place since."""
    if torch.is_grad_enabled() and bank.scale.requires_grad:
        raise RuntimeError("adapter_linear gives no gradient for the bank's scale, but it requires one")
    if torch.is_grad_enabled() and (x.requires_grad or bank.a.requires_grad or bank.b.requires_grad):
        return _AdapterLinear.apply(x, bank.a, bank.b, bank, plan, w, cb)
    y = compressed_linear(x, w, cb, bank.n, bank.k)
    return adapter_apply(_rows(x, bank.k), bank, plan, y, out=y)
