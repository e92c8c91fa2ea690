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

from . import binding as B
from .matmul import compressed_linear, compressed_linear_input_grad


_BF16 = torch.bfloat16


class AdapterBank:
    """The adapters of one projection of k to n columns: a [adapters, R, k] and
    b [adapters, n, R] in BF16, scale [adapters] in float32, ranks [adapters]
    in int32 (the ranks that each adapter uses; None: all R).  All contiguous,
    on one CUDA device; the tensors stay the caller's, and their values may
    change between calls."""

    __slots__ = ("a", "b", "scale", "ranks", "adapters", "rank", "k", "n", "device", "desc")

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor, ranks: torch.Tensor | None = None):
        if a.dim() != 3 or b.dim() != 3:
            raise ValueError("expected a [adapters, R, k] and b [adapters, n, R]")
        self.adapters, self.rank, self.k = a.shape
        adapters, self.n, rank = b.shape
        if adapters != self.adapters or rank != self.rank:
            raise ValueError("expected a [adapters, R, k] and b [adapters, n, R]")
        if a.dtype is not _BF16 or b.dtype is not _BF16:
            raise ValueError("a and b must be BF16")
        if scale.dtype is not torch.float32 or scale.shape != (adapters,):
            raise ValueError("scale must be float32 [adapters]")
        self.device = device = a.get_device()
        if device < 0 or b.get_device() != device or scale.get_device() != device or not a.is_contiguous() \
                or not b.is_contiguous() or not scale.is_contiguous():
            raise ValueError("the bank's tensors must be contiguous, on one CUDA device")
        if ranks is not None and (ranks.dtype is not torch.int32 or ranks.shape != (adapters,)
                                  or not ranks.is_contiguous() or ranks.get_device() != device):
            raise ValueError("ranks must be contiguous int32 [adapters] on the bank's device")
        self.a, self.b, self.scale, self.ranks = a, b, scale, ranks
        self.desc = B.lct_adapters(a.data_ptr(), b.data_ptr(), scale.data_ptr(),
                                   None if ranks is None else ranks.data_ptr(), adapters, rank, self.k, self.n)


class AdapterPlan:
    """A batch's tokens grouped by adapter, as ``adapter_plan`` makes it:
    order [tokens], starts [adapters + 2] and tiles [rows, 4], all int32."""

    __slots__ = ("order", "starts", "tiles", "tokens", "adapters", "device", "desc")

    def __init__(self, order: torch.Tensor, starts: torch.Tensor, tiles: torch.Tensor):
        self.tokens, self.adapters = tokens, adapters = order.numel(), starts.numel() - 2
        if adapters <= 0 or tiles.shape != (B.lct_adapter_tile_rows(tokens, adapters), 4):
            raise ValueError("the tables do not belong to one plan")
        self.device = device = tiles.get_device()
        for t in (order, starts, tiles):
            if t.dtype is not torch.int32 or t.get_device() != device or device < 0 or not t.is_contiguous():
                raise ValueError("the plan's tables must be contiguous int32, on one CUDA device")
        self.order, self.starts, self.tiles = order, starts, tiles
        self.desc = B.lct_token_plan(order.data_ptr(), starts.data_ptr(), tiles.data_ptr(), tokens, adapters)

    def status(self) -> int:
        """The plan's latched status (0 is fine); synchronises."""
        return int(self.tiles[0, 3].item())


def adapter_plan(index: torch.Tensor, adapters: int) -> AdapterPlan:
    """Group a batch's tokens by adapter; index is each token's adapter (int32,
    any shape, flattened), -1 for none."""
    if index.dtype is not torch.int32 or not index.is_cuda or not index.is_contiguous():
        raise ValueError("index must be a contiguous int32 CUDA tensor")
    tokens, adapters = index.numel(), int(adapters)
    if not 0 < adapters <= B.LCT_ADAPTER_MAX:
        raise B.LctError(B.LCT_ERR_UNSUPPORTED if adapters > 0 else B.LCT_ERR_INVALID_ARG, "adapter_plan")
    rows = B.lct_adapter_tile_rows(tokens, adapters)
    device = index.device
    tiles = torch.empty((rows, 4), dtype=torch.int32, device=device)
    order = torch.empty(tokens, dtype=torch.int32, device=device)
    starts = torch.empty(adapters + 2, dtype=torch.int32, device=device)
    plan = AdapterPlan(order, starts, tiles)
    d = plan.desc
    B.lct_adapter_plan(index, adapters, d.d_order, d.d_starts, d.d_tiles)
    return plan


def _rows(t: torch.Tensor, cols: int, tokens: int, device: int, what: str) -> tuple[int, int]:
    """t [..., cols] as a matrix of `tokens` rows: (address, row stride)."""
    if t.dtype is not _BF16 or t.get_device() != device or t.shape[-1:] != (cols,) or t.numel() != tokens * cols:
        raise ValueError("%s: expected a BF16 tensor of %d rows of %d on CUDA device %d" % (what, tokens, cols, device))
    if t.dim() != 2:
        t = t.view(tokens, cols)
    ld, one = t.stride()
    if tokens <= 1:  # the stride of a single row means nothing
        ld = cols
    if (one != 1 and cols > 1) or ld < cols:
        raise ValueError("%s: values of a row must lie side by side, and rows must not overlap" % what)
    return t.data_ptr(), ld


def _match(bank: AdapterBank, plan: AdapterPlan) -> None:
    if plan.adapters != bank.adapters or plan.device != bank.device:
        raise ValueError("the plan must be for the bank's adapters, on its device")


def _new(t: torch.Tensor) -> torch.Tensor:
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=_BF16, device=t.device)


def adapter_apply(x: torch.Tensor, bank: AdapterBank, plan: AdapterPlan, y: torch.Tensor,
                  out: torch.Tensor | None = None, keep: bool = False):
    """out = y + s_a (x A_a^T) B_a^T for every token (out = y for tokens without
    an adapter); x [..., k], y and out [..., n], BF16, rows at any stride.  out
    may be y itself; by default it is a new tensor.  With `keep`, returns (out,
    xa): xa = x A_a^T, float32 [tokens, R], is what ``adapter_grads`` needs."""
    _match(bank, plan)
    tokens, device = plan.tokens, bank.device
    xm, ym = _rows(x, bank.k, tokens, device, "x"), _rows(y, bank.n, tokens, device, "y")
    if out is None:
        out = _new(y)
    om = _rows(out, bank.n, tokens, device, "out")
    xa = torch.empty((tokens, bank.rank), dtype=torch.float32, device=x.device) if keep else None
    B.lct_adapter_forward(bank.desc, plan.desc, device, xm, ym, om, xa.data_ptr() if keep else None)
    return (out, xa) if keep else out


def adapter_grads(dy: torch.Tensor, x: torch.Tensor, xa: torch.Tensor, bank: AdapterBank, plan: AdapterPlan,
                  dx: torch.Tensor | None, out: torch.Tensor | None = None):
    """(dx', da, db): the gradients of ``adapter_apply`` for dy, the gradient of
    its out.  dx is the shared projection's gradient of x, to which the
    adapters' part is added, into `out` (may be dx itself) or a new tensor; None
    where no gradient of x is wanted, and dx' is then None."""
    _match(bank, plan)
    tokens, device = plan.tokens, bank.device
    dym, xm = _rows(dy, bank.n, tokens, device, "dy"), _rows(x, bank.k, tokens, device, "x")
    if xa.dtype is not torch.float32 or xa.shape != (tokens, bank.rank) or not xa.is_contiguous() \
            or xa.get_device() != device:
        raise ValueError("xa: expected contiguous float32 [tokens, R] on the bank's device")
    dxm = om = (None, 0)
    if dx is not None:
        dxm = _rows(dx, bank.k, tokens, device, "dx")
        if out is None:
            out = _new(dx)
        om = _rows(out, bank.k, tokens, device, "out")
    da, db = torch.empty_like(bank.a), torch.empty_like(bank.b)
    work = torch.empty(B.lct_adapter_work_bytes(tokens, bank.rank), dtype=torch.uint8, device=x.device)
    B.lct_adapter_backward(bank.desc, plan.desc, device, dym, xm, xa.data_ptr(), dxm, om, da.data_ptr(),
                           db.data_ptr(), work.data_ptr())
    return (None if dx is None else out), da, db


class _AdapterLinear(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, b, bank, plan, w, cb):
        y = compressed_linear(x, w, cb, bank.n, bank.k)
        out, xa = adapter_apply(x, bank, plan, y, out=y, keep=True)
        ctx.save_for_backward(x, xa)
        ctx.rest = (bank, plan, w, cb)
        return out

    @staticmethod
    def backward(ctx, dy):
        x, xa = ctx.saved_tensors
        bank, plan, w, cb = ctx.rest
        dy = dy.contiguous()
        dx = compressed_linear_input_grad(dy, w, cb, bank.n, bank.k) if ctx.needs_input_grad[0] else None
        dx, da, db = adapter_grads(dy, x, xa, bank, plan, dx, out=dx)
        return dx, da, db, None, None, None, None


def adapter_linear(x: torch.Tensor, w: B.CompressedTensor, cb: B.lct_codebook, bank: AdapterBank,
                   plan: AdapterPlan) -> torch.Tensor:
    """y = x W^T + s_a (x A_a^T) B_a^T for a compressed frozen W [n, k] and each
    token's own adapter; x [..., k] BF16 on CUDA.  Differentiable in x and in
    the bank's a and b (leaves such as ``torch.nn.Parameter``); the weight is
    decoded again for the gradient of x.  What it saves for backward goes
    through ``compressed_activations`` like any other saved tensor."""
    if torch.is_grad_enabled() and (x.requires_grad or bank.a.requires_grad or bank.b.requires_grad):
        return _AdapterLinear.apply(x, bank.a, bank.b, bank, plan, w, cb)
    y = compressed_linear(x, w, cb, bank.n, bank.k)
    return adapter_apply(x, bank, plan, y, out=y)
