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


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


class AdapterBank:
    """The adapters of one projection of k to n columns: a [adapters, R, k] and
    b [adapters, n, R] in BF16, scale [adapters] in float32, ranks [adapters]
    in int32 (the ranks that each adapter uses; None: all R).  All contiguous,
    on one CUDA device; the tensors stay the caller's, and their values may
    change between calls."""

    def __init__(self, a: torch.Tensor, b: torch.Tensor, scale: torch.Tensor, ranks: torch.Tensor | None = None):
        _need(a.dim() == 3 and b.dim() == 3 and b.shape[0] == a.shape[0] and b.shape[2] == a.shape[1],
              "expected a [adapters, R, k] and b [adapters, n, R]")
        _need(a.dtype == torch.bfloat16 and b.dtype == torch.bfloat16, "a and b must be BF16")
        _need(scale.dtype == torch.float32 and scale.shape == a.shape[:1], "scale must be float32 [adapters]")
        _need(ranks is None or (ranks.dtype == torch.int32 and ranks.shape == a.shape[:1]),
              "ranks must be int32 [adapters]")
        for t in (a, b, scale, ranks):
            _need(t is None or (t.is_cuda and t.is_contiguous() and t.device == a.device),
                  "the bank's tensors must be contiguous, on one CUDA device")
        self.a, self.b, self.scale, self.ranks = a, b, scale, ranks
        self.adapters, self.rank, self.k = a.shape
        self.n = b.shape[1]
        self.device = a.device
        self.desc = B.lct_adapters(a.data_ptr(), b.data_ptr(), scale.data_ptr(),
                                   None if ranks is None else ranks.data_ptr(), self.adapters, self.rank, self.k,
                                   self.n)


class AdapterPlan:
    """A batch's tokens grouped by adapter, as ``adapter_plan`` makes it:
    order [tokens], starts [adapters + 2] and tiles [rows, 4], all int32."""

    def __init__(self, order: torch.Tensor, starts: torch.Tensor, tiles: torch.Tensor):
        self.tokens, self.adapters = order.numel(), starts.numel() - 2
        _need(tiles.dim() == 2 and tiles.shape[1] == 4 and self.adapters > 0
              and tiles.shape[0] == B.lct_adapter_tile_rows(self.tokens, self.adapters),
              "the tables do not belong to one plan")
        for t in (order, starts, tiles):
            _need(t.dtype == torch.int32 and t.is_cuda and t.is_contiguous() and t.device == tiles.device,
                  "the plan's tables must be contiguous int32, on one CUDA device")
        self.order, self.starts, self.tiles = order, starts, tiles
        self.device = tiles.device
        self.desc = B.lct_token_plan(order.data_ptr(), starts.data_ptr(), tiles.data_ptr(), self.tokens,
                                     self.adapters)

    def status(self) -> int:
        """The plan's latched status (0 is fine); synchronises."""
        return int(self.tiles[0, 3].item())


def adapter_plan(index: torch.Tensor, adapters: int) -> AdapterPlan:
    """Group a batch's tokens by adapter; index is each token's adapter (int32,
    any shape, flattened), -1 for none."""
    _need(index.dtype == torch.int32 and index.is_cuda and index.is_contiguous(),
          "index must be a contiguous int32 CUDA tensor")
    tokens, adapters = index.numel(), int(adapters)
    if not 0 < adapters <= B.LCT_ADAPTER_MAX:
        raise B.LctError(B.LCT_ERR_UNSUPPORTED if adapters > 0 else B.LCT_ERR_INVALID_ARG, "adapter_plan")
    rows = B.lct_adapter_tile_rows(tokens, adapters)
    # one allocation: the tile table first, which has to be aligned
    buf = torch.empty(4 * rows + tokens + adapters + 2, dtype=torch.int32, device=index.device)
    tiles, order, starts = buf.split([4 * rows, tokens, adapters + 2])
    plan = AdapterPlan(order, starts, tiles.view(rows, 4))
    with B.on_device(index.device.index):
        B.lct_adapter_plan(index, adapters, order, starts, plan.tiles)
    return plan


def _rows(t: torch.Tensor, cols: int, tokens: int, device: torch.device, what: str) -> torch.Tensor:
    """t [..., cols] as a matrix of `tokens` rows."""
    if t.dtype != torch.bfloat16 or t.device != device or t.shape[-1:] != (cols,) or t.numel() != tokens * cols:
        raise ValueError("%s: expected a BF16 tensor of %d rows of %d on %s" % (what, tokens, cols, device))
    m = t if t.dim() == 2 else t.view(tokens, cols)
    if m.stride(1) != 1 and cols > 1:
        raise ValueError("%s: values of a row must lie side by side" % what)
    if m.stride(0) < cols:  # the stride of a single row means nothing
        _need(tokens <= 1, "%s: rows must not overlap" % what)
        m = m.as_strided((tokens, cols), (cols, 1))
    return m


def _match(bank: AdapterBank, plan: AdapterPlan) -> None:
    _need(plan.adapters == bank.adapters and plan.device == bank.device,
          "the plan must be for the bank's adapters, on its device")


def adapter_apply(x: torch.Tensor, bank: AdapterBank, plan: AdapterPlan, y: torch.Tensor,
                  out: torch.Tensor | None = None, keep: bool = False):
    """out = y + s_a (x A_a^T) B_a^T for every token (out = y for tokens without
    an adapter); x [..., k], y and out [..., n], BF16, rows at any stride.  out
    may be y itself; by default it is a new tensor.  With `keep`, returns (out,
    xa): xa = x A_a^T, float32 [tokens, R], is what ``adapter_grads`` needs."""
    _match(bank, plan)
    tokens = plan.tokens
    xm, ym = _rows(x, bank.k, tokens, bank.device, "x"), _rows(y, bank.n, tokens, bank.device, "y")
    if out is None:
        out = torch.empty(y.shape, dtype=torch.bfloat16, device=bank.device)
    om = _rows(out, bank.n, tokens, bank.device, "out")
    xa = torch.empty(tokens, bank.rank, dtype=torch.float32, device=bank.device) if keep else None
    with B.on_device(bank.device.index):
        B.lct_adapter_forward(bank.desc, plan.desc, xm, ym, om, xa)
    return (out, xa) if keep else out


def adapter_grads(dy: torch.Tensor, x: torch.Tensor, xa: torch.Tensor, bank: AdapterBank, plan: AdapterPlan,
                  dx: torch.Tensor | None, out: torch.Tensor | None = None):
    """(dx', da, db): the gradients of ``adapter_apply`` for dy, the gradient of
    its out.  dx is the shared projection's gradient of x, to which the
    adapters' part is added, into `out` (may be dx itself) or a new tensor; None
    where no gradient of x is wanted, and dx' is then None."""
    _match(bank, plan)
    tokens = plan.tokens
    dym, xm = _rows(dy, bank.n, tokens, bank.device, "dy"), _rows(x, bank.k, tokens, bank.device, "x")
    if xa.dtype != torch.float32 or xa.shape != (tokens, bank.rank) or not xa.is_contiguous() \
            or xa.device != bank.device:
        raise ValueError("xa: expected contiguous float32 [tokens, R] on the bank's device")
    dxm = om = None
    if dx is not None:
        dxm = _rows(dx, bank.k, tokens, bank.device, "dx")
        if out is None:
            out = torch.empty(dx.shape, dtype=torch.bfloat16, device=bank.device)
        om = _rows(out, bank.k, tokens, bank.device, "out")
    da, db = torch.empty_like(bank.a), torch.empty_like(bank.b)
    work = torch.empty(B.lct_adapter_work_bytes(tokens, bank.rank), dtype=torch.uint8, device=bank.device)
    with B.on_device(bank.device.index):
        B.lct_adapter_backward(bank.desc, plan.desc, dym, xm, xa, dxm, om, da, db, work)
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
