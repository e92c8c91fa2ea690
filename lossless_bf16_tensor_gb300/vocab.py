"""The two ends of a language model, around the matrix of its vocabulary: the
lookup of tokens' rows, and the cross entropy of a projection onto the
vocabulary, both with gradients, for dense and for compressed matrices.

    h = embedding(tokens, table)                           # tokens' rows
    loss = linear_cross_entropy(h, weight, targets)        # mean over the tokens with a target; no logits are kept
    loss.backward()

    loss = compressed_cross_entropy(h, w, cb, vocab, cols, targets)    # a frozen CompressedTensor, decoded by pieces
    dx, dw = compressed_cross_entropy_grads(...)                       # dw: the dense gradient of the fused steps

A negative id is none: a row of zeros, a loss of 0, no gradients, not counted in
the mean.  An id of the vocabulary's size or more gives NaN.  Forward-mode
derivatives are not there: operands that carry a tangent are refused.  Only orchestration
lives here: everything runs in liblct's kernels, on the current stream, and
nothing synchronises.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import binding as B
from .calls import calls
from .matmul import default_tile_blocks, tile_rows
from .once import once

_BACKWARD, _WEIGHT, _UNALIGNED = 1, 2, 4  # LCT_LOSS_*


# ------------------------------------------------------------------ lookup

class _Embedding(torch.autograd.Function):
    @staticmethod
    def forward(ctx, table, tokens, scale):
        ctx.save_for_backward(tokens)
        ctx.rest = (table.shape[0], scale)
        return calls.embedding(tokens, table, 0, 0, scale, None)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        rows, scale = ctx.rest
        return calls.embedding_grad(_rows(dy, dy.shape[-1]), ctx.saved_tensors[0], rows, scale, None, None), None, None


def embedding(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0,
              out: torch.Tensor | None = None) -> torch.Tensor:
    """scale * table[tokens], rounded once: tokens int32 or int64 of any shape,
    table [rows, columns] in BF16 or float32.  Differentiable (once) in the table, whose
    gradient is dense; not into `out`."""
    tokens = tokens.contiguous()
    if out is None and table.requires_grad and torch.is_grad_enabled():
        return _Embedding.apply(table, tokens, scale)
    return calls.embedding(tokens, table, 0, 0, scale, out)


def embedding_grad(dy: torch.Tensor, tokens: torch.Tensor, rows: int, scale: float = 1.0,
                   base: torch.Tensor | None = None, out: torch.Tensor | None = None) -> torch.Tensor:
    """base + scale * (the sum of dy over the tokens of each row), [rows, columns]
    in dy's type: the dense gradient of ``embedding``.  base None is zero.  `out`
    may be base itself, whose rows without tokens are then left alone; by
    default it is a new tensor.  Autograd does not see this call: it raises where
    dy, base or out requires a gradient and gradients are enabled."""
    return calls.embedding_grad(dy, tokens.contiguous(), rows, scale, base, out)


# -------------------------------------------------------------------- loss

def _rows(x, k):
    """x [..., k] as a matrix whose rows the kernels can read: a copy where its leading dimensions make no single row
    index, or a row's values do not lie side by side."""
    if x.dim() == 0 or x.shape[-1] != k:
        raise ValueError("expected x [..., %d]" % k)
    rows = x.reshape(-1, k)
    return rows if rows.stride(1) == 1 and rows.stride(0) >= k else rows.contiguous()


def cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor):
    """(loss, lse), float32 in the shape of the targets: lse = log sum_v exp(x W_v)
    and loss = lse - x W_target (0 without a target).  x [..., k] and weight
    [vocabulary, k] in BF16, rows at any one stride; targets int32 or int64,
    contiguous.  Keeps no logits.  Autograd does not see this call
    (``linear_cross_entropy`` gives gradients, and takes operands at any strides)."""
    return calls.cross_entropy(x, weight, targets)


def cross_entropy_grads(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor, loss: torch.Tensor,
                        lse: torch.Tensor, dloss: torch.Tensor, weight_grad: bool = True):
    """(dx, dw): the gradients of ``cross_entropy``'s loss for dloss, float32, a
    value a token or one for all.  dw is None without `weight_grad` (a frozen
    projection)."""
    return calls.cross_entropy_grads(x, weight, targets, loss, lse, dloss, bool(weight_grad))


_REDUCTIONS = ("mean", "sum", "none")


def _reduction(name):
    if name not in _REDUCTIONS:
        raise ValueError("reduction must be one of %s" % (_REDUCTIONS,))
    return _REDUCTIONS.index(name)


def _reduced(reduction, loss, total):
    return loss if reduction == "none" else total[0] if reduction == "sum" else total[1]


def _upstream(reduction, dy, total):
    """dloss and its factor, as the calls take them."""
    dy = dy.float().contiguous()
    return dy, total[2:] if reduction == "mean" else None


def linear_cross_entropy(x: torch.Tensor, weight: torch.Tensor, targets: torch.Tensor,
                         reduction: str = "mean") -> torch.Tensor:
    """The cross entropy of the projection x W^T against targets, float32: its mean
    over the tokens with a target (0 if there is none), its sum, or
    (reduction "none") each token's.  x [..., k] and weight [vocabulary, k] in
    BF16, at any strides.  Differentiable (once) in x and weight; neither pass
    keeps logits."""
    return calls.linear_cross_entropy(x, weight, targets.contiguous(), _reduction(reduction))


# ------------------------------------------------------ compressed matrices

def _pieces(w, rows, cols, device, tile_blocks):
    """A compressed [rows, cols] matrix as (first row, rows) of its pieces, and the blocks of one."""
    if w.n != rows * cols:
        raise ValueError("weight size does not match its shape")
    if tile_blocks is None:
        tile_blocks = default_tile_blocks(w, cols, device)
    if tile_blocks >= w.nblocks:
        return [(0, rows)], w.nblocks
    step = tile_rows(w, cols, tile_blocks)
    return [(r, min(step, rows - r)) for r in range(0, rows, step)], tile_blocks


def _decoded(w, cb, rows, cols, device, tile_blocks):
    """The pieces of a compressed matrix one after another, each decoded into the same buffer on the current stream."""
    pieces, blocks = _pieces(w, rows, cols, device, tile_blocks)
    dense = torch.empty(pieces[0][1] * cols, dtype=torch.bfloat16, device=device)
    for i, (first, count) in enumerate(pieces):
        piece = dense[:count * cols]
        B.lct_decode_blocks(w, cb, i * blocks, min(blocks, w.nblocks - i * blocks), piece.view(torch.int16),
                            torch.cuda.current_stream(device))
        yield first, piece.view(count, cols)


def compressed_embedding(tokens: torch.Tensor, w: B.CompressedTensor, cb: B.lct_codebook, rows: int, cols: int,
                         scale: float = 1.0, tile_blocks: int | None = None) -> torch.Tensor:
    """``embedding`` from a compressed BF16 table [rows, cols], which is decoded
    `tile_blocks` blocks (whole rows) at a time; by default one wave of decode
    CTAs, as ``compressed_linear`` does."""
    tokens = tokens.contiguous()
    out = torch.empty(*tokens.shape, cols, dtype=torch.bfloat16, device=tokens.device)
    for first, piece in _decoded(w, cb, rows, cols, tokens.device, tile_blocks):
        calls.embedding(tokens, piece, first, rows, scale, out)
    return out


def _unaligned(x, cols):
    """Whether a row of x, or of a piece, begins off a 16-byte boundary."""
    return cols % 8 != 0 or x.data_ptr() % 16 != 0 or (x.shape[0] > 1 and x.stride(0) % 8 != 0)


def _compressed_forward(x, w, cb, rows, cols, targets, tile_blocks):
    x = _rows(x, cols)
    pieces, _ = _pieces(w, rows, cols, x.device, tile_blocks)
    size = calls.loss_work_bytes(targets.numel(), rows, cols, pieces[0][1], _UNALIGNED * _unaligned(x, cols))
    work = torch.empty(size, dtype=torch.uint8, device=x.device)
    loss, lse = (torch.empty(targets.shape, dtype=torch.float32, device=x.device) for _ in range(2))
    total = torch.empty(3, dtype=torch.float32, device=x.device)
    for first, piece in _decoded(w, cb, rows, cols, x.device, tile_blocks):
        calls.cross_entropy_piece(x, piece, first, rows, targets, loss, lse, total, work)
    return x, loss, lse, total


def _compressed_backward(x, w, cb, rows, cols, targets, loss, lse, dloss, scale, weight_grad, tile_blocks):
    x = _rows(x, cols)
    pieces, _ = _pieces(w, rows, cols, x.device, tile_blocks)
    flags = _BACKWARD | _WEIGHT * bool(weight_grad) | _UNALIGNED * _unaligned(x, cols)
    work = torch.empty(calls.loss_work_bytes(targets.numel(), rows, cols, pieces[0][1], flags), dtype=torch.uint8,
                       device=x.device)
    dx = torch.empty(x.shape, dtype=torch.bfloat16, device=x.device)
    dw = torch.empty(rows, cols, dtype=torch.bfloat16, device=x.device) if weight_grad else None
    for first, piece in _decoded(w, cb, rows, cols, x.device, tile_blocks):
        calls.cross_entropy_grads_piece(x, piece, first, rows, targets, loss, lse, dloss, scale, dx,
                                        None if dw is None else dw[first:first + piece.shape[0]], work)
    return dx, dw


class _CompressedCrossEntropy(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, targets, w, cb, rows, cols, reduction, tile_blocks):
        xr, loss, lse, total = _compressed_forward(x, w, cb, rows, cols, targets, tile_blocks)
        ctx.save_for_backward(xr, targets, loss, lse, total)
        ctx.rest = (w, cb, rows, cols, reduction, tile_blocks, x.shape)
        return _reduced(reduction, loss, total).clone()

    @staticmethod
    def backward(ctx, dy):
        x, targets, loss, lse, total = ctx.saved_tensors
        w, cb, rows, cols, reduction, tile_blocks, shape = ctx.rest
        with torch.no_grad():
            dloss, scale = _upstream(reduction, dy, total)
            dx, _ = _compressed_backward(x, w, cb, rows, cols, targets, loss, lse, dloss, scale, False, tile_blocks)
        return once("compressed_cross_entropy", dx.view(shape)) + (None,) * 7


def compressed_cross_entropy(x: torch.Tensor, w: B.CompressedTensor, cb: B.lct_codebook, rows: int, cols: int,
                             targets: torch.Tensor, reduction: str = "mean",
                             tile_blocks: int | None = None) -> torch.Tensor:
    """``linear_cross_entropy`` on a compressed weight [rows, cols], which is
    decoded a piece at a time (and again in backward, until when it has to stay as
    it is): neither the dense weight nor the logits are ever there.  Differentiable
    (once) in x; the weight is frozen (``compressed_cross_entropy_grads`` gives its
    gradient)."""
    _reduction(reduction)
    targets = targets.contiguous()
    if torch.is_grad_enabled() and x.requires_grad:
        return _CompressedCrossEntropy.apply(x, targets, w, cb, rows, cols, reduction, tile_blocks)
    _, loss, _, total = _compressed_forward(x, w, cb, rows, cols, targets, tile_blocks)
    return _reduced(reduction, loss, total)


def compressed_cross_entropy_grads(x: torch.Tensor, w: B.CompressedTensor, cb: B.lct_codebook, rows: int, cols: int,
                                   targets: torch.Tensor, tile_blocks: int | None = None):
    """(loss, dx, dw) of the mean loss on a compressed weight that is being
    trained: dw [rows, cols] is the dense BF16 gradient that the fused steps
    (``lct_adamw_step_fused`` and the others) take."""
    targets = targets.contiguous()
    with torch.no_grad():
        xr, loss, lse, total = _compressed_forward(x, w, cb, rows, cols, targets, tile_blocks)
        one = torch.ones(1, dtype=torch.float32, device=xr.device)
        dx, dw = _compressed_backward(xr, w, cb, rows, cols, targets, loss, lse, one, total[2:], True, tile_blocks)
    return total[1], dx.view(x.shape), dw
