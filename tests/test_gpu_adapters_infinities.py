"""Values that are not finite give what the formulas give: the same infinities and
NaN in the same places, and the usual bound on everything else.  Weights are
positive here, so that an infinity in a row comes through both products as one
instead of meeting its opposite."""
import math

import pytest
import torch

from lossless_bf16_tensor_gb300.adapters import adapter_apply, adapter_grads
from test_gpu_adapters import Case

pytestmark = pytest.mark.gpu


def same(got, want, n, rounded=True):
    """`close` of the other tests where the formula is finite; its infinities and NaN elsewhere."""
    want, s = want
    got = got.double()
    assert got.shape == want.shape and torch.equal(got.isnan(), want.isnan())
    inf = want.isinf()
    assert torch.equal(got[inf], want[inf])
    fine = want.isfinite()
    tol = (2.0 ** -8 * want.abs() + 2.0 ** -16 * s if rounded else 0.0) + n * 2.0 ** -22 * s
    assert bool(((got - want).abs()[fine] <= tol[fine]).all())


def case(t, n, r, k, m, ranks=None, seed=0):
    c = Case(t, n, r, k, m, seed=seed, ranks=ranks, index=[i % (n + 1) - 1 for i in range(t)])
    c.a.abs_().add_(2.0 ** -10)
    c.b.abs_().add_(2.0 ** -10)
    return c


# few tokens (passes of 16 and of 32 rows) and tiles; ranks that fill their sixteenths and ranks that do not; rows at
# 16-byte boundaries and at others
SHAPES = [(5, 3), (16, 2), (30, 1), (400, 2), (1000, 3)]
RANKS = [(1, None), (5, None), (16, None), (24, None), (48, None), (72, None), (100, None), (40, [0, 9, 40])]


@pytest.mark.parametrize("k,m", [(256, 136), (201, 131)])
@pytest.mark.parametrize("r,ranks", RANKS, ids=[str(r) if q is None else "own" for r, q in RANKS])
@pytest.mark.parametrize("t,n", SHAPES)
def test_infinite_rows_forward(t, n, r, ranks, k, m):
    c = case(t, n, r, k, m, ranks and ranks[:n], seed=r)
    c.x[1 % t, 7], c.x[t // 2, 0], c.x[t - 1, k - 1] = math.inf, -math.inf, math.nan
    out, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    want = c.exact()
    same(out, want[0], c.k + 2 * c.r)
    same(xa, want[1], c.k, rounded=False)
    if ranks is None:  # an infinity came through
        assert bool(out.isinf().any()) == bool((c.index[[1 % t, t // 2]] >= 0).any())


@pytest.mark.parametrize("k,m", [(256, 136), (201, 131)])
@pytest.mark.parametrize("r,ranks", RANKS, ids=[str(r) if q is None else "own" for r, q in RANKS])
@pytest.mark.parametrize("t,n", SHAPES)
def test_infinite_gradient_rows(t, n, r, ranks, k, m):
    """dx and da (an infinity in dy reaches all of its token's adapter)."""
    c = case(t, n, r, k, m, ranks and ranks[:n], seed=r)
    _, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    c.dy[t // 3, 5] = math.inf
    dx, da, _ = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    want = c.exact(back=True)
    same(dx, want[0], c.m + 2 * c.r)
    same(da, want[1], c.m + 2 * c.t)


def test_an_infinite_scale():
    for t, n, r in ((6, 2, 24), (300, 2, 24), (300, 2, 72)):
        c = case(t, n, r, 128, 64)
        c.scale[0] = math.inf
        out = adapter_apply(c.x.abs_(), c.bank, c.plan, c.y)
        same(out, c.exact()[0], c.k + 2 * c.r)
        assert bool(out[c.index == 0].isinf().all()) and bool(out[c.index != 0].isfinite().all())


@pytest.mark.parametrize("k,m", [(256, 136), (201, 131)])
@pytest.mark.parametrize("r,ranks", RANKS, ids=[str(r) if q is None else "own" for r, q in RANKS])
@pytest.mark.parametrize("t,n", SHAPES)
def test_infinities_against_finite_values_in_the_banks_gradients(t, n, r, ranks, k, m):
    """da where x is infinite, db where dy is: the finite factor is carried in two parts, which may have opposite
    signs.  (One adapter has both kinds of tokens where the batch is large enough.)"""
    c = case(t, n, r, k, m, ranks and ranks[:n], seed=r + 1)
    _, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    rows = (c.index >= 0).nonzero()[:, 0]
    c.x[rows[0], 3], c.x[rows[-1], k - 1] = math.inf, -math.inf
    c.dy[rows[len(rows) // 2], 11] = math.inf
    _, da, db = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    want = c.exact(back=True)
    same(da, want[1], c.m + 2 * c.t)
    # x's infinities came after the forward pass: db is that of the x of then
    c.x[rows[0], 3], c.x[rows[-1], k - 1] = 0.5, 0.25
    _, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    _, da, db = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    want = c.exact(back=True)
    same(da, want[1], c.m + 2 * c.t)
    same(db, want[2], c.k + 2 * c.t)
