"""Low-rank adapters of many requests, against the formulas in 64 bits.

Tolerances.  Every result is one BF16 rounding (at most 2^-8 of the value)
beside the error of what is rounded.  With S the same formula on absolute
values: the narrow product is carried as hi + lo, two BF16, which leaves at
most 2^-16 of it; float32 sums of n products, in the tensor cores' order, are
off by at most n * 2^-22 of S (2^-23 a step for sums that are cut off instead
of rounded, twice over for the two products in a row).  So the bound is
2^-8 |want| + (2^-16 + n * 2^-22) S with n all the inner dimensions together;
the kept x A^T has float32 sums alone.
"""
import math
import random

import numpy as np
import pytest
import torch

from lossless_bf16_tensor_gb300 import binding as B
from lossless_bf16_tensor_gb300 import synth
from lossless_bf16_tensor_gb300.activations import compressed_activations
from lossless_bf16_tensor_gb300.adapters import (AdapterBank, AdapterPlan, adapter_apply, adapter_grads,
                                                 adapter_linear, adapter_plan)
from lossless_bf16_tensor_gb300.grads import clip_grads
from lossless_bf16_tensor_gb300.matmul import compressed_linear

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def rnd(gen, *shape, scale=1.0):
    return (torch.randn(*shape, generator=gen, device="cuda") * scale).to(BF)


class Case:
    """Inputs of one call; index is drawn from -1 .. n - 1, or given."""

    def __init__(self, t, n, r, k, m, seed=0, ranks=None, index=None):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = random.Random(seed)
        if index is None:
            index = [rng.randint(-1, n - 1) for _ in range(t)]
        self.index = torch.tensor(index, dtype=torch.int32, device="cuda")
        self.x, self.y = rnd(gen, t, k), rnd(gen, t, m)
        self.dy, self.dx = rnd(gen, t, m, scale=0.1), rnd(gen, t, k, scale=0.1)
        self.a, self.b = rnd(gen, n, r, k, scale=1 / math.sqrt(k)), rnd(gen, n, m, r, scale=0.1)
        self.scale = torch.rand(n, generator=gen, device="cuda") + 0.5
        self.ranks = None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device="cuda")
        self.bank = AdapterBank(self.a, self.b, self.scale, self.ranks)
        self.plan = adapter_plan(self.index, n)
        self.t, self.n, self.r, self.k, self.m = t, n, r, k, m

    def exact(self, back=False):
        """[(want, S)] of forward (out, xa) or backward (dx, da, db)."""
        out = []
        for f in (lambda v: v.double(), lambda v: v.double().abs()):
            x, y, dy, dx, s = f(self.x), f(self.y), f(self.dy), f(self.dx), f(self.scale)
            xa = torch.zeros(self.t, self.r, dtype=torch.float64, device="cuda")
            res, ndx = y.clone(), dx.clone()
            da, db = (torch.zeros_like(v, dtype=torch.float64) for v in (self.a, self.b))
            for i in range(self.n):
                u = self.r if self.ranks is None else max(0, min(self.r, int(self.ranks[i])))
                rows = (self.index == i).nonzero()[:, 0]
                if not u or not rows.numel():
                    continue
                a, b = f(self.a[i, :u]), f(self.b[i, :, :u])
                v = x[rows] @ a.t()
                xa[rows, :u] = v
                d = dy[rows] @ b * s[i]
                da[i, :u] = d.t() @ x[rows]
                db[i, :, :u] = dy[rows].t() @ v * s[i]
                res[rows] += v @ b.t() * s[i]
                ndx[rows] += d @ a
            out.append((ndx, da, db) if back else (res, xa))
        return list(zip(*out))


def close(got, want, n, rounded=True):
    want, s = want
    tol = (2.0 ** -8 * want.abs() + 2.0 ** -16 * s if rounded else 0.0) + n * 2.0 ** -22 * s
    bad = ~((got.double() - want).abs() <= tol)
    assert got.shape == want.shape and not bool(bad.any()), \
        "%d of %d values are off, first at %s" % (int(bad.sum()), bad.numel(), bad.nonzero()[0].tolist())


def check_forward(c, got, xa=None):
    want = c.exact()
    close(got, want[0], c.k + 2 * c.r)
    if xa is not None:
        close(xa, want[1], c.k, rounded=False)


def check_backward(c, got):
    want = c.exact(back=True)
    for g, w, n in zip(got, want, (c.m + 2 * c.r, c.m + 2 * c.t, c.k + 2 * c.t)):
        if g is not None:
            assert g.dtype == BF
            close(g, w, n)


def both(c):
    out, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    check_forward(c, out, xa)
    check_backward(c, adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx))
    assert c.plan.status() == 0


# ------------------------------------------------------------------- plan

def plan_of(index, n):
    """The tables from the definition."""
    group = [i if 0 <= i < n else n for i in index]
    order = sorted(range(len(index)), key=lambda t: group[t])
    starts = [sum(g < a for g in group) for a in range(n + 2)]
    tiles = [[a if a < n else -1, f, min(128, starts[a + 1] - f), 0] for a in range(n + 1)
             for f in range(starts[a], starts[a + 1], 128)]
    rows = -(-len(index) // 128) + min(n + 1, len(index)) if index else 1
    assert len(tiles) <= rows
    return order, starts, tiles + [[0, 0, 0, 0]] * (rows - len(tiles))


@pytest.mark.parametrize("t,n,runs", [(1, 1, False), (1, 500, False), (31, 3, False), (33, 3, True), (128, 1, True),
                                      (129, 1, True), (1000, 7, False), (1024, 1025, False), (5000, 64, True),
                                      (20_011, 3, False), (3000, 16_384, False), (700, 2047, True), (4096, 9, True),
                                      (4097, 9, True), (40_000, 5, True), (150_001, 40, False), (9000, 16_384, False)])
def test_plan(t, n, runs):
    rng = random.Random(t * n)
    index = []
    while len(index) < t:
        index += [rng.randint(-1, n - 1)] * (rng.randint(1, 300) if runs else 1)
    index = index[:t]
    p = adapter_plan(torch.tensor(index, dtype=torch.int32, device="cuda"), n)
    order, starts, tiles = plan_of(index, n)
    assert p.order.tolist() == order and p.starts.tolist() == starts and p.tiles.tolist() == tiles


def test_plan_without_tokens_and_with_bad_indices():
    p = adapter_plan(torch.empty(0, dtype=torch.int32, device="cuda"), 3)
    assert p.order.numel() == 0 and p.starts.tolist() == [0] * 5 and p.tiles.tolist() == [[0] * 4]
    index = [0, 3, -2, 1, 2 ** 31 - 1, -2 ** 31, 2]
    p = adapter_plan(torch.tensor(index, dtype=torch.int32, device="cuda"), 3)
    order, starts, _ = plan_of(index, 3)
    assert p.order.tolist() == order and p.starts.tolist() == starts
    assert p.status() == B.LCT_ERR_INVALID_ARG
    c = Case(7, 3, 8, 64, 64, index=index)
    check_forward(c, adapter_apply(c.x, c.bank, c.plan, c.y))  # they count as none


# ------------------------------------------------------- sizes and layouts

@pytest.mark.parametrize("t", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300])
def test_tokens(t):
    both(Case(t, 2, 16, 128, 192, seed=t))


@pytest.mark.parametrize("r", [1, 2, 7, 8, 15, 16, 17, 24, 33, 48, 63, 64, 65, 72, 96, 100, 127, 128])
def test_ranks(r):
    both(Case(150, 2, r, 320, 256, seed=r))


@pytest.mark.parametrize("k,m", [(1, 1), (1, 200), (200, 1), (7, 9), (8, 8), (63, 65), (64, 64), (72, 40), (127, 129),
                                 (1001, 2047), (1000, 2056), (4096, 64), (64, 4096), (2500, 1032), (640, 136)])
@pytest.mark.parametrize("r", [5, 16, 72])
def test_widths(k, m, r):
    both(Case(70, 3, r, k, m, seed=k + m))


@pytest.mark.parametrize("t,n,r,k,m", [(1, 1, 16, 4096, 4096), (5, 5, 8, 2048, 8192), (64, 64, 16, 4096, 1024),
                                       (64, 3, 32, 1024, 4096), (2000, 5, 64, 1024, 1024), (4000, 1, 16, 512, 512),
                                       (700, 130, 4, 256, 512), (3, 1000, 16, 256, 256), (9000, 2, 8, 64, 128)])
def test_batches(t, n, r, k, m):
    both(Case(t, n, r, k, m, seed=t + n))


@pytest.mark.parametrize("r", [3, 16, 31, 64, 128])
@pytest.mark.parametrize("t,n,k,m", [(17, 1, 128, 128), (32, 1, 4096, 4096), (25, 2, 1000, 136), (31, 3, 201, 1031),
                                     (32, 3, 8192, 64), (29, 1, 64, 8192)])
def test_a_batch_of_a_few_adapters(t, n, r, k, m):
    both(Case(t, n, r, k, m, seed=t + r))


@pytest.mark.parametrize("t,n,r,k,m", [(128, 1, 16, 4096, 4096), (300, 3, 64, 8192, 256), (33, 1, 5, 200, 4160),
                                       (500, 1, 64, 4097, 8191), (700, 1, 33, 4096, 1000), (200, 2, 64, 64, 8192)])
def test_wide_batches_of_few_tiles(t, n, r, k, m):
    """One or a few tiles, which the largest clusters share."""
    both(Case(t, n, r, k, m, seed=t + r))


def test_ranks_of_their_own_and_unused_values_are_not_read():
    c = Case(400, 6, 40, 256, 320, ranks=[0, 1, 16, 17, 40, 100], seed=1)
    for i, u in enumerate((0, 1, 16, 17)):
        c.a[i, u:] = math.nan
        c.b[i, :, u:] = math.inf
    both(c)


def test_only_tokens_without_an_adapter():
    c = Case(200, 3, 8, 100, 260, index=[-1] * 200)
    out, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    assert torch.equal(out, c.y) and not bool(xa.any())
    dx, da, db = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    assert torch.equal(dx, c.dx) and not bool(da.any()) and not bool(db.any())
    y = c.y.clone()
    assert adapter_apply(c.x, c.bank, c.plan, y, out=y) is y and torch.equal(y, c.y)


def test_no_tokens():
    c = Case(0, 2, 8, 64, 72, index=[])
    out, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    dx, da, db = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    assert out.shape == (0, 72) and dx.shape == (0, 64) and not bool(da.any()) and not bool(db.any())


def strided(v, ld, lead):
    """v at a row stride of ld values, `lead` values into a buffer."""
    t, cols = v.shape
    buf = torch.full((t * ld + lead + 8,), 7.0, dtype=v.dtype, device="cuda")
    view = buf.as_strided((t, cols), (ld, 1), lead)
    view.copy_(v)
    return buf, view


@pytest.mark.parametrize("extra,lead", [(0, 1), (8, 8), (3, 0), (1, 3), (16, 4)])
@pytest.mark.parametrize("k,m", [(256, 136), (250, 131)])
def test_strides(extra, lead, k, m):
    c = Case(140, 3, 16, k, m, seed=extra + lead)
    _, x = strided(c.x, k + extra, lead)
    _, y = strided(c.y, m + extra, lead)
    obuf, out = strided(torch.zeros_like(c.y), m + extra + 8, lead)
    keep = obuf.clone()
    got, xa = adapter_apply(x, c.bank, c.plan, y, out=out, keep=True)
    assert got is out
    check_forward(c, out, xa)
    out.fill_(0)
    assert torch.equal(obuf, keep)  # nothing else was written
    _, dy = strided(c.dy, m + extra, lead)
    _, dx = strided(c.dx, k + extra, lead)
    nbuf, new = strided(torch.zeros_like(c.dx), k + extra + 8, lead)
    keep = nbuf.clone()
    check_backward(c, adapter_grads(dy, x, xa, c.bank, c.plan, dx, out=new))
    new.fill_(0)
    assert torch.equal(nbuf, keep)


def test_slices_of_one_buffer():
    """x, y and out as column slices of the same rows."""
    c = Case(90, 2, 16, 128, 64, seed=4)
    buf = torch.cat([c.x, c.y, torch.zeros_like(c.y)], 1).contiguous()
    x, y, out = buf[:, :128], buf[:, 128:192], buf[:, 192:]
    adapter_apply(x, c.bank, c.plan, y, out=out)
    check_forward(c, out)
    assert torch.equal(x, c.x) and torch.equal(y, c.y)


@pytest.mark.parametrize("t,n,r,k,m", [(300, 2, 64, 1001, 2047), (500, 3, 128, 513, 257), (260, 2, 33, 2050, 1026),
                                       (20, 9, 7, 131, 129), (1500, 1, 16, 4097, 65), (400, 2, 100, 64, 1031)])
def test_slices_and_in_place_at_odd_widths(t, n, r, k, m):
    """Rows of x, y, dy and dx one after another in one buffer: pieces that hold the end of one and the start of the
    next; the results in place."""
    c = Case(t, n, r, k, m, seed=k)
    buf = torch.cat([c.x, c.y, c.dy, c.dx], 1).contiguous()
    x, y, dy, dx = buf.split([k, m, m, k], 1)
    _, xa = adapter_apply(x, c.bank, c.plan, y, out=y, keep=True)
    check_forward(c, y, xa)
    assert torch.equal(x, c.x) and torch.equal(dy, c.dy) and torch.equal(dx, c.dx)
    new, da, db = adapter_grads(dy, x, xa, c.bank, c.plan, dx, out=dx)
    check_backward(c, (dx, da, db))
    assert new is dx and torch.equal(x, c.x) and torch.equal(dy, c.dy)
    check_forward(c, y)


def test_in_place_and_more_dimensions():
    c = Case(60, 2, 16, 128, 192, seed=5)
    want, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    y = c.y.clone().view(3, 20, 192)
    got = adapter_apply(c.x.view(3, 20, 128), c.bank, c.plan, y, out=y)
    assert got is y and torch.equal(y.view(60, 192), want)
    new = adapter_apply(c.x.view(3, 20, 128), c.bank, c.plan, c.y.view(3, 20, 192))
    assert new.shape == (3, 20, 192) and torch.equal(new.view(60, 192), want)
    ref = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    dx = c.dx.clone()
    got = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, dx, out=dx)
    assert got[0] is dx and all(torch.equal(a, b) for a, b in zip(got, ref))
    got = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, None)
    assert got[0] is None and all(torch.equal(a, b) for a, b in zip(got[1:], ref[1:]))


def test_offsets_past_32_bits():
    """Rows 2^22 values apart: the last one lies 9 GB into the buffer."""
    c = Case(1100, 2, 16, 128, 64, seed=6)
    far = 1 << 22
    buf = torch.empty(1099 * far + 256, dtype=BF, device="cuda")
    x, y = buf.as_strided((1100, 128), (far, 1)), buf.as_strided((1100, 64), (far, 1), 128)
    out = buf.as_strided((1100, 64), (far, 1), 192)
    x.copy_(c.x)
    y.copy_(c.y)
    _, xa = adapter_apply(x, c.bank, c.plan, y, out=out, keep=True)
    check_forward(c, out, xa)
    y.copy_(c.dy)
    check_backward(c, adapter_grads(y, x, xa, c.bank, c.plan, c.dx))


# -------------------------------------------------------- values and order

def test_a_row_that_is_not_finite_stays_alone():
    c = Case(200, 2, 24, 256, 136, seed=7)
    clean = adapter_apply(c.x, c.bank, c.plan, c.y)
    for row, bad in ((3, math.nan), (77, math.inf), (150, -math.inf)):
        c.x[row, 5] = bad
    out = adapter_apply(c.x, c.bank, c.plan, c.y)
    rows = torch.ones(200, dtype=torch.bool)
    rows[[3, 77, 150]] = False
    assert torch.equal(out[rows], clean[rows])
    mine = (c.index[[3, 77, 150]] >= 0).tolist()
    for row, has in zip((3, 77, 150), mine):
        assert bool((~out[row].isfinite()).all()) == has


def test_gradient_rows_that_are_not_finite():
    c = Case(150, 3, 16, 128, 64, index=[t % 3 for t in range(150)], seed=8)
    _, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    ref = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    c.dy[31, 7] = math.nan  # a token of adapter 1
    dx, da, db = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    assert bool(dx[31].isnan().all()) and bool(da[1].isnan().all()) and bool(db[1, 7].isnan().all())
    keep = torch.arange(150, device="cuda") != 31
    assert torch.equal(dx[keep], ref[0][keep])
    for i in (0, 2):
        assert torch.equal(da[i], ref[1][i]) and torch.equal(db[i], ref[2][i])
    assert torch.equal(db[1, :7], ref[2][1, :7]) and torch.equal(db[1, 8:], ref[2][1, 8:])


def test_large_and_small_values():
    c = Case(100, 2, 16, 256, 128, seed=9)
    c.x.mul_(2.0 ** 40)
    c.a.mul_(2.0 ** -60)
    c.b.mul_(2.0 ** 20)
    both(c)


def test_same_result_every_time_and_for_every_order_of_adapters():
    c = Case(1000, 4, 32, 512, 512, seed=10)
    out, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    grads = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    for _ in range(3):
        o2, xa2 = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
        assert torch.equal(out, o2) and torch.equal(xa, xa2)
        assert all(torch.equal(a, b) for a, b in zip(grads, adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)))


def test_on_another_stream_and_in_a_graph():
    c = Case(300, 3, 16, 256, 256, seed=11)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        out, xa = adapter_apply(c.x, c.bank, adapter_plan(c.index, 3), c.y, keep=True)
        grads = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx)
    s.synchronize()
    check_forward(c, out, xa)
    check_backward(c, grads)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan = adapter_plan(c.index, 3)
        out, xa = adapter_apply(c.x, c.bank, plan, c.y, keep=True)
        grads = adapter_grads(c.dy, c.x, xa, c.bank, plan, c.dx)
    c.index.copy_(c.index.flip(0))
    c.x.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    check_forward(c, out, xa)
    check_backward(c, grads)


# ------------------------------------------------------------- differences

def test_gradients_against_differences():
    """L = sum(dy * out) is linear in A, in B and in x alone, so a difference of
    two passes over any distance is its slope.  Along E = sign of the gradient
    the slope is the gradient's sum of absolutes.  Both passes' rounding is at
    most 2^-8 |out| a value (weighed with |dy|), the gradient's 2^-8 of itself,
    and E is exact in BF16 where it is added with exact sums (multiples of
    2^-10 at magnitudes below 2^-3)."""
    c = Case(260, 2, 16, 128, 96, seed=12)
    grid = 2.0 ** -10

    def snap(v):
        v.copy_((v.float() / grid).round().clamp(-100, 100) * grid)
    snap(c.a), snap(c.b), snap(c.x)
    c.y.zero_()
    _, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    dx, da, db = adapter_grads(c.dy, c.x, xa, c.bank, c.plan, torch.zeros_like(c.dx))
    dy = c.dy.double()
    for v, g in ((c.a, da), (c.b, db), (c.x, dx)):
        e = torch.sign(g.float()) * grid * 16
        before = v.clone()
        sides = []
        for sign in (1, -1):
            v.copy_((before.float() + sign * e).to(BF))
            assert torch.equal(v.float(), before.float() + sign * e)
            sides.append(adapter_apply(c.x, c.bank, c.plan, c.y).double())
        v.copy_(before)
        slope = float((dy * (sides[0] - sides[1])).sum()) / 2
        want = float((g.double() * e.double()).sum())
        tol = 2.0 ** -8 * (float((dy.abs() * (sides[0].abs() + sides[1].abs())).sum()) / 2 + abs(want))
        assert abs(slope - want) <= 1.01 * tol and abs(want) > 2 * tol


# -------------------------------------------------- beside the shared weight

def compressed_weight(n, k, seed):
    bits = synth.normal(n * k, 0.02, seed)
    cb = B.lct_codebook_build("gaussian", 0.02)
    w = B.CompressedTensor(n * k, "CLEAN")
    dense = torch.from_numpy(bits.view(np.int16)).cuda()
    B.lct_encode(dense, cb, w)
    return w, cb, dense.view(BF).view(n, k)


def test_adapter_linear_and_its_gradients():
    n, k = 512, 256
    w, cb, dense = compressed_weight(n, k, 21)
    c = Case(300, 3, 16, k, n, seed=13)
    x = c.x.view(3, 100, k).clone().requires_grad_(True)
    a, b = torch.nn.Parameter(c.a), torch.nn.Parameter(c.b)
    y = adapter_linear(x, w, cb, AdapterBank(a, b, c.scale), c.plan)
    c.y = compressed_linear(c.x, w, cb, n, k)
    check_forward(c, y.detach().view(300, n))
    y.backward(c.dy.view(3, 100, n))
    c.dx = c.dy @ dense
    check_backward(c, (x.grad.view(300, k), a.grad, b.grad))
    with torch.no_grad():
        served = adapter_linear(c.x, w, cb, AdapterBank(a, b, c.scale), c.plan)
    assert torch.equal(served, y.detach().view(300, n))


def test_saved_activations_kept_compressed_change_nothing():
    n, k = 256, 512
    w, cb, _ = compressed_weight(n, k, 22)
    acts = B.lct_codebook_build("gaussian", 1.0)
    c = Case(600, 2, 8, k, n, seed=14)
    grads = []
    for hook in (None, compressed_activations(acts, level="MEDIUM")):
        x = c.x.clone().requires_grad_(True)
        a, b = torch.nn.Parameter(c.a.clone()), torch.nn.Parameter(c.b.clone())
        bank = AdapterBank(a, b, c.scale)
        if hook is None:
            y = adapter_linear(x * 1.0, w, cb, bank, c.plan)
        else:
            with hook:
                y = adapter_linear(x * 1.0, w, cb, bank, c.plan)
        (y.float() ** 2).sum().backward()
        grads.append((x.grad, a.grad, b.grad))
    assert all(torch.equal(p, q) for p, q in zip(*grads)) and hook.stats["compressed"] >= 1


def test_a_step_on_compressed_adapter_weights():
    """Backward, clipping by the global norm, and the fused AdamW step on the
    adapters' compressed weights lower the loss."""
    n, k, r = 512, 256, 16
    w, cb, _ = compressed_weight(n, k, 23)
    c = Case(256, 2, r, k, n, index=[t % 2 for t in range(256)], seed=15)
    target = torch.zeros_like(c.y)
    cbs = [B.lct_codebook_build("gaussian", s) for s in (0.05, 1e-3)]
    state = []
    for p in (c.a, c.b):
        packed = [B.CompressedTensor(p.numel(), "MEDIUM") for _ in range(3)]
        for t, v, book in zip(packed, (p, torch.zeros_like(p), torch.zeros_like(p)), (cbs[0], cbs[1], cbs[1])):
            B.lct_encode(v.view(torch.int16).view(-1), book, t)
        state.append(packed)
    losses = []
    a, b = torch.nn.Parameter(c.a), torch.nn.Parameter(c.b)
    for step in range(1, 7):
        y = adapter_linear(c.x, w, cb, AdapterBank(a, b, c.scale), c.plan)
        loss = (y.float() - target.float()).square().mean()
        losses.append(loss.item())
        a.grad = b.grad = None
        loss.backward()
        clip_grads([a.grad, b.grad], 0.05)
        for p, packed in zip((a, b), state):
            new = [B.CompressedTensor(p.numel(), "MEDIUM") for _ in range(3)]
            B.lct_adamw_step_fused(packed[0], cbs[0], packed[1], cbs[1], packed[2], cbs[1],
                                   p.grad.view(torch.int16).view(-1), 3e-3, 0.9, 0.99, 1e-8, 0.0, step, *new)
            packed[:] = new
            B.lct_decode(new[0], cbs[0], p.data.view(torch.int16).view(-1))
            assert all(t.state().status == 0 for t in new)
    assert all(q < p for p, q in zip(losses, losses[1:]))


# ---------------------------------------------------------------- refusals

def test_refusals():
    c = Case(20, 2, 8, 64, 72, seed=16)
    ok = lambda **kw: adapter_apply(**{**dict(x=c.x, bank=c.bank, plan=c.plan, y=c.y), **kw})  # noqa: E731
    for kw in (dict(x=c.x.float()), dict(x=c.x.cpu()), dict(x=c.x[:, :60]), dict(x=c.x[:19]), dict(y=c.y[:, :64]),
               dict(x=c.x.t().contiguous().t()), dict(out=torch.empty(20, 72, device="cuda")),
               dict(out=torch.empty(1, 72, dtype=BF, device="cuda").expand(20, 72)),
               dict(plan=adapter_plan(c.index, 3))):
        with pytest.raises((ValueError, RuntimeError)):
            ok(**kw)
    buf = torch.zeros(21 * 72, dtype=BF, device="cuda")
    with pytest.raises(B.LctError):
        ok(y=buf[:1440].view(20, 72), out=buf[72:].view(20, 72))  # out one row into y
    with pytest.raises(B.LctError):
        adapter_apply(buf[:1280].view(20, 64), c.bank, c.plan, c.y, out=buf[:1440].view(20, 72))
    with pytest.raises(B.LctError):
        big = AdapterBank(torch.zeros(2, 129, 64, dtype=BF, device="cuda"),
                          torch.zeros(2, 72, 129, dtype=BF, device="cuda"), c.scale)
        ok(bank=big)
    for bad in (dict(a=c.a.float()), dict(a=c.a[:1]), dict(scale=c.scale.double()), dict(a=c.a[:, :, :63]),
                dict(b=c.b.transpose(1, 2)), dict(ranks=torch.zeros(2, device="cuda")), dict(scale=c.scale.cpu())):
        with pytest.raises(ValueError):
            AdapterBank(**{**dict(a=c.a, b=c.b, scale=c.scale), **bad})
    for index, n in ((c.index.long(), 2), (c.index.cpu(), 2), (c.index[::2], 2)):
        with pytest.raises(ValueError):
            adapter_plan(index, n)
    for n in (0, -1, 16_385):
        with pytest.raises(B.LctError):
            adapter_plan(c.index, n)
    with pytest.raises(ValueError):
        AdapterPlan(c.plan.order, c.plan.starts, c.plan.tiles[:1])
    _, xa = ok(keep=True)
    for kw in (dict(xa=xa[:, :7]), dict(xa=xa.double()), dict(dy=c.dy[:, :64]), dict(dx=c.dx.float())):
        with pytest.raises((ValueError, RuntimeError)):
            adapter_grads(**{**dict(dy=c.dy, x=c.x, xa=xa, bank=c.bank, plan=c.plan, dx=c.dx), **kw})
    with pytest.raises(B.LctError):
        adapter_grads(c.dy, c.x, xa, c.bank, c.plan, c.dx, out=c.x)


@pytest.mark.parametrize("what", ["order", "tiles", "starts"])
@pytest.mark.parametrize("t,n", [(40, 40), (300, 2)])
def test_tables_that_are_not_a_plan(what, t, n):
    """Entries out of range reach nothing; the plan says so where it shows."""
    c = Case(t, n, 16, 128, 128, index=[i % n for i in range(t)], seed=17)
    _, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    bad = AdapterPlan(c.plan.order.clone(), c.plan.starts.clone(), c.plan.tiles.clone())
    if what == "order":
        bad.order[3::7] = 2 ** 31 - 1
        bad.order[5::7] = -4
    elif what == "tiles":
        bad.tiles[1, 1] = t - 1
        bad.tiles[1, 2] = 100_000
    else:
        bad.starts[1] = -5
        bad.starts[2:] = 2 ** 30
    out = adapter_apply(c.x, c.bank, bad, c.y)
    grads = adapter_grads(c.dy, c.x, xa, c.bank, bad, c.dx)
    torch.cuda.synchronize()
    assert out.shape == c.y.shape and grads[0].shape == c.dx.shape
    if what != "starts":
        assert bad.status() == B.LCT_ERR_CORRUPT
    check_forward(c, adapter_apply(c.x, c.bank, c.plan, c.y))
    assert c.plan.status() == 0


@pytest.mark.parametrize("t,n", [(1, 9), (3, 200), (30, 31), (90, 700), (400, 1000)])
def test_more_adapters_than_tokens(t, n):
    rng = random.Random(t)
    both(Case(t, n, 8, 128, 136, seed=t, index=[rng.choice([-1, 0, n - 1, rng.randint(0, n - 1)]) for _ in range(t)]))


@pytest.mark.parametrize("r", [16, 40, 80])
@pytest.mark.parametrize("k,m", [(512, 768), (1000, 264)])
def test_runs_of_consecutive_tokens(r, k, m):
    """Runs longer and shorter than the boxes that they are loaded by."""
    index = [0] * 200 + [1] * 33 + [-1] * 70 + [0] * 95 + [2] * 1 + [1] * 300 + [0] * 7 + [2] * 128 + [-1] * 3
    both(Case(len(index), 3, r, k, m, seed=r + k, index=index))


def test_many_tiles_a_block():
    """More tiles than blocks fit on the GPU: blocks go on to further ones."""
    both(Case(30_000, 2, 8, 64, 72, seed=18, index=[(i // 70) % 2 for i in range(30_000)]))
    both(Case(26_000, 3, 72, 72, 64, seed=19, index=[i % 4 - 1 for i in range(26_000)]))
