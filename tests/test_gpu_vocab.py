"""The lookup of tokens' rows, its gradient, and the cross entropy of a projection
onto the vocabulary with its gradients, against their formulas in 64 bits.

Bounds: a rounding to a type is off by at most finfo(type).eps / 2 of the value.
A product of k terms adds 16 at a time in float32: k / 16 sums, each off by at
most 2^-23 of the terms' absolute sum, and as much again for 16 terms that are
aligned to the largest.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def vocab():
    from lossless_bf16_tensor_gb300 import vocab
    return vocab


def half(dtype):
    return torch.finfo(dtype).eps / 2


def generator(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def make_ids(t, v, gen, none=0.0, dtype=torch.int64):
    ids = (torch.exp(torch.rand(t, generator=gen, device="cuda", dtype=torch.float64) * math.log(v + 1)) - 1).long()
    ids = ids.clamp(0, v - 1)
    if none:
        ids[torch.rand(t, generator=gen, device="cuda") < none] = -100
    return ids.to(dtype)


# ------------------------------------------------------------------ lookup

@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("t,v,k", [(1, 1, 1), (1, 1000, 4096), (3, 7, 8), (65, 300, 1001), (5000, 513, 264), (40, 50, 5000)])
def test_lookup(vocab, t, v, k, dtype):
    gen = generator(t * v + k)
    table = torch.randn(v, k, generator=gen, device="cuda").to(dtype)
    for scale in (1.0, 31.7):
        for kind in (torch.int32, torch.int64):
            ids = make_ids(t, v, gen, 0.2, kind)
            want = (table.float() * scale).to(dtype)[ids.long().clamp(min=0)]
            want[ids < 0] = 0
            assert torch.equal(vocab.embedding(ids, table, scale), want)


def test_lookup_shapes_strides_and_impossible_ids(vocab):
    gen = generator(1)
    wide = torch.randn(50, 130, generator=gen, device="cuda").to(BF16)
    table = wide[:, 1:129]                                       # rows at odd addresses
    ids = make_ids(24, 50, gen).view(2, 3, 4)
    assert torch.equal(vocab.embedding(ids, table), table[ids])
    assert torch.equal(vocab.embedding(ids.transpose(0, 1), table), table[ids.transpose(0, 1)])
    out = torch.full((2, 3, 4, 200), 7.0, device="cuda", dtype=BF16)
    assert vocab.embedding(ids, table, out=out[..., 8:136]).data_ptr() == out[..., 8:136].data_ptr()
    assert torch.equal(out[..., 8:136], table[ids]) and (out[..., :8] == 7).all() and (out[..., 136:] == 7).all()
    bad = torch.tensor([-1, 0, 49, 50, 2 ** 40, -2 ** 40], device="cuda")
    got = vocab.embedding(bad, table)
    assert (got[0] == 0).all() and (got[5] == 0).all() and got[3:5].isnan().all() and torch.equal(got[1:3], table[[0, 49]])
    assert vocab.embedding(bad[:0], table).shape == (0, 128)


# ---------------------------------------------------------------- gradient

def grad_bound(dy, ids, v, scale, base):
    """The gradient in 64 bits, and how far it may be off."""
    some = ids >= 0
    some &= ids < v
    rows = dy.double()[some]
    want = torch.zeros(v, dy.shape[-1], dtype=torch.float64, device="cuda")
    mass, count = want.clone(), torch.zeros(v, dtype=torch.float64, device="cuda")
    want.index_add_(0, ids[some].long(), rows)
    mass.index_add_(0, ids[some].long(), rows.abs())
    count.index_add_(0, ids[some].long(), torch.ones(rows.shape[0], dtype=torch.float64, device="cuda"))
    want = want * scale + (0 if base is None else base.double())
    off = (count[:, None] + 2) * 2.0 ** -24 * (mass * abs(scale) + (0 if base is None else base.double().abs()))
    return want, off * (1 + half(dy.dtype)) + half(dy.dtype) * want.abs() + 1e-40


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("t,v,k,none", [(1, 1, 1, 0.0), (1, 5000, 64, 0.0), (31, 3, 8, 0.0), (32, 1, 520, 0.0), (33, 1, 520, 0.0),
                                        (64, 64, 1001, 0.3), (4097, 700, 136, 0.1), (5000, 100_000, 40, 0.0),
                                        (20_000, 2, 2056, 0.0), (9000, 300_000, 17, 0.5), (700, 9, 24, 1.0)])
def test_lookup_gradient(vocab, t, v, k, none, dtype):
    gen = generator(t + v + k)
    ids = make_ids(t, v, gen, none, torch.int32 if t % 2 else torch.int64)
    dy = torch.randn(t, k, generator=gen, device="cuda").to(dtype)
    base = torch.randn(v, k, generator=gen, device="cuda").to(dtype)
    for scale, b in ((1.0, None), (-3.3, base)):
        want, off = grad_bound(dy, ids, v, scale, b)
        got = vocab.embedding_grad(dy, ids, v, scale, base=b)
        assert ((got.double() - want).abs() <= off).all()
        if b is not None:
            again = b.clone()
            assert vocab.embedding_grad(dy, ids, v, scale, base=again, out=again) is again
            assert torch.equal(again, got)


@pytest.mark.parametrize("t,v,k", [(3, 200_000, 40), (500, 131_072, 64), (5000, 131_072, 256), (20_000, 900_000, 63), (1, 9000, 1001)])
def test_lookup_gradient_of_tables_too_large_to_write_while_ids_are_sorted(vocab, t, v, k):
    """Short and long rows that are left to the blocks beside the sums."""
    gen = generator(t + v)
    ids = make_ids(t, v, gen, 0.1 if t > 1 else 0.0)
    ids[0] = v - 1
    dy = torch.randn(t, k, generator=gen, device="cuda").to(BF16)
    base = torch.randn(v, k, generator=gen, device="cuda").to(BF16)
    for scale, b in ((1.0, None), (-3.3, base)):
        got = vocab.embedding_grad(dy, ids, v, scale, base=b)
        there = torch.zeros(v, dtype=torch.bool, device="cuda")
        there[ids[ids >= 0]] = True
        assert torch.equal(got[~there], b[~there] if b is not None else torch.zeros_like(got[~there]))
        rows = there.nonzero()[:, 0]
        place = torch.where(ids < 0, -1, torch.searchsorted(rows, ids.clamp(min=0)))
        want, off = grad_bound(dy, place, len(rows), scale, b[rows] if b is not None else None)
        assert ((got[rows].double() - want).abs() <= off).all()


def test_lookup_gradient_keeps_its_bits_and_what_is_around(vocab):
    gen = generator(3)
    t, v, k = 3000, 40, 96
    ids = make_ids(t, v, gen, 0.1)
    ids[5], ids[6] = v, 2 ** 33                                   # impossible: they add nothing
    dy = torch.randn(t, 200, generator=gen, device="cuda").to(BF16)[:, 3:99]
    out = torch.full((v + 2, 128), 5.0, device="cuda", dtype=BF16)
    got = vocab.embedding_grad(dy, ids, v, out=out[1:-1, 16:112])
    want, off = grad_bound(dy, ids, v, 1.0, None)
    assert ((got.double() - want).abs() <= off).all()
    assert (out[0] == 5).all() and (out[-1] == 5).all() and (out[:, :16] == 5).all() and (out[:, 112:] == 5).all()
    for _ in range(3):
        assert torch.equal(vocab.embedding_grad(dy, ids, v), got)
    inf = dy.clone()
    inf[ids == 0] = math.inf
    inf[ids < 0] = math.nan                                       # rows without an id reach nothing
    got = vocab.embedding_grad(inf, ids, v)
    assert (got[0] == math.inf).all() and got[1:].isfinite().all()
    assert (vocab.embedding_grad(dy[:0], ids[:0], 3) == 0).all()


def test_lookup_under_autograd(vocab):
    gen = generator(4)
    table = torch.randn(60, 24, generator=gen, device="cuda", requires_grad=True)
    ids = make_ids(50, 60, gen, 0.2).view(5, 10)
    out = vocab.embedding(ids, table, 2.5)
    up = torch.randn(out.shape, generator=gen, device="cuda")
    (got,) = torch.autograd.grad(out, table, up, retain_graph=True)
    want, off = grad_bound(up.view(-1, 24), ids.view(-1), 60, 2.5, None)
    assert ((got.double() - want).abs() <= off).all()
    with pytest.raises(RuntimeError):
        vocab.embedding(ids, table, out=torch.empty_like(out))
    g = up.requires_grad_(True)
    (first,) = torch.autograd.grad(out, table, g, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(first.sum(), g)


# -------------------------------------------------------------------- loss

def loss_case(t, v, k, none=0.0, dtype=torch.int64, seed=0, lean=4.0):
    gen = generator(seed + t + v + k)
    ids = make_ids(t, v, gen, none, dtype)
    w = (torch.randn(v, k, generator=gen, device="cuda") * (2 / math.sqrt(k))).to(BF16)
    x = torch.randn(t, k, generator=gen, device="cuda")
    x += torch.rand(t, 1, generator=gen, device="cuda") * lean * w[ids.long().clamp(0, v - 1)].float()
    c = torch.rand(t, generator=gen, device="cuda") / t
    return x.to(BF16), w, ids, c


def summed(k):
    """How far a product of k terms may be off, as a share of the terms' absolute sum."""
    return (k / 16 + 17) * 2.0 ** -23


def loss_bounds(x, w, ids, c):
    """loss, lse, dx and dW in 64 bits, each with how far it may be off."""
    x, w, c = x.double(), w.double(), c.double()
    t, v, k = x.shape[0], w.shape[0], x.shape[1]
    z, mass = x @ w.t(), x.abs() @ w.abs().t()
    lse = torch.logsumexp(z, 1)
    off_z = summed(k) * mass.amax(1)
    # exponents of base 2 are off by a rounding of their size; 2^-20 for the exponentials and their sums
    off_lse = off_z + 2.0 ** -20 + 2.0 ** -22 * (z.abs().amax(1) + lse.abs())
    have = ids >= 0
    at = ids.long().clamp(min=0)[:, None]
    loss = torch.where(have, lse - z.gather(1, at)[:, 0], 0.0)
    off_loss = off_lse + off_z + 2.0 ** -23 * loss.abs()
    one = torch.zeros_like(z).scatter_(1, at, 1.0)
    p = torch.softmax(z, 1)
    c = torch.where(have, c, 0.0)[:, None]
    rest, mine = p * (1 - one) * c, torch.where(have, torch.expm1(-loss), 0.0)[:, None] * c * one
    off_p = (off_z + off_lse + 2.0 ** -20)[:, None] * rest + half(BF16) * rest
    # expm1(-loss) moves by at most exp(-loss) times the loss's error
    off_mine = (off_loss + 2.0 ** -22)[:, None] * (c * one) + 2.0 ** -22 * mine.abs()
    g, off_g = rest + mine, off_p + off_mine
    dx, dw = g @ w, g.t() @ x
    off_dx = off_g @ w.abs() + (summed(v) + v / 64 * 2.0 ** -23) * (g.abs() @ w.abs())
    off_dw = off_g.t() @ x.abs() + (summed(t) + t * 2.0 ** -23) * (g.abs().t() @ x.abs())
    tiny = 2.0 ** -133  # half of BF16's smallest step
    return ((loss, off_loss), (lse, off_lse), (dx, off_dx + half(BF16) * (dx.abs() + off_dx) + tiny),
            (dw, off_dw + half(BF16) * (dw.abs() + off_dw) + tiny))


def within(got, bound, what):
    want, off = bound
    far = (got.double() - want).abs() - off
    assert (far <= 0).all(), "%s: %g beyond its bound" % (what, float(far.max()))


LOSS_CASES = [(1, 1, 1), (1, 2, 8), (1, 5000, 64), (2, 255, 100), (127, 129, 63), (128, 128, 64), (129, 257, 72), (255, 300, 1001),
              (256, 256, 128), (257, 1000, 200), (300, 70_000, 40), (1000, 513, 2056), (1500, 4000, 96), (33, 3, 4096),
              # few tokens, whose boxes are low
              (8, 1000, 512), (9, 333, 264), (16, 5000, 1024), (32, 700, 2048), (3, 40, 8192), (17, 1024, 8), (31, 15, 64), (1, 16, 4096)]


@pytest.mark.parametrize("t,v,k", LOSS_CASES)
def test_loss_and_gradients(vocab, t, v, k):
    x, w, ids, c = loss_case(t, v, k, 0.2 if t > 2 else 0.0, torch.int32 if t % 2 else torch.int64)
    loss, lse = vocab.cross_entropy(x, w, ids)
    bounds = loss_bounds(x, w, ids, c)
    within(loss, bounds[0], "loss")
    within(lse, bounds[1], "lse")
    dx, dw = vocab.cross_entropy_grads(x, w, ids, loss, lse, c)
    within(dx, bounds[2], "dx")
    within(dw, bounds[3], "dw")
    frozen = vocab.cross_entropy_grads(x, w, ids, loss, lse, c, weight_grad=False)
    assert frozen[1] is None and torch.equal(frozen[0], dx)
    again = vocab.cross_entropy_grads(x, w, ids, loss, lse, c)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("k", [1, 7, 8, 9, 250, 256, 263, 2049, 4100])
def test_rows_at_any_address(vocab, k, dtype):
    """Tables, gradients and bases that begin anywhere, rows any distance apart, and what lies around them."""
    gen = generator(k)
    t, v = 70, 23
    ids = make_ids(t, v, gen, 0.2)
    for i in range(9):
        ld = k + 9 + i
        def view(rows, at):  # noqa: E306
            whole = torch.randn(rows + 2, ld, generator=gen, device="cuda").to(dtype)
            return whole, whole[1:-1, at:at + k]
        _, table = view(v, i)
        whole, out = view(t, (3 * i) % 9)
        before = whole.clone()
        want = (table.float() * 1.7).to(dtype)[ids.clamp(min=0)]
        want[ids < 0] = 0
        vocab.embedding(ids, table, 1.7, out=out)
        assert torch.equal(out, want)
        out.copy_(before[1:-1, (3 * i) % 9:(3 * i) % 9 + k])
        assert torch.equal(whole, before)
        _, dy = view(t, i)
        _, base = view(v, (5 * i) % 9)
        whole, out = view(v, (2 * i) % 9)
        before = whole.clone()
        vocab.embedding_grad(dy, ids, v, 1.7, base=base, out=out)
        want, off = grad_bound(dy, ids, v, 1.7, base)
        assert ((out.double() - want).abs() <= off).all()
        out.copy_(before[1:-1, (2 * i) % 9:(2 * i) % 9 + k])
        assert torch.equal(whole, before)


@pytest.mark.parametrize("t,k", [(1, 4096), (5, 1024), (200, 8192), (300, 4096)])
def test_losses_of_sure_tokens(vocab, t, k):
    """Losses far smaller than their logits are as exact as the logits' differences are, not their roundings."""
    x, w, ids, _ = loss_case(t, 3000, k, seed=30, lean=0.0)
    x = (x.float() * 0.5 + 3.0 * w[ids].float()).to(BF16)
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1) - z.gather(1, ids[:, None])[:, 0]
    assert float(want.median()) < 0.1
    loss, lse = vocab.cross_entropy(x, w, ids)
    # sums of 512 of depth drop at most 2^-23 of their size at each of their steps
    mass = x.double().abs() @ w.double().abs().t()
    part = 512
    off = 2 * (part / 16 + 17 + k / part) * 2.0 ** -23 * mass.amax(1)
    # a loss moves by its own size times what the logits do
    assert ((loss.double() - want).abs() <= off * want + 2.0 ** -21 * want + 2.0 ** -22).all()
