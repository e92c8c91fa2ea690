"""The vocabulary's operators as programs use them: under autograd, on compressed
matrices, on other streams and in graphs, with masked tokens and values that are
not finite, at rows of any address and beyond 32 bits; and waits that run out."""
import ctypes
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_vocab import BF16, generator, grad_bound, half, loss_bounds, loss_case, make_ids, within  # noqa: E402
from test_vocab_abi import Ids  # noqa: E402


@pytest.fixture(scope="module")
def vocab():
    from lossless_bf16_tensor_gb300 import vocab
    return vocab


def compressed(w, level="CLEAN", ovf=None):
    """w [rows, cols] as a CompressedTensor and its codebook."""
    from lossless_bf16_tensor_gb300 import binding as B
    cb = B.lct_codebook_build("gaussian", float(w.float().std()))
    ct = B.CompressedTensor(w.numel(), level, ovf_cap=w.numel())
    B.lct_encode(w.contiguous().view(torch.int16).view(-1), cb, ct)
    torch.cuda.synchronize()
    assert ct.state().status == 0
    return ct, cb


# ---------------------------------------------------------------- autograd

@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_loss_under_autograd(vocab, reduction):
    x, w, ids, _ = loss_case(150, 300, 72, 0.2, seed=1)
    shape = (3, 50)
    leaf, weight = x.view(*shape, 72).clone().requires_grad_(True), torch.nn.Parameter(w.clone())
    loss = vocab.linear_cross_entropy(leaf, weight, ids.view(shape), reduction)
    up = torch.rand(loss.shape, generator=generator(2), device="cuda") + 0.5
    dx, dw = torch.autograd.grad(loss, (leaf, weight), up, retain_graph=True)
    assert dx.shape == leaf.shape and dw.shape == weight.shape
    count = int((ids >= 0).sum())
    c = up.reshape(-1).expand(150) / (count if reduction == "mean" else 1)
    bounds = loss_bounds(x, w, ids, c)
    # the upstream's product with 1 / count is rounded twice on the way
    within(dx.view(150, 72), (bounds[2][0], bounds[2][1] * (1 + 2 ** -20)), "dx")
    within(dw, (bounds[3][0], bounds[3][1] * (1 + 2 ** -20)), "dw")
    each, off = bounds[0]
    if reduction == "none":
        within(loss.view(-1), bounds[0], "loss")
    else:
        n = count if reduction == "mean" else 1
        value = float(loss.detach())
        assert abs(value - float(each.sum() / n)) <= float(off.sum() / n) + 2 ** -23 * abs(value)
    # once more: the graph was kept; only one of the leaves; without gradients
    again = torch.autograd.grad(loss, (leaf, weight), up)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
    frozen = vocab.linear_cross_entropy(leaf, w, ids.view(shape), reduction)
    assert torch.equal(torch.autograd.grad(frozen, leaf, up)[0], dx)
    other = vocab.linear_cross_entropy(x.view(*shape, 72), weight, ids.view(shape), reduction)
    assert torch.equal(torch.autograd.grad(other, weight, up)[0], dw)
    with torch.no_grad():
        assert torch.equal(vocab.linear_cross_entropy(leaf, weight, ids.view(shape), reduction), loss)


def test_loss_gradients_against_differences(vocab):
    """Along a direction: the loss at x + d and x - d in 64 bits, for values that BF16 holds."""
    x, w, ids, _ = loss_case(40, 90, 64, 0.1, seed=3)
    leaf, weight = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss = vocab.linear_cross_entropy(leaf, weight, ids, "sum")
    dx, dw = torch.autograd.grad(loss, (leaf, weight))
    gen = generator(4)

    def at(p, q):
        z = p @ q.t()
        have = ids >= 0
        return (torch.logsumexp(z, 1) - z.gather(1, ids.clamp(min=0)[:, None])[:, 0])[have].sum()

    bounds = loss_bounds(x, w, ids, torch.ones(40, device="cuda"))
    for got, off, which in ((dx, bounds[2][1], 0), (dw, bounds[3][1], 1)):
        d = torch.randn(got.shape, generator=gen, device="cuda", dtype=torch.float64) * 1e-5
        p, q = x.double(), w.double()
        want = float((at(p + d, q) - at(p - d, q)) / 2 if which == 0 else (at(p, q + d) - at(p, q - d)) / 2)
        # the values' errors come with either sign: six times what they add up to on average; differences of 1e-5 are good to 1e-9
        assert abs(float((got.double() * d).sum()) - want) <= 6 * float((off * d).norm()) + 1e-9


def test_operands_at_any_strides(vocab):
    x, w, ids, _ = loss_case(60, 50, 64, 0.1, seed=31)
    want_x, want_w = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    want = vocab.linear_cross_entropy(want_x, want_w, ids)
    grads = torch.autograd.grad(want, (want_x, want_w))
    leaf, weight = x.t().contiguous().requires_grad_(True), w.t().contiguous().requires_grad_(True)
    wide = torch.stack([ids, ids], 1)
    loss = vocab.linear_cross_entropy(leaf.t(), weight.t(), wide[:, 0])
    assert torch.equal(loss.detach(), want.detach())
    got = torch.autograd.grad(loss, (leaf, weight))
    assert torch.equal(got[0].t(), grads[0]) and torch.equal(got[1].t(), grads[1])
    one = x[:1].expand(60, 64).clone()
    rows = x[:1].expand(60, 64)                       # one row in memory
    assert torch.equal(vocab.linear_cross_entropy(rows, w, ids), vocab.linear_cross_entropy(one, w, ids))


def test_saved_tensors_go_through_hooks(vocab):
    """What the loss saves for backward is kept compressed like any other saved tensor; a parameter is not copied."""
    from lossless_bf16_tensor_gb300 import binding as B
    from lossless_bf16_tensor_gb300.activations import compressed_activations
    x, w, ids, _ = loss_case(600, 300, 256, 0.1, seed=32)
    leaf, weight = x.clone().requires_grad_(True), torch.nn.Parameter(w.clone())
    h = leaf * 1.5
    want = torch.autograd.grad(vocab.linear_cross_entropy(h, weight, ids), (leaf, weight), retain_graph=True)
    with compressed_activations(B.lct_codebook_build("gaussian", 2.0)) as kept:
        loss = vocab.linear_cross_entropy(h, weight, ids)
    kept.flush()
    assert kept.stats["compressed"] == 1 and kept.stats["fallback"] == 0
    got = torch.autograd.grad(loss, (leaf, weight))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_second_derivatives_raise(vocab):
    x, w, ids, _ = loss_case(20, 30, 16, seed=5)
    leaf, weight = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss = vocab.linear_cross_entropy(leaf, weight, ids)
    dx, dw = torch.autograd.grad(loss, (leaf, weight), create_graph=True)
    for g, p in ((dx, leaf), (dw, weight)):
        with pytest.raises(RuntimeError):
            torch.autograd.grad(g.float().sum(), p, retain_graph=True)


def test_changed_operands_are_noticed(vocab):
    x, w, ids, _ = loss_case(20, 30, 16, seed=6)
    leaf, weight = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss = vocab.linear_cross_entropy(leaf, weight, ids)
    with torch.no_grad():
        weight.mul_(2)
    with pytest.raises(RuntimeError):
        loss.backward()


def test_refusals(vocab):
    from lossless_bf16_tensor_gb300.binding import LctError
    x, w, ids, c = loss_case(20, 30, 16, seed=7)
    loss, lse = vocab.cross_entropy(x, w, ids)
    for call in (lambda: vocab.cross_entropy(x[:, :8], w, ids), lambda: vocab.cross_entropy(x, w, ids[:5]),
                 lambda: vocab.cross_entropy(x, w, ids.float()), lambda: vocab.cross_entropy(x.t(), w, ids),
                 lambda: vocab.cross_entropy(x, w, ids.cpu()), lambda: vocab.cross_entropy(x.cpu(), w, ids),
                 lambda: vocab.cross_entropy_grads(x, w, ids, loss[:3], lse, c),
                 lambda: vocab.cross_entropy_grads(x, w, ids, loss, lse, c[:3]),
                 lambda: vocab.cross_entropy_grads(x, w, ids, loss, lse, c.double()),
                 lambda: vocab.embedding(ids, w, out=x[:3]), lambda: vocab.embedding_grad(x, ids[:3], 30),
                 lambda: vocab.embedding_grad(x, ids, -1), lambda: vocab.embedding_grad(x, ids, 30, base=w.float()),
                 lambda: vocab.linear_cross_entropy(x, w, ids, "all")):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: vocab.cross_entropy(x.half(), w.half(), ids), lambda: vocab.embedding(ids, w.half()),
                 lambda: vocab.embedding_grad(x.half(), ids, 30), lambda: vocab.embedding(ids, w, out=w[:20]),
                 lambda: vocab.embedding_grad(w[:20], ids, 30, out=w)):
        with pytest.raises(LctError):
            call()
    grown = x.clone().requires_grad_(True)
    for call in (lambda: vocab.cross_entropy(grown, w, ids), lambda: vocab.cross_entropy_grads(grown, w, ids, loss, lse, c),
                 lambda: vocab.embedding_grad(grown, ids, 30)):
        with pytest.raises(RuntimeError):
            call()


# ----------------------------------------------------- masked tokens, infinities

def test_tokens_without_a_target_reach_nothing(vocab):
    x, w, ids, c = loss_case(700, 400, 136, 0.4, seed=8)
    none = ids < 0
    bounds = loss_bounds(x, w, ids, c)
    for junk in (math.nan, math.inf, -math.inf, torch.finfo(BF16).min):
        y = x.clone()
        y[none] = junk
        loss, lse = vocab.cross_entropy(y, w, ids)
        assert (loss[none] == 0).all()
        within(loss[~none], tuple(b[~none] for b in bounds[0]), "loss")
        dloss = torch.where(none, math.nan, c)                    # nor does what stands in their upstream
        dx, dw = vocab.cross_entropy_grads(y, w, ids, loss, lse, dloss)
        within(dx, bounds[2], "dx")
        within(dw, bounds[3], "dw")


@pytest.mark.parametrize("t", [1, 300])
def test_no_targets_at_all(vocab, t):
    x, w, _, _ = loss_case(t, 500, 64, seed=9)
    ids = torch.full((t,), -100, device="cuda")
    leaf, weight = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    loss = vocab.linear_cross_entropy(leaf, weight, ids)
    assert float(loss.detach()) == 0
    dx, dw = torch.autograd.grad(loss, (leaf, weight))
    assert not dx.any() and not dw.any()
    empty = vocab.linear_cross_entropy(x[:0], w, ids[:0])
    assert float(empty) == 0
    loss, lse = vocab.cross_entropy(x[:0], w, ids[:0])
    assert loss.shape == lse.shape == (0,)
    dx, dw = vocab.cross_entropy_grads(x[:0], w, ids[:0], loss, lse, loss)
    assert dx.shape == (0, 64) and not dw.any()


def test_impossible_targets(vocab):
    x, w, ids, c = loss_case(100, 60, 64, seed=10)
    bad = torch.zeros(100, dtype=torch.bool, device="cuda")
    bad[[3, 50]] = True
    wrong = ids.clone()
    wrong[3], wrong[50] = 60, 2 ** 40
    loss, lse = vocab.cross_entropy(x, w, wrong)
    assert loss[bad].isnan().all() and not loss[~bad].isnan().any() and not lse.isnan().any()
    dx, dw = vocab.cross_entropy_grads(x, w, wrong, loss, lse, c)
    assert dx[bad].isnan().all()
    bounds = loss_bounds(x, w, torch.where(bad, -1, ids), c)
    within(dx[~bad], tuple(b[~bad] for b in bounds[2]), "dx")
    within(dw, bounds[3], "dw")
    assert vocab.linear_cross_entropy(x, w, wrong).isnan()


def test_infinities_stay_in_their_rows(vocab):
    x, w, ids, _ = loss_case(300, 200, 64, seed=11)
    y = x.clone()
    y[17] = math.inf
    y[18, 5] = math.nan
    good = torch.ones(300, dtype=torch.bool, device="cuda")
    good[17:19] = False
    loss, lse = vocab.cross_entropy(y, w, ids)
    assert loss[~good].isnan().all() and lse[~good].isnan().all()
    clean, clean_lse = vocab.cross_entropy(x, w, ids)
    assert torch.equal(loss[good], clean[good]) and torch.equal(lse[good], clean_lse[good])


def test_large_and_small_logits(vocab):
    """Logits of thousands: nothing overflows, a sure token has loss 0 and an impossible one its distance."""
    x = torch.zeros(4, 64, device="cuda", dtype=BF16)
    w = torch.zeros(500, 64, device="cuda", dtype=BF16)
    x[:, 0] = torch.tensor([4096.0, -4096.0, 64.0, 0.0], device="cuda").to(BF16)
    w[7, 0], w[9, 0] = 1.0, -1.0
    ids = torch.tensor([7, 7, 9, 7], device="cuda")
    loss, lse = vocab.cross_entropy(x, w, ids)
    want = torch.tensor([0.0, 8192.0, 128.0, math.log(500)], device="cuda")
    assert torch.allclose(loss, want, rtol=2 ** -22, atol=1e-6)
    dx, dw = vocab.cross_entropy_grads(x, w, ids, loss, lse, torch.ones(4, device="cuda"))
    assert dx.isfinite().all() and dw.isfinite().all()
    assert float(dx[0].abs().max()) == 0 and float(dx[1, 0]) == -2.0 and float(dx[2, 0]) == 2.0


# ------------------------------------------------------------------ addresses

@pytest.mark.parametrize("where", ["x", "w", "both", "strided"])
def test_rows_at_any_address(vocab, where):
    x, w, ids, c = loss_case(200, 333, 70 if where == "strided" else 72, 0.2, seed=12)
    k = x.shape[1]
    a, b = torch.randn(201, 160, device="cuda").to(BF16), torch.randn(400, 160, device="cuda").to(BF16)
    xs = a[1:, 3:3 + k] if where in ("x", "both") else a[1:, 8:8 + k] if where == "strided" else x
    ws = b[7:340, 5:5 + k] if where in ("w", "both") else b[7:340, 16:16 + k] if where == "strided" else w
    if xs is not x:
        xs.copy_(x)
    if ws is not w:
        ws.copy_(w)
    bounds = loss_bounds(x, w, ids, c)
    loss, lse = vocab.cross_entropy(xs, ws, ids)
    within(loss, bounds[0], "loss")
    dx, dw = vocab.cross_entropy_grads(xs, ws, ids, loss, lse, c)
    within(dx, bounds[2], "dx")
    within(dw, bounds[3], "dw")


def test_tables_beyond_32_bits(vocab):
    """2.2e9 values: rows at the end of a table, its gradient and its logits."""
    v, k, t = 1_100_000, 2048, 40
    gen = generator(13)
    table = torch.empty(v, k, device="cuda", dtype=BF16)
    for r in range(0, v, 100_000):
        table[r:r + 100_000] = (torch.randn(min(100_000, v - r), k, generator=gen, device="cuda") * 0.02).to(BF16)
    ids = torch.randint(v - 1000, v, (t,), generator=gen, device="cuda")
    rows = vocab.embedding(ids, table)
    assert torch.equal(rows, table[ids])
    grad = vocab.embedding_grad(rows, ids, v)
    want, off = grad_bound(rows, ids - (v - 1000), 1000, 1.0, None)
    assert ((grad[v - 1000:].double() - want).abs() <= off).all() and not grad[:v - 1000:997].any()
    x = (rows.float() * 20).to(BF16)
    loss, lse = vocab.cross_entropy(x, table, ids)
    z = torch.cat([x.float() @ table[r:r + 100_000].float().t() for r in range(0, v, 100_000)], 1).double()
    want = torch.logsumexp(z, 1)
    assert torch.allclose(lse.double(), want, rtol=1e-5, atol=1e-5)
    assert torch.allclose(loss.double(), want - z.gather(1, ids[:, None])[:, 0], rtol=1e-4, atol=1e-4)
    dx, dw = vocab.cross_entropy_grads(x, table, ids, loss, lse, torch.ones(t, device="cuda"))
    p = torch.exp(z - want[:, None])
    p[torch.arange(t), ids] -= 1
    want_dw = p[:, v - 1000:].t() @ x.double()
    assert float((dw[v - 1000:].double() - want_dw).norm()) <= 4e-3 * float(want_dw.norm())
    want_dw = p[:, :1000].t() @ x.double()
    assert float((dw[:1000].double() - want_dw).norm()) <= 6e-3 * float(want_dw.norm())
    want_dx = sum(p[:, r:r + 100_000].float() @ table[r:r + 100_000].float() for r in range(0, v, 100_000))
    assert float((dx.float() - want_dx).norm()) <= 4e-3 * float(want_dx.norm())


# ------------------------------------------------------------ compressed matrices

@pytest.mark.parametrize("rows,cols,tile", [(2048, 64, None), (2048, 64, 1), (3000, 256, 2), (700, 1024, 3)])
def test_compressed_lookup(vocab, rows, cols, tile):
    gen = generator(rows + cols)
    table = (torch.randn(rows, cols, generator=gen, device="cuda") * 0.02).to(BF16)
    ct, cb = compressed(table)
    ids = make_ids(333, rows, gen, 0.2).view(3, 111)
    want = (table.float() * 3.5).to(BF16)[ids.clamp(min=0)]
    want[ids < 0] = 0
    assert torch.equal(vocab.compressed_embedding(ids, ct, cb, rows, cols, 3.5, tile_blocks=tile), want)
    for call in (lambda: vocab.compressed_embedding(ids, ct, cb, rows + 1, cols),
                 lambda: vocab.compressed_cross_entropy(table[:333], ct, cb, rows, 2 * cols, ids.view(-1))):
        with pytest.raises(ValueError):
            call()
    bad = torch.tensor([rows, -1, rows - 1], device="cuda", dtype=torch.int32)
    got = vocab.compressed_embedding(bad, ct, cb, rows, cols, tile_blocks=tile)
    assert got[0].isnan().all() and not got[1].any() and torch.equal(got[2], table[-1])


@pytest.mark.parametrize("rows,cols,tile,t", [(2048, 64, None, 100), (2048, 64, 1, 100), (3000, 256, 2, 300), (700, 1024, 3, 1),
                                              (2560, 512, 1, 600)])
def test_compressed_loss(vocab, rows, cols, tile, t):
    x, w, ids, _ = loss_case(t, rows, cols, 0.2 if t > 1 else 0.0, seed=rows)
    ct, cb = compressed(w)
    count = max(1, int((ids >= 0).sum()))
    c = torch.full((t,), 1.0 / count, device="cuda")
    bounds = loss_bounds(x, w, ids, c)
    leaf = x.clone().requires_grad_(True)
    loss = vocab.compressed_cross_entropy(leaf, ct, cb, rows, cols, ids, tile_blocks=tile)
    want, off = bounds[0]
    value = float(loss.detach())
    assert abs(value - float(want.sum()) / count) <= float(off.sum()) / count + 2 ** -22 * abs(value)
    (dx,) = torch.autograd.grad(loss, leaf)
    within(dx, bounds[2], "dx")
    each = vocab.compressed_cross_entropy(x, ct, cb, rows, cols, ids, "none", tile)
    within(each, bounds[0], "loss")
    total, gx, gw = vocab.compressed_cross_entropy_grads(x, ct, cb, rows, cols, ids, tile)
    assert float(total) == value
    within(gx, bounds[2], "dx")
    within(gw, bounds[3], "dw")
    moved = torch.randn(t, cols + 3, device="cuda").to(BF16)[:, 1:1 + cols]
    moved.copy_(x)
    total, gx, gw = vocab.compressed_cross_entropy_grads(moved, ct, cb, rows, cols, ids, tile)
    within(gx, bounds[2], "dx")
    within(gw, bounds[3], "dw")


def test_a_step_of_a_tied_matrix(vocab):
    """Lookup, loss, both gradients of the one compressed matrix, clipping, and the fused AdamW step on it."""
    from lossless_bf16_tensor_gb300 import binding as B
    from lossless_bf16_tensor_gb300.activations import compressed_activations
    from lossless_bf16_tensor_gb300.grads import clip_grads
    gen = generator(20)
    rows, cols, t = 3000, 512, 700
    w = (torch.randn(rows, cols, generator=gen, device="cuda") * 0.05).to(BF16)
    ct, cb = compressed(w)
    moments = [compressed((torch.rand(rows, cols, generator=gen, device="cuda") * 1e-6).to(BF16)) for _ in range(2)]
    tokens, targets = make_ids(t, rows, gen), make_ids(t, rows, gen, 0.1)
    mix = (torch.randn(cols, cols, generator=gen, device="cuda") / math.sqrt(cols)).to(BF16)
    scale = math.sqrt(cols)

    def body(h, m):
        return torch.tanh(h @ m)

    losses = []
    for step in range(1, 9):
        dense = torch.empty(rows * cols, device="cuda", dtype=BF16)
        B.lct_decode(ct, cb, dense.view(torch.int16))
        dense = dense.view(rows, cols)
        h = vocab.compressed_embedding(tokens, ct, cb, rows, cols, scale, tile_blocks=8).requires_grad_(True)
        with compressed_activations(B.lct_codebook_build("gaussian", 1.0)):
            y = body(h, mix)
        loss, dy, dw = vocab.compressed_cross_entropy_grads(y.detach(), ct, cb, rows, cols, targets, tile_blocks=8)
        (dh,) = torch.autograd.grad(y, h, dy)
        head = dw.clone()
        assert vocab.embedding_grad(dh, tokens, rows, scale, base=dw, out=dw) is dw
        # the lookup's part against its formula
        want, off = grad_bound(dh, tokens, rows, scale, head)
        assert ((dw.double() - want).abs() <= off).all()
        # the whole against torch's own autograd in 32 bits, on the same values
        if step == 1:
            p = dense.float().requires_grad_(True)
            out = torch.nn.functional.cross_entropy(body(p[tokens] * scale, mix.float()) @ p.t(), targets, ignore_index=-100)
            (all_of,) = torch.autograd.grad(out, p)
            assert float((dw.float() - all_of).norm()) <= 2e-2 * float(all_of.norm())
        clip_grads([dw], 1.0)
        # the update is in place; its overflow and scratch are apart
        outs = []
        for one in (ct, moments[0][0], moments[1][0]):
            outs.append(B.CompressedTensor(rows * cols, "CLEAN", ovf_cap=rows * cols))
        B.lct_adamw_step_fused(ct, cb, moments[0][0], moments[0][1], moments[1][0], moments[1][1],
                               dw.view(torch.int16).view(-1), 1e-3, 0.9, 0.99, 1e-8, 0.0, step, *outs)
        torch.cuda.synchronize()
        assert all(o.state().status == 0 for o in outs)
        ct, moments = outs[0], [(outs[1], moments[0][1]), (outs[2], moments[1][1])]
        losses.append(float(loss))
    assert all(math.isfinite(v) for v in losses) and len(set(losses)) > 1


# --------------------------------------------------------------- streams, graphs

def test_other_streams_and_graphs(vocab):
    x, w, ids, c = loss_case(300, 700, 128, 0.2, seed=14)
    table = w.clone()

    def everything():
        loss, lse = vocab.cross_entropy(x, w, ids)
        dx, dw = vocab.cross_entropy_grads(x, w, ids, loss, lse, c)
        h = vocab.embedding(ids, table, 2.0)
        return loss, lse, dx, dw, h, vocab.embedding_grad(dx, ids, 700, 2.0, base=dw)

    want = everything()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = everything()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = everything()
        graphs.append((g, out))
    for _ in range(3):
        for g, out in graphs:
            g.replay()
    torch.cuda.synchronize()
    for g, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    # other inputs in the same places, both graphs at once on two streams
    y, ids2 = loss_case(300, 700, 128, 0.5, seed=15)[0::2]
    x.copy_(y)
    ids.copy_(ids2)
    want = everything()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        graphs[0][0].replay()
    graphs[1][0].replay()
    torch.cuda.synchronize()
    for g, out in graphs:
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_a_captured_training_step(vocab):
    """Forward and backward captured.  (No eager graph of the same leaves may live then: torch's engine would wait for the
    stream that it was made on, which a capture does not allow.  That raises, and the next call works.)"""
    x, w, ids, _ = loss_case(200, 300, 64, 0.1, seed=16)
    leaf, weight = x.clone().requires_grad_(True), w.clone().requires_grad_(True)
    alive = vocab.linear_cross_entropy(leaf, weight, ids)
    want = torch.autograd.grad(alive, (leaf, weight))
    value = alive.detach().clone()
    del alive
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(vocab.linear_cross_entropy(leaf, weight, ids), (leaf, weight))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        loss = vocab.linear_cross_entropy(leaf, weight, ids)
        got = torch.autograd.grad(loss, (leaf, weight))
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(loss.detach(), value) and all(torch.equal(a, b) for a, b in zip(got, want))


def test_two_streams_at_once(vocab):
    """Eager calls of two streams, each with its own products of pairs, in flight together."""
    cases = [loss_case(1000, 9000, 256, 0.2, seed=21), loss_case(700, 12_000, 512, 0.1, seed=22)]

    def everything(x, w, ids, c):
        loss, lse = vocab.cross_entropy(x, w, ids)
        dx, dw = vocab.cross_entropy_grads(x, w, ids, loss, lse, c)
        return loss, lse, dx, vocab.embedding_grad(dx, ids, w.shape[0], 2.0, base=dw)

    want = [everything(*c) for c in cases]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in cases], [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(everything(*cases[i]))
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        assert all(torch.equal(a, b) for g in got[i] for a, b in zip(g, w))


@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_a_loss_that_is_changed_in_place(vocab, reduction):
    """As where gradients accumulate over several batches: the backward pass reads nothing of what the caller owns."""
    x, w, ids, _ = loss_case(90, 200, 64, 0.2, seed=23)
    leaf = x.clone().requires_grad_(True)
    (want,) = torch.autograd.grad((vocab.linear_cross_entropy(leaf, w, ids, reduction) * 0.25).sum(), leaf)
    loss = vocab.linear_cross_entropy(leaf, w, ids, reduction)
    loss *= 0.25
    (got,) = torch.autograd.grad(loss.sum(), leaf)
    assert torch.equal(got, want)


def test_smallest_shapes(vocab):
    from lossless_bf16_tensor_gb300.binding import LctError
    x, w, ids, _ = loss_case(1, 50, 64, seed=24)
    whole = vocab.linear_cross_entropy(x, w, ids)
    leaf = x[0].clone().requires_grad_(True)
    one = vocab.linear_cross_entropy(leaf, w, ids[0])             # a token without a batch
    assert one.shape == () and torch.equal(one.detach(), whole)
    assert torch.autograd.grad(one, leaf)[0].shape == (64,)
    assert vocab.embedding(ids[0], w).shape == (64,)
    none = torch.zeros(0, 5, 64, device="cuda", dtype=BF16, requires_grad=True)
    loss = vocab.linear_cross_entropy(none, w, torch.zeros(0, 5, device="cuda", dtype=torch.long))
    assert float(loss.detach()) == 0 and torch.autograd.grad(loss, none)[0].shape == (0, 5, 64)
    with pytest.raises(LctError):                                 # nothing to project: the C call refuses it
        vocab.cross_entropy(x[:, :0], w[:, :0], ids)
    with pytest.raises(LctError):
        vocab.embedding(ids, w[:, :0])


# ------------------------------------------------------- pieces, long batches

def test_many_tokens_in_several_products(vocab):
    """More tokens than one product of the forward pass takes."""
    x, w, ids, _ = loss_case(40_000, 300, 16, 0.1, seed=17)
    loss, lse = vocab.cross_entropy(x, w, ids)
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1)
    assert torch.allclose(lse.double(), want, rtol=1e-6, atol=1e-5)
    mean = vocab.linear_cross_entropy(x, w, ids)
    each = torch.where(ids < 0, 0.0, want - z.gather(1, ids.clamp(min=0)[:, None])[:, 0])
    assert abs(float(mean) - float(each.sum() / (ids >= 0).sum())) <= 1e-5
    one = torch.ones(1, device="cuda")
    dx, dw = vocab.cross_entropy_grads(x, w, ids, loss, lse, one)
    p = torch.exp(z - want[:, None])
    p[torch.arange(40_000), ids.clamp(min=0)] -= 1
    p[ids < 0] = 0
    for got, ref in ((dx, p @ w.double()), (dw, p.t() @ x.double())):
        assert float((got.double() - ref).norm()) <= 2.5e-3 * float(ref.norm())


# ------------------------------------------------------------- waits that run out

@pytest.mark.parametrize("t,v,k", [(300, 600, 128), (1, 5000, 64), (300, 600, 100)])
def test_waits_that_run_out(vocab, t, v, k):
    from lossless_bf16_tensor_gb300 import binding as B
    x, w, ids, c = loss_case(t, v, k, seed=18)
    loss, lse = vocab.cross_entropy(x, w, ids)
    want = vocab.cross_entropy_grads(x, w, ids, loss, lse, c)
    lib, stream = B.library(), torch.cuda.current_stream().cuda_stream
    P, U = ctypes.c_void_p, ctypes.c_uint64
    arg = Ids(ids.data_ptr(), 1, t, v)
    flags = 4 if k % 8 else 0
    call = lib.lct_debug_loss_forward_timeout
    call.argtypes = [P, P, U, U, P, U, U, U, P, P, P, P, U, P]
    size = vocab.calls.loss_work_bytes(t, v, k, v, flags)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    a, b, total = torch.zeros(t, device="cuda"), torch.zeros(t, device="cuda"), torch.zeros(3, device="cuda")
    assert call(ctypes.addressof(arg), x.data_ptr(), k, k, w.data_ptr(), k, 0, v, a.data_ptr(), b.data_ptr(), total.data_ptr(),
                work.data_ptr(), size, stream) == B.LCT_OK
    torch.cuda.synchronize()
    assert a.isnan().all() and total[:2].isnan().all() and int(work[:4].view(torch.int32)) == B.LCT_ERR_TIMEOUT
    call = lib.lct_debug_loss_backward_timeout
    call.argtypes = [P, P, U, U, P, U, U, U, P, P, P, U, P, P, U, P, U, P, U, P]
    size = vocab.calls.loss_work_bytes(t, v, k, v, flags | 3)
    work = torch.empty(size, dtype=torch.uint8, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    assert call(ctypes.addressof(arg), x.data_ptr(), k, k, w.data_ptr(), k, 0, v, loss.data_ptr(), lse.data_ptr(), c.data_ptr(), 1,
                None, dx.data_ptr(), k, dw.data_ptr(), k, work.data_ptr(), size, stream) == B.LCT_OK
    torch.cuda.synchronize()
    assert dx.isnan().all() and int(work[:4].view(torch.int32)) == B.LCT_ERR_TIMEOUT
    again = vocab.cross_entropy_grads(x, w, ids, *vocab.cross_entropy(x, w, ids), c)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])
