"""What autograd can and cannot do with the adapters: what it cannot raises instead
of giving a gradient that is wrong or not there."""
import pytest
import torch

from lossless_bf16_tensor_gb300 import binding as B
from lossless_bf16_tensor_gb300.activations import compressed_activations
from lossless_bf16_tensor_gb300.adapters import AdapterBank, adapter_apply, adapter_grads, adapter_linear, adapter_plan
from lossless_bf16_tensor_gb300.grads import clip_grads, grad_norm
from test_gpu_adapters import Case, compressed_weight

pytestmark = pytest.mark.gpu

N, K = 256, 128


@pytest.fixture(scope="module")
def weight():
    return compressed_weight(N, K, 31)


def leaves(seed=0, t=200):
    """A batch, with a and b as parameters and x as a leaf."""
    c = Case(t, 3, 16, K, N, seed=seed)
    a, b = torch.nn.Parameter(c.a.clone()), torch.nn.Parameter(c.b.clone())
    return c, c.x.clone().requires_grad_(True), AdapterBank(a, b, c.scale)


def test_second_derivatives_raise(weight):
    w, cb, _ = weight
    c, x, bank = leaves()
    y = adapter_linear(x, w, cb, bank, c.plan)
    (gx,) = torch.autograd.grad(y.float().square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        gx.float().square().sum().backward()


@pytest.mark.parametrize("hooks", [False, True], ids=["plain", "compressed"])
@pytest.mark.parametrize("what", ["a", "b", "scale", "ranks", "order", "starts", "tiles"])
def test_operands_modified_before_backward_raise(weight, what, hooks):
    w, cb, _ = weight
    c, x, bank = leaves(seed=1, t=600)
    bank = AdapterBank(bank.a, bank.b, bank.scale, torch.full((3,), 12, dtype=torch.int32, device="cuda"))
    saved = compressed_activations(B.lct_codebook_build("gaussian", 1.0))
    if hooks:
        with saved:
            y = adapter_linear(x * 1.0, w, cb, bank, c.plan)
    else:
        y = adapter_linear(x * 1.0, w, cb, bank, c.plan)
    loss = y.float().square().sum()
    loss.backward(retain_graph=True)
    first = [v.grad.clone() for v in (x, bank.a, bank.b)]
    x.grad = bank.a.grad = bank.b.grad = None
    loss.backward(retain_graph=True)  # nothing was modified: the same again
    assert all(torch.equal(v.grad, g) for v, g in zip((x, bank.a, bank.b), first))
    operand = getattr(bank, what, None)
    with torch.no_grad():
        (operand if operand is not None else getattr(c.plan, what)).add_(0)
    with pytest.raises(RuntimeError, match=what):
        loss.backward()


def test_a_bank_with_other_tensors_before_backward(weight):
    """A bank that is given other tensors afterwards changes nothing for a forward pass that was made."""
    w, cb, _ = weight
    c, x, bank = leaves(seed=2)
    adapter_linear(x, w, cb, bank, c.plan).float().square().sum().backward()
    want = x.grad.clone(), bank.a.grad.clone()
    x.grad = bank.a.grad = None
    loss = adapter_linear(x, w, cb, bank, c.plan).float().square().sum()
    a, bank.a = bank.a, torch.nn.Parameter(torch.zeros_like(bank.a))
    loss.backward()
    assert torch.equal(x.grad, want[0]) and torch.equal(a.grad, want[1]) and bank.a.grad is None


def test_operands_made_in_inference_mode(weight):
    """They have no versions; a frozen bank of such tensors still gives x its gradient."""
    w, cb, _ = weight
    c = Case(200, 3, 16, K, N, seed=3)
    with torch.inference_mode():
        frozen = AdapterBank(c.a.clone(), c.b.clone(), c.scale.clone())
    grads = []
    for bank in (c.bank, frozen):
        x = c.x.clone().requires_grad_(True)
        adapter_linear(x, w, cb, bank, c.plan).float().square().sum().backward()
        grads.append(x.grad)
    assert torch.equal(*grads)


def test_what_is_written_in_place_gets_another_version():
    c = Case(50, 2, 8, 64, 72, seed=4)
    y, dx = c.y.clone(), c.dx.clone()
    _, xa = adapter_apply(c.x, c.bank, c.plan, y, out=y, keep=True)
    adapter_grads(c.dy, c.x, xa, c.bank, c.plan, dx, out=dx)
    assert (y._version, dx._version) == (1, 1)
    gs = [v.clone() for v in (c.x, c.y)]
    out = [torch.empty_like(g) for g in gs]
    clip_grads(gs, 1.0, out=out)
    assert [g._version for g in gs] == [0, 0] and [o._version for o in out] == [1, 1]
    clip_grads(gs, 1.0)
    assert [g._version for g in gs] == [1, 1]
    flat = torch.zeros(100, device="cuda")
    clip_grads([flat[:40], flat[40:]], 1.0)  # views share their base's version
    assert flat._version == 2
    grad_norm(gs)
    adapter_grads(c.dy, c.x, xa, c.bank, c.plan, dx)
    assert [v._version for v in (*gs, c.x, c.y, c.dy, dx, xa, c.a, c.b)] == [1, 1, 0, 0, 0, 1, 0, 0, 0]


def test_a_saved_tensor_that_is_written_over_is_noticed():
    c = Case(50, 2, 8, 64, 72, seed=5)

    def loss(v):
        v = v.clone().requires_grad_(True) * 1.0
        return v, v.square().sum()

    for write in (lambda v: adapter_apply(c.x, c.bank, c.plan, c.y, out=v),
                  lambda v: adapter_apply(c.x, c.bank, c.plan, v, out=v),
                  lambda v: clip_grads([v], 1.0)):
        v, s = loss(c.y)
        with torch.no_grad():
            write(v)
        with pytest.raises(RuntimeError):
            s.backward()


def test_tensors_made_in_inference_mode_are_written():
    c = Case(50, 2, 8, 64, 72, seed=6)
    want = adapter_apply(c.x, c.bank, c.plan, c.y)
    with torch.inference_mode():
        y, g = c.y.clone(), c.dy.clone()
        adapter_apply(c.x, c.bank, c.plan, y, out=y)
    assert torch.equal(y, want)
    z = c.y.clone()
    with torch.inference_mode():
        adapter_apply(c.x, c.bank, c.plan, z, out=z)
    assert torch.equal(z, want)
    with torch.no_grad():
        clip_grads([g], 1e-3)
        adapter_apply(c.x, c.bank, c.plan, y, out=y)
    assert abs(float(g.double().norm()) - 1e-3) < 1e-5


def test_gradients_that_are_not_there_raise(weight):
    w, cb, _ = weight
    c = Case(50, 2, 8, K, N, seed=7)
    want = adapter_apply(c.x, c.bank, c.plan, c.y)

    def grad(v):
        return v.clone().requires_grad_(True)

    ok = dict(x=c.x, bank=c.bank, plan=c.plan, y=c.y)
    for kw in (dict(x=grad(c.x)), dict(y=grad(c.y)), dict(out=grad(c.y)),
               dict(bank=AdapterBank(torch.nn.Parameter(c.a), c.b, c.scale)),
               dict(bank=AdapterBank(c.a, torch.nn.Parameter(c.b), c.scale)),
               dict(bank=AdapterBank(c.a, c.b, grad(c.scale)))):
        with pytest.raises(RuntimeError, match="adapter_linear"):
            adapter_apply(**{**ok, **kw})
        with torch.no_grad():
            assert torch.equal(adapter_apply(**{**ok, **kw}), want)
        with torch.inference_mode():
            assert torch.equal(adapter_apply(**{**ok, **kw}), want)
    learnt = AdapterBank(c.a, c.b, grad(c.scale))
    with pytest.raises(RuntimeError, match="scale"):
        adapter_linear(c.x, w, cb, learnt, c.plan)
    with torch.no_grad():
        assert adapter_linear(c.x, w, cb, learnt, c.plan).shape == (50, N)
    # the gradients' own call is for those who make them by hand
    _, xa = adapter_apply(c.x, c.bank, c.plan, c.y, keep=True)
    bank = AdapterBank(torch.nn.Parameter(c.a), torch.nn.Parameter(c.b), c.scale)
    assert adapter_grads(c.dy, c.x, xa, bank, c.plan, c.dx)[1].shape == c.a.shape


@pytest.mark.parametrize("layout", ["permuted", "expanded row", "expanded batch", "columns", "strided", "one token"])
def test_x_at_any_strides(weight, layout):
    """As compressed_linear takes it: the same results and gradients as for a contiguous copy."""
    w, cb, _ = weight
    c = Case(60, 2, 8, K, N, seed=8)
    base = c.x

    def views(v):
        return {"permuted": lambda: v.view(3, 20, K).transpose(0, 1),
                "expanded row": lambda: v[:1].expand(60, K),
                "expanded batch": lambda: v.view(3, 20, K)[:, :1].expand(3, 20, K),
                "columns": lambda: v.view(K, 60).t(),
                "strided": lambda: torch.cat([v, v], 1)[:, 8:8 + K],
                "one token": lambda: v[7:8, :]}[layout]()

    plan = c.plan if layout != "one token" else adapter_plan(c.index[7:8], 2)
    results = []
    for copy in (False, True):
        leaf = base.clone().requires_grad_(True)
        a, b = torch.nn.Parameter(c.a.clone()), torch.nn.Parameter(c.b.clone())
        x = views(leaf)
        x = x.contiguous() if copy else x
        bank = AdapterBank(a, b, c.scale)
        y = adapter_linear(x, w, cb, bank, plan)
        assert y.shape == (*x.shape[:-1], N)
        y.float().square().sum().backward()
        with torch.no_grad():
            assert torch.equal(adapter_linear(x, w, cb, bank, plan), y)
        results.append((y.detach(), leaf.grad, a.grad, b.grad))
    assert all(torch.equal(p, q) for p, q in zip(*results))
