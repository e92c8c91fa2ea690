"""Gradients whose own gradients are not there: asking for them raises, whichever operands are leaves, whether or not
the call had to copy them, and with an upstream that needs no gradient."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_vocab import loss_case  # noqa: E402


@pytest.fixture(scope="module")
def vocab():
    from lossless_bf16_tensor_gb300 import vocab
    return vocab


def raises(loss, leaf):
    """A penalty on loss's gradient does not lose its term in silence."""
    (g,) = torch.autograd.grad(loss, leaf, create_graph=True)
    assert g.requires_grad
    with pytest.raises(RuntimeError):
        g.float().square().sum().backward()
    assert leaf.grad is None


CASES = ["plain", "shifted", "transposed"]


def leaf_and_view(kind, x):
    """A leaf, and what the call takes of it: itself, all but a sequence's last token (no single row index), a transpose."""
    if kind == "shifted":
        leaf = torch.cat([x.view(2, 10, -1), x.view(2, 10, -1)[:, :1]], 1).requires_grad_(True)
        return leaf, leaf[:, :-1]
    if kind == "transposed":
        leaf = x.t().contiguous().requires_grad_(True)
        return leaf, leaf.t()
    leaf = x.clone().requires_grad_(True)
    return leaf, leaf


@pytest.mark.parametrize("reduction", ["mean", "none"])
@pytest.mark.parametrize("kind", CASES)
def test_loss_of_a_frozen_weight(vocab, kind, reduction):
    x, w, ids, _ = loss_case(20, 30, 16, seed=50)
    leaf, view = leaf_and_view(kind, x)
    raises(vocab.linear_cross_entropy(view, w, ids, reduction).sum(), leaf)


@pytest.mark.parametrize("kind", ["plain", "transposed"])
def test_loss_of_frozen_activations(vocab, kind):
    x, w, ids, _ = loss_case(20, 30, 16, seed=51)
    leaf, view = leaf_and_view(kind, w)
    raises(vocab.linear_cross_entropy(x, view, ids), leaf)


@pytest.mark.parametrize("kind", CASES)
def test_loss_on_a_compressed_matrix(vocab, kind):
    from test_gpu_vocab_use import compressed
    x, w, ids, _ = loss_case(20, 2048, 64, seed=52)
    ct, cb = compressed(w)
    leaf, view = leaf_and_view(kind, x)
    for reduction in ("mean", "none"):
        loss = vocab.compressed_cross_entropy(view, ct, cb, 2048, 64, ids, reduction).sum()
        (want,) = torch.autograd.grad(loss, leaf, retain_graph=True)
        assert not want.requires_grad
        (got,) = torch.autograd.grad(loss, leaf, create_graph=True, retain_graph=True)
        assert torch.equal(got.detach(), want)
        raises(loss, leaf)
