"""Operands that require a gradient, or carry a forward-mode tangent, where the call would give none: it raises."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_vocab import loss_case  # noqa: E402


@pytest.fixture(scope="module")
def vocab():
    from lossless_bf16_tensor_gb300 import vocab
    return vocab


def test_a_base_that_requires_a_gradient(vocab):
    x, w, ids, _ = loss_case(20, 30, 16, seed=60)
    base = w.clone().requires_grad_(True)
    want = vocab.embedding_grad(x, ids, 30, base=w)
    with pytest.raises(RuntimeError, match="embedding_grad"):
        vocab.embedding_grad(x, ids, 30, base=base)
    with torch.no_grad():
        assert torch.equal(vocab.embedding_grad(x, ids, 30, base=base), want)


def test_tangents_are_refused(vocab):
    import torch.autograd.forward_ad as fw
    from lossless_bf16_tensor_gb300.adapters import adapter_apply, adapter_linear
    from test_gpu_adapters import Case, compressed_weight
    from test_gpu_vocab_use import compressed
    x, w, ids, c = loss_case(20, 2048, 64, seed=61)
    ct, cb = compressed(w)
    loss, lse = vocab.cross_entropy(x, w, ids)
    grown = x.clone().requires_grad_(True)
    cw, ccb, _ = compressed_weight(256, 128, 31)
    a = Case(20, 3, 16, 128, 256, seed=0)
    calls = {
        "embedding": lambda t: vocab.embedding(ids, t(w)),
        "embedding into out": lambda t: vocab.embedding(ids, w, out=t(x.clone())),
        "embedding_grad": lambda t: vocab.embedding_grad(t(x), ids, 2048),
        "its base": lambda t: vocab.embedding_grad(x, ids, 2048, base=t(w)),
        "cross_entropy": lambda t: vocab.cross_entropy(t(x), w, ids),
        "its weight": lambda t: vocab.cross_entropy(x, t(w), ids),
        "cross_entropy_grads": lambda t: vocab.cross_entropy_grads(x, w, ids, loss, lse, t(c)),
        "linear_cross_entropy": lambda t: vocab.linear_cross_entropy(t(x), w, ids),
        "its weight, transposed": lambda t: vocab.linear_cross_entropy(x, t(w.t().contiguous()).t(), ids),
        "beside a leaf": lambda t: vocab.linear_cross_entropy(grown, t(w), ids),
        "compressed_cross_entropy": lambda t: vocab.compressed_cross_entropy(t(x), ct, cb, 2048, 64, ids),
        "compressed_cross_entropy_grads": lambda t: vocab.compressed_cross_entropy_grads(t(x), ct, cb, 2048, 64, ids),
        "adapter_apply": lambda t: adapter_apply(t(a.x), a.bank, a.plan, a.y),
        "its y": lambda t: adapter_apply(a.x, a.bank, a.plan, t(a.y)),
        "adapter_linear": lambda t: adapter_linear(t(a.x), cw, ccb, a.bank, a.plan),
    }
    with fw.dual_level():
        for name, call in calls.items():
            for mode in (torch.enable_grad, torch.no_grad):
                if name == "beside a leaf" and mode is torch.no_grad:
                    continue
                with mode(), pytest.raises(RuntimeError):
                    call(lambda t: fw.make_dual(t, torch.ones_like(t)))
                    pytest.fail(name)
    for call in calls.values():
        call(lambda t: t)                                         # without a tangent each of them works
