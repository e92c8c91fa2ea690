"""Operands that require a gradient where the call would give none: it raises."""
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
