"""What a call of the loss divides by itself: rows of an odd length that are moved a part of the vocabulary at a time,
and depths that are summed in several parts where tokens are many."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_vocab import loss_bounds, loss_case, within  # noqa: E402


@pytest.fixture(scope="module")
def vocab():
    from lossless_bf16_tensor_gb300 import vocab
    return vocab


@pytest.mark.parametrize("t,v,k", [(40, 70_000, 1001), (2000, 3000, 2056), (1100, 500, 4096)])
def test_loss_and_gradients(vocab, t, v, k):
    """2^26 values of the first one's rows are 65,536 of them: two parts.  Sums of the others are of 1024 of depth, three
    (the last of 8) and four."""
    x, w, ids, c = loss_case(t, v, k, 0.2, seed=70)
    last = ids.clone()
    last[:5] = v - 1                                              # targets of the last part too
    last[5:9] = min(v - 1, 65_535)
    bounds = loss_bounds(x, w, last, c)
    loss, lse = vocab.cross_entropy(x, w, last)
    within(loss, bounds[0], "loss")
    within(lse, bounds[1], "lse")
    dx, dw = vocab.cross_entropy_grads(x, w, last, loss, lse, c)
    within(dx, bounds[2], "dx")
    within(dw, bounds[3], "dw")
    again = vocab.cross_entropy(x, w, last)
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)


def test_losses_of_many_sure_tokens(vocab):
    """As exact as sums of 1024 of depth are: what a sum over the whole depth drops would show."""
    t, k = 1100, 8192
    x, w, ids, _ = loss_case(t, 3000, k, seed=71, lean=0.0)
    x = (x.float() * 0.5 + 3.0 * w[ids].float()).to(x.dtype)
    z = x.double() @ w.double().t()
    want = torch.logsumexp(z, 1) - z.gather(1, ids[:, None])[:, 0]
    assert float(want.median()) < 0.1
    loss, _ = vocab.cross_entropy(x, w, ids)
    # each of a part's sums drops at most 2^-23 of the terms' size, the parts' sum as much for each part; twice, as both
    # logits of a difference are off; a loss moves by its own size times what the logits do
    mass, part = x.double().abs() @ w.double().abs().t(), 1024
    off = 2 * (part / 16 + 17 + k / part) * 2.0 ** -23 * mass.amax(1)
    assert ((loss.double() - want).abs() <= off * want + 2.0 ** -21 * want + 2.0 ** -22).all()
