"""The loss's forward pass where its tiles' maxima and sums would pass their room: tokens, and above 2^20 rows the
vocabulary too, are worked on in parts of one call."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_vocab import loss_case, summed  # noqa: E402


@pytest.fixture(scope="module")
def vocab():
    from lossless_bf16_tensor_gb300 import vocab
    return vocab


@pytest.mark.parametrize("t,v", [(9000, 262_144), (2100, 1_100_000)])
def test_parts_of_tokens_and_rows(vocab, t, v):
    k = 8
    x, w, ids, _ = loss_case(t, v, k, 0.1, seed=80)
    ids[:3] = v - 1
    loss, lse = vocab.cross_entropy(x, w, ids)
    # 64 bits, a part of the vocabulary at a time
    top = torch.full((t,), -torch.inf, device="cuda", dtype=torch.float64)
    total, mass, mine = torch.zeros_like(top), torch.zeros_like(top), torch.zeros_like(top)
    step = 50_000
    for r in range(0, v, step):
        part = w[r:r + step].double()
        z = x.double() @ part.t()
        high = torch.maximum(top, z.amax(1))
        total = total * torch.exp(top - high) + torch.exp(z - high[:, None]).sum(1)
        top = high
        mass = torch.maximum(mass, (x.double().abs() @ part.abs().t()).amax(1))
        here = (ids >= r) & (ids < r + step)
        mine = torch.where(here, z.gather(1, (ids - r).clamp(0, part.shape[0] - 1)[:, None])[:, 0], mine)
    want = top + torch.log(total)
    # the bounds of loss_bounds: sums of products, exponentials and their sums (of v terms in pairs of tiles), roundings
    off_z = summed(k) * mass
    off = off_z + 2.0 ** -20 + 2.0 ** -22 * (mass + want.abs())
    assert ((lse.double() - want).abs() <= off).all()
    have = ids >= 0
    exact = torch.where(have, want - mine, 0.0)
    assert ((loss.double() - exact).abs() <= torch.where(have, off + off_z + 2.0 ** -23 * exact.abs(), 0.0)).all()
    # a token's result does not go by how many others there are
    if v <= 2 ** 20:
        for some in (slice(0, 8192), slice(8192, t), slice(4000, 5000 + 1024)):
            one = vocab.cross_entropy(x[some], w, ids[some])
            assert torch.equal(one[0], loss[some]) and torch.equal(one[1], lse[some])


def test_a_smaller_last_piece(vocab):
    """Scratch for the first of two pieces is enough for the second, whose 64 rows less let more tokens be done at a time."""
    t, k, first, rest = 9000, 8, 262_208, 262_144
    v = first + rest
    x, w, ids, _ = loss_case(t, v, k, 0.1, seed=81)
    want = vocab.cross_entropy(x, w, ids)
    work = torch.empty(vocab.calls.loss_work_bytes(t, v, k, first, 0), dtype=torch.uint8, device="cuda")
    loss, lse, total = (torch.zeros(n, device="cuda") for n in (t, t, 3))
    vocab.calls.cross_entropy_piece(x, w[:first], 0, v, ids, loss, lse, total, work)
    vocab.calls.cross_entropy_piece(x, w[first:], first, v, ids, loss, lse, total, work)
    # the same products; exponentials and sums, joined in another order, are off as in the test above, here on both sides
    off = 2 * (2.0 ** -20 + 2.0 ** -22 * 2 * want[1].abs())
    assert ((lse - want[1]).abs() <= off).all()
    assert ((loss - want[0]).abs() <= off + 2.0 ** -22 * want[0].abs()).all()
    assert torch.equal(loss[ids < 0], want[0][ids < 0])
