"""What follows a call in the stream comes after all of it, when no adapter has
work too: the backward call's second kernel may start early, and what is
enqueued next is ordered behind that one."""
import pytest
import torch

from lossless_bf16_tensor_gb300.adapters import AdapterBank, adapter_grads, adapter_plan

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def no_work(kind, t, n, r, k, m):
    """A batch in which no adapter has anything to do: no tokens, or no ranks."""
    gen = torch.Generator(device="cuda").manual_seed(t)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(BF)

    index = torch.full((t,), -1, dtype=torch.int32, device="cuda")
    ranks = None
    if kind == "no ranks":
        index = torch.arange(t, dtype=torch.int32, device="cuda") % n
        ranks = torch.zeros(n, dtype=torch.int32, device="cuda")
    bank = AdapterBank(normal(n, r, k), normal(n, m, r), torch.ones(n, device="cuda"), ranks)
    return bank, adapter_plan(index, n), normal(t, m), normal(t, k), torch.zeros(t, r, device="cuda"), normal(t, k)


@pytest.mark.parametrize("kind", ["no tokens", "no ranks"])
@pytest.mark.parametrize("t,n", [(16_000, 2), (300, 400)])
def test_a_reader_behind_a_batch_without_work(kind, t, n):
    bank, plan, dy, x, xa, dx = no_work(kind, t, n, 8, 4096, 64)
    torch.cuda.synchronize()
    for _ in range(5):
        out, da, db = adapter_grads(dy, x, xa, bank, plan, dx, out=torch.zeros_like(dx))
        seen = out.clone()
        assert torch.equal(seen, dx) and not bool(da.any()) and not bool(db.any())


@pytest.mark.parametrize("kind", ["no tokens", "no ranks"])
def test_a_reader_behind_it_in_a_graph(kind):
    bank, plan, dy, x, xa, dx = no_work(kind, 16_000, 2, 8, 4096, 64)
    out = torch.zeros_like(dx)
    adapter_grads(dy, x, xa, bank, plan, dx, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out.zero_()
        adapter_grads(dy, x, xa, bank, plan, dx, out=out)
        seen = out.clone()
    for _ in range(5):
        dx.neg_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(seen, dx)
