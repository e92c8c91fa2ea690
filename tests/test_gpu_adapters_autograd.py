"""What autograd can and cannot do with the adapters: what it cannot raises instead
of giving a gradient that is wrong or not there."""
import pytest
import torch

from lossless_bf16_tensor_gb300.adapters import AdapterBank, adapter_linear
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
