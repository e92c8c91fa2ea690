"""A penalty on a gradient of adapter_linear raises, whichever operand is a leaf and whatever the upstream needs."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_second_derivatives import raises  # noqa: E402


@pytest.mark.parametrize("which", ["x", "a", "b"])
def test_adapters(which):
    """dx depends on a and b, their gradients on x: a sum's upstream needs no gradient."""
    from lossless_bf16_tensor_gb300.adapters import AdapterBank, adapter_linear
    from test_gpu_adapters import Case, compressed_weight
    w, cb, _ = compressed_weight(256, 128, 31)
    c = Case(200, 3, 16, 128, 256, seed=0)
    ops = {name: t.clone().requires_grad_(name == which) for name, t in (("x", c.x), ("a", c.a), ("b", c.b))}
    y = adapter_linear(ops["x"], w, cb, AdapterBank(ops["a"], ops["b"], c.scale), c.plan)
    raises(y.float().sum(), ops[which])
