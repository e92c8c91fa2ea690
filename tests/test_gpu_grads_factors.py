"""Clipping where the norm, or the factor, lies far from 1: c = min(1, max_norm /
(norm + 1e-6)) in 64 bits, with the tolerances of the norm's and the clipping's
other tests."""
import math

import pytest
import torch

from lossless_bf16_tensor_gb300.grads import clip_grads
from test_gpu_grads import STEP, exact_norm

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def gradients(sizes, dtypes, norm):
    """Tensors with about that norm, their values within a factor of four of each other."""
    gen = torch.Generator(device="cuda").manual_seed(len(sizes))
    total = sum(sizes)
    out = []
    for i, n in enumerate(sizes):
        v = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64) * 0.75 + 0.25
        v *= torch.where(torch.rand(n, generator=gen, device="cuda") < 0.5, -1.0, 1.0)
        # (a root mean square of 0.66)
        out.append((v * (norm / math.sqrt(total) / 0.66)).clamp(-3.38e38, 3.38e38).to(dtypes[i % len(dtypes)]))
    return out


def check(gs, max_norm):
    before = [g.clone() for g in gs]
    norm = exact_norm(gs)
    c = min(1.0, max_norm / (norm + 1e-6))
    out = [torch.zeros_like(g) for g in gs]
    got = clip_grads(gs, max_norm, out=out).item()
    assert all(torch.equal(a, b) for a, b in zip(gs, before))
    assert got == math.inf if norm > 3.4028235e38 else abs(got - norm) <= 2.1e-6 * norm
    clip_grads(gs, max_norm)
    for g, o, b in zip(gs, out, before):
        assert torch.equal(g, o)
        if c == 1.0:
            assert torch.equal(g, b)
            continue
        rel, tiny = STEP[g.dtype]
        want = b.double() * c
        assert bool(((o.double() - want).abs() <= want.abs() * rel + tiny).all())


# one launch of a cluster, and a launch for each step
SIZES = {"few": [1000, 7, 4099], "many": [300_000, 5, 123_457]}


@pytest.mark.parametrize("dtypes", [[BF], [F32], [BF, F32]], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=list(SIZES))
@pytest.mark.parametrize("exponent", [99, 100, 101, 102, 110, 120, 126, 127, 129, 134])
@pytest.mark.parametrize("max_norm", [1e-20, 1.0, 1e31, 3e38])
def test_large_norms(exponent, max_norm, sizes, dtypes):
    check(gradients(SIZES[sizes], dtypes, 1.3 * 2.0 ** exponent), max_norm)


@pytest.mark.parametrize("dtypes", [[BF], [F32]], ids=["bf16", "f32"])
@pytest.mark.parametrize("sizes", SIZES, ids=list(SIZES))
@pytest.mark.parametrize("norm,max_norm", [(1e30, 1e-10), (1e30, 1e-8), (1e37, 1e-30), (1.0, 1e-38), (1.0, 1e-44),
                                           (1e-3, 1e-42), (1e38, 1e-41), (2.0 ** 127, 2.0 ** -100)])
def test_factors_below_floats_normal_range(norm, max_norm, sizes, dtypes):
    check(gradients(SIZES[sizes], dtypes, norm), max_norm)


def test_a_limit_above_a_huge_norm_changes_nothing():
    for values, max_norm in (([1e31] * 4, 1e35), ([1e33] * 4, 3e38)):
        g = torch.tensor(values, device="cuda")
        h = g.clone()
        clip_grads([g], max_norm)
        assert torch.equal(g, h)
