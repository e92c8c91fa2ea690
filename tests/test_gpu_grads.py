"""The global gradient norm and clipping, against sums in 64 bits.

Tolerances.  The norm: partial sums of at most 64 squares are float32 (each
square and each sum is off by at most 2^-24, so a partial sum by at most
64 * 2^-24 = 2^-18), everything above them double; the root halves a relative
error and the result is rounded to float32 once: 2^-19 + 2^-24 < 2.1e-6.
Clipped values: the factor carries the norm's error in no digit a comparison
could see but 2^-19, and a value is rounded once: 2^-8 (half a BF16 step at
the most, relative) or 2^-23 beside it.  Values below the type's normal range
are compared to within half its smallest step.
"""
import math

import numpy as np
import pytest
import torch

from lossless_bf16_tensor_gb300 import binding as B
from lossless_bf16_tensor_gb300.grads import clip_grads, grad_norm

pytestmark = pytest.mark.gpu

NORM_TOL = 2.1e-6
STEP = {torch.bfloat16: (2.0 ** -8 + 2.0 ** -18, 2.0 ** -134), torch.float32: (2.0 ** -18, 2.0 ** -149)}
BF, F32 = torch.bfloat16, torch.float32


def make(sizes, dtypes, seed=0, scale=1e-2):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * scale).to(dtypes[i % len(dtypes)])
            for i, n in enumerate(sizes)]


def packed(sizes, dtype, seed=0, scale=1e-2, lead=1):
    """Views of one buffer at whatever offsets the sizes give, `lead` values in."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    buf = (torch.randn(sum(sizes) + lead + 7, generator=gen, device="cuda") * scale).to(dtype)
    at, out = lead, []
    for n in sizes:
        out.append(buf[at:at + n])
        at += n
    return buf, out


def exact_norm(gs):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in gs))


def check_norm(got, gs):
    want = exact_norm(gs)
    assert got.dtype == torch.float32 and got.shape == ()
    assert abs(got.item() - want) <= NORM_TOL * want


def check_clipped(norm, outs, before, max_norm):
    check_norm(norm, before)
    c = min(1.0, max_norm / (exact_norm(before) + 1e-6))
    for o, g in zip(outs, before):
        rel, tiny = STEP[g.dtype]
        want = g.double() * c
        assert o.dtype == g.dtype and bool(((o.double() - want).abs() <= want.abs() * rel + tiny).all())


SIZES = {
    "one": [1],
    "empty_and_one": [0, 1, 0],
    "vector_edges": [7, 8, 9, 15, 16, 17, 2047, 2048, 2049, 4095, 4097],
    "block_edges": [8 * 256 * 8 - 1, 8 * 256 * 8, 8 * 256 * 8 + 1, 3],
    "many_small": [1 + (37 * i) % 501 for i in range(300)],
    "more_than_a_table": [1 + (i % 5) for i in range(2500)] + [100_001],
    "large": [5_000_003, 1, 1_234_567],
}


@pytest.mark.parametrize("dtypes", [[BF], [F32], [BF, F32]], ids=["bf16", "f32", "mixed"])
@pytest.mark.parametrize("sizes", SIZES, ids=list(SIZES))
def test_norm_and_clip(sizes, dtypes):
    gs = make(SIZES[sizes], dtypes, seed=len(sizes))
    check_norm(grad_norm(gs), gs)
    before = [g.clone() for g in gs]
    max_norm = 0.3 * exact_norm(gs) + 1e-9
    out = [torch.empty_like(g) for g in gs]
    check_clipped(clip_grads(gs, max_norm, out=out), out, before, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(gs, before))
    norm = clip_grads(gs, max_norm)
    check_clipped(norm, gs, before, max_norm)
    assert all(torch.equal(a, b) for a, b in zip(gs, out))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("lead", [0, 1, 2, 3, 5, 7])
def test_views_of_a_bucket(dtype, lead):
    """Slices at odd offsets, clipped in place and into a bucket of another
    phase; nothing beside the slices changes."""
    sizes = [1, 2, 3, 5, 8, 13, 2051, 70_001, 9]
    buf, gs = packed(sizes, dtype, seed=lead, lead=lead)
    before = [g.clone() for g in gs]
    whole = buf.clone()
    max_norm = 0.5 * exact_norm(gs)
    obuf, outs = packed(sizes, dtype, seed=99, lead=(3 * lead + 1) % 8)
    keep = obuf.clone()
    check_clipped(clip_grads(gs, max_norm, out=outs), outs, before, max_norm)
    assert torch.equal(buf, whole)
    lo = (3 * lead + 1) % 8
    assert torch.equal(obuf[:lo], keep[:lo]) and torch.equal(obuf[lo + sum(sizes):], keep[lo + sum(sizes):])
    check_clipped(clip_grads(gs, max_norm), gs, before, max_norm)
    assert torch.equal(buf[:lead], whole[:lead]) and torch.equal(buf[lead + sum(sizes):], whole[lead + sum(sizes):])
    assert all(torch.equal(a, b) for a, b in zip(gs, outs))


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e-30, 1e-25, 1e-12, 1e12, 1e25, 1e30])
def test_squares_outside_floats_range(dtype, scale):
    """Squares of 1e-30 vanish and squares of 1e30 overflow in float32."""
    gs = make([4099, 1, 33_333], [dtype], seed=3, scale=scale)
    check_norm(grad_norm(gs), gs)
    before = [g.clone() for g in gs]
    max_norm = 0.25 * exact_norm(gs)
    if max_norm > 1e-4:  # the formula's 1e-6 would decide below
        check_clipped(clip_grads(gs, max_norm), gs, before, max_norm)


def test_one_large_value_beside_tiny_ones():
    g = torch.full((100_000,), 1e-22, device="cuda")
    g[77_777] = 3e19
    check_norm(grad_norm([g]), [g])
    h = torch.full((1 << 20,), 1e-22, device="cuda")
    check_norm(grad_norm([h]), [h])


def test_norm_above_floats_range_still_clips():
    g = torch.full((1 << 20,), 3e38, device="cuda", dtype=BF)
    before = g.clone()
    norm = clip_grads([g], 1.0)
    assert norm.item() == math.inf
    c = 1.0 / exact_norm([before])
    want = before.double() * c
    assert bool(((g.double() - want).abs() <= want.abs() * STEP[BF][0]).all())


def test_zeros_and_empty_lists():
    z = [torch.zeros(5000, device="cuda", dtype=BF), -torch.zeros(3, device="cuda")]
    assert grad_norm(z).item() == 0.0
    assert clip_grads(z, 1.0).item() == 0.0
    assert grad_norm([]).item() == 0.0
    assert clip_grads([], 1.0).item() == 0.0
    assert grad_norm([torch.empty(0, device="cuda")]).item() == 0.0


def test_below_the_limit_nothing_changes():
    gs = make([1000, 77], [BF, F32], seed=5)
    before = [g.clone() for g in gs]
    norm = clip_grads(gs, 1e6)
    check_norm(norm, before)
    assert all(torch.equal(a, b) for a, b in zip(gs, before))
    out = [torch.zeros_like(g) for g in gs]
    clip_grads(gs, 1e6, out=out)
    assert all(torch.equal(a, b) for a, b in zip(out, before))


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_not_finite(bad):
    gs = make([10_000, 5], [BF, F32], seed=6)
    gs[0][1234] = bad
    norm = clip_grads(gs, 1.0)
    assert math.isnan(norm.item()) if math.isnan(bad) else norm.item() == math.inf
    if math.isnan(bad):
        assert all(bool(g.isnan().all()) for g in gs)
    else:
        assert gs[0][1234].isnan() and int((gs[0] != 0).sum()) == 1 and not bool((gs[1] != 0).any())


def test_same_result_every_time():
    gs = make([3_000_001, 17, 999_999], [BF, F32], seed=7)
    want = grad_norm(gs)
    for _ in range(5):
        assert torch.equal(grad_norm(gs), want)
    out = [torch.empty_like(g) for g in gs]
    assert torch.equal(clip_grads(gs, 1.0, out=out), want)


def test_on_another_stream():
    gs = make([2_000_000, 123], [BF], seed=8)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        a = grad_norm(gs)
    s.synchronize()
    check_norm(a, gs)


def test_in_a_graph():
    gs = make([300_000, 123, 5], [BF, F32], seed=9)
    out = [torch.empty_like(g) for g in gs]
    clip_grads(gs, 0.5, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        norm = clip_grads(gs, 0.5, out=out)
    for g in gs:
        g.mul_(2)
    graph.replay()
    torch.cuda.synchronize()
    check_clipped(norm, out, gs, 0.5)


def test_refusals():
    g = make([100, 50], [BF])
    with pytest.raises(B.LctError):
        grad_norm([torch.zeros(4, device="cuda", dtype=torch.float16)])
    with pytest.raises(ValueError):
        grad_norm([torch.zeros(4)])
    with pytest.raises(ValueError):
        grad_norm([torch.zeros(8, 8, device="cuda").t()[1:]])
    for bad in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(B.LctError):
            clip_grads(g, bad)
    with pytest.raises(ValueError):
        clip_grads(g, 1.0, out=[g[0]])
    with pytest.raises(ValueError):
        clip_grads(g, 1.0, out=[g[0], g[1].float()])
    with pytest.raises(B.LctError):
        clip_grads([g[0], g[0]], 1.0)                      # the same tensor twice
    with pytest.raises(B.LctError):
        clip_grads(g, 1.0, out=[torch.empty_like(g[0]), g[0][:50]])
    buf = torch.zeros(300, device="cuda", dtype=BF)
    with pytest.raises(B.LctError):
        clip_grads([buf[:100], buf[99:199]], 1.0)
    clip_grads([buf[:100], buf[100:200]], 1.0, out=[buf[:100], buf[200:300]])


def test_clipped_gradient_into_a_fused_step():
    """Clipping, then the fused momentum step, equals the step on gradients
    scaled outside: the two meet in memory as plain BF16."""
    from lossless_bf16_tensor_gb300 import synth
    n = 70_000
    w, m = (torch.from_numpy(synth.normal(n, s, k).view(np.int16)).cuda() for s, k in ((0.02, 1), (1e-3, 2)))
    cbw, cbm = B.lct_codebook_build("gaussian", 0.02), B.lct_codebook_build("gaussian", 1e-3)
    g = make([n], [BF], seed=10, scale=1.0)[0]
    h = g.clone()
    clip_grads([g], 1.0)
    h = (h.float() * float(np.float32(1.0 / (exact_norm([h]) + 1e-6)))).to(BF)
    res = []
    for grad in (g, h):
        W, M = B.CompressedTensor(n, 0), B.CompressedTensor(n, 0)
        B.lct_encode(w, cbw, W)
        B.lct_encode(m, cbm, M)
        W2, M2 = B.CompressedTensor(n, 0), B.CompressedTensor(n, 0)
        B.lct_sgd_momentum_step_fused(W, cbw, M, cbm, grad.view(torch.int16), 1e-3, 0.9, W2, M2)
        y = torch.empty(n, dtype=torch.int16, device="cuda")
        B.lct_decode(W2, cbw, y)
        assert W2.state().status == 0
        res.append(y.view(BF).double())
    assert bool(((res[0] - res[1]).abs() <= 2.0 ** -7 * res[1].abs() + 1e-5).all())
