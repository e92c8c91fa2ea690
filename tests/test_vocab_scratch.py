"""What the loss's scratch is bounded by (no GPU)."""
import random

import pytest

from test_vocab_abi import UNSUPPORTED, backward, forward, gradient, lib, lookup  # noqa: F401

SIZES = [(1, 2 ** 24, 64), (100, 2 ** 24, 64), (2048, 2 ** 20, 64), (2048, 2 ** 24, 4096), (8192, 32_768, 4096),
         (10_000, 1_000_001, 1001), (32_768, 262_144, 4096), (100_000, 2 ** 24, 8), (2 ** 20, 131_072, 512),
         (2 ** 24, 50_257, 768), (2 ** 24, 2 ** 24, 64)]


@pytest.mark.parametrize("t,v,k", SIZES)
def test_forward(lib, t, v, k):  # noqa: F811
    """256 MB for the tiles' maxima and sums, a few words a token, and (rows that have to be moved) x and 2^26 values of W."""
    lines = (k + 63) // 64 * 64
    for flags in (0, 4):
        bound = (1 << 28) + 13 * t + 4096
        if flags and t > 2:
            bound += 2 * t * lines + max(1 << 27, 512 * lines)
        assert 0 < lib.lct_loss_work_bytes(t, v, k, v, flags) <= bound


@pytest.mark.parametrize("t,v,k", SIZES)
def test_backward(lib, t, v, k):  # noqa: F811
    """g: 256 MB, or 256 columns of it; dx's parts: 256 MB, or one; beside them x, the targets' sums, a few words a token and
    (with dW) one a row."""
    lines, floats = (k + 63) // 64 * 64, (k + 7) // 8 * 8
    for flags in (1, 3, 5, 7):
        g = max(1 << 28, 512 * ((t + 255) // 256 * 256))
        parts = max(1 << 28, 4 * t * floats)
        bound = g + parts + 2 * t * lines + 28 * t + 8192
        if flags & 2:
            # the partial sums of the targets' terms share g's room
            bound += 4 * v + 4 * t * floats + 8 * (t // 8 + 1) * (floats + 8)
        if flags & 4:
            bound += max(1 << 27, 512 * lines)
        assert 0 < lib.lct_loss_work_bytes(t, v, k, v, flags) <= bound


def test_columns_beyond_the_limit(lib):  # noqa: F811
    wide = 2 ** 16 + 1
    assert lookup(lib, cols=wide, ldt=2 ** 17, ldo=2 ** 17) == UNSUPPORTED
    assert gradient(lib, cols=wide, ldd=2 ** 17, ldo=2 ** 17) == UNSUPPORTED
    assert forward(lib, cols=wide, ldx=2 ** 17, ldw=2 ** 17) == UNSUPPORTED
    assert backward(lib, cols=wide, ldx=2 ** 17, ldw=2 ** 17, ldd=2 ** 17, lddw=2 ** 17) == UNSUPPORTED


def test_forward_of_smaller_pieces(lib):  # noqa: F811
    """Scratch for pieces of at most some rows is enough for every smaller one: the last of a matrix is."""
    rng = random.Random(1)
    v = 2 ** 24
    for t in (1, 2, 777, 2048, 2500, 10_000, 32_768, 100_000):
        for _ in range(300):
            rows = int(2 ** rng.uniform(0, 24))
            less = rng.choice([rows - 1, rows - 64, rows - 256, rows // 2, rng.randint(1, rows), rows // 64 * 64])
            if less < 1:
                continue
            for flags in (0, 4):
                assert lib.lct_loss_work_bytes(t, v, 64, less, flags) <= lib.lct_loss_work_bytes(t, v, 64, rows, flags), (t, rows, less)
