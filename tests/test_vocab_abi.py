"""Host-side checks of the lookup and the loss (no GPU): every call here is
refused, or has nothing to do, before anything is enqueued."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p
U64 = ctypes.c_uint64
A, B, X, OUT, WORK = (0x10000000 * i for i in range(1, 6))  # addresses that nobody reads


class Ids(ctypes.Structure):
    _fields_ = [("ids", P), ("wide", ctypes.c_int32), ("tokens", U64), ("vocab", U64)]


def ids(**kw):
    return Ids(**{**dict(ids=A, wide=1, tokens=10, vocab=100), **kw})


@pytest.fixture
def lib(lct_lib):
    lib = lct_lib.library()
    lib.lct_embedding.argtypes = [P, P, U64, ctypes.c_int32, U64, U64, U64, ctypes.c_float, P, U64, P]
    lib.lct_embedding_grad.argtypes = [P, P, U64, ctypes.c_int32, U64, ctypes.c_float, P, U64, P, U64, P, P]
    lib.lct_loss_work_bytes.argtypes = [U64, U64, U64, U64, ctypes.c_int32]
    lib.lct_loss_work_bytes.restype = U64
    lib.lct_loss_forward.argtypes = [P, P, U64, U64, P, U64, U64, U64, P, P, P, P, U64, P]
    lib.lct_loss_backward.argtypes = [P, P, U64, U64, P, U64, U64, U64, P, P, P, U64, P, P, U64, P, U64, P, U64, P]
    return lib


def lookup(lib, i=None, table=X, ldt=64, dtype=0, first=0, rows=100, cols=64, out=OUT, ldo=64):
    i = i or ids()
    return lib.lct_embedding(ctypes.addressof(i), table, ldt, dtype, first, rows, cols, 1.0, out, ldo, None)


def gradient(lib, i=None, dy=X, ldd=64, dtype=0, cols=64, base=None, ldb=64, out=OUT, ldo=64, work=WORK):
    i = i or ids()
    return lib.lct_embedding_grad(ctypes.addressof(i), dy, ldd, dtype, cols, 1.0, base, ldb, out, ldo, work, None)


def forward(lib, i=None, x=X, ldx=64, cols=64, w=B, ldw=64, first=0, rows=100, loss=OUT, lse=OUT + 4096, total=None, work=WORK,
            size=1 << 30):
    i = i or ids()
    return lib.lct_loss_forward(ctypes.addressof(i), x, ldx, cols, w, ldw, first, rows, loss, lse, total, work, size, None)


def backward(lib, i=None, x=X, ldx=64, cols=64, w=B, ldw=64, first=0, rows=100, loss=OUT, lse=OUT + 4096, dloss=OUT + 8192,
             stride=1, scale=None, dx=OUT + 0x100000, ldd=64, dw=OUT + 0x200000, lddw=64, work=WORK, size=1 << 30):
    i = i or ids()
    return lib.lct_loss_backward(ctypes.addressof(i), x, ldx, cols, w, ldw, first, rows, loss, lse, dloss, stride, scale, dx,
                                 ldd, dw, lddw, work, size, None)


@pytest.mark.parametrize("call", [lookup, gradient, forward, backward])
def test_refusals_of_ids(lib, call):
    for kw in (dict(ids=None), dict(ids=A + 4), dict(ids=A + 2, wide=0), dict(wide=2), dict(vocab=0)):
        assert call(lib, ids(**kw)) == INVALID, kw
    for kw in (dict(tokens=2 ** 24 + 1), dict(vocab=2 ** 24 + 1)):
        assert call(lib, ids(**kw)) == UNSUPPORTED, kw
    assert call(lib, cols=0) == INVALID
    assert call(lib, cols=2 ** 16 + 1, **({} if call in (forward, backward) else {})) in (INVALID, UNSUPPORTED)


def test_refusals_of_the_lookup(lib):
    for kw in (dict(table=None), dict(table=X + 1), dict(ldt=63), dict(out=None), dict(out=OUT + 1), dict(ldo=63),
               dict(first=101), dict(first=1), dict(rows=101), dict(out=X), dict(out=X + 64), dict(out=A),
               dict(dtype=1, table=X + 2)):
        assert lookup(lib, **kw) == INVALID, kw
    for kw in (dict(dtype=2), dict(dtype=-1), dict(cols=2 ** 16 + 1, ldt=2 ** 17, ldo=2 ** 17)):
        assert lookup(lib, **kw) == UNSUPPORTED, kw
    assert lookup(lib, ids(tokens=0, ids=None)) == OK


def test_refusals_of_the_lookups_gradient(lib):
    for kw in (dict(dy=None), dict(dy=X + 1), dict(ldd=63), dict(out=None), dict(ldo=63), dict(base=B + 1), dict(base=B, ldb=63),
               dict(out=X), dict(out=A), dict(base=OUT + 2), dict(base=OUT, ldb=128), dict(work=None), dict(work=WORK + 8),
               dict(work=OUT), dict(work=X), dict(base=WORK), dict(work=A)):
        assert gradient(lib, **kw) == INVALID, kw
    assert gradient(lib, dtype=3) == UNSUPPORTED


def test_refusals_of_the_loss(lib):
    for kw in (dict(x=None), dict(x=X + 1), dict(ldx=63), dict(w=None), dict(w=B + 1), dict(ldw=63), dict(first=101),
               dict(rows=0), dict(first=1), dict(loss=None), dict(lse=None), dict(loss=OUT + 2), dict(lse=OUT),
               dict(lse=OUT + 36), dict(loss=X), dict(lse=B), dict(loss=A), dict(work=None), dict(work=WORK + 128),
               dict(work=X - 256), dict(size=100), dict(total=OUT + 2), dict(total=OUT), dict(loss=WORK)):
        assert forward(lib, **kw) == INVALID, kw
    assert forward(lib, cols=2 ** 16 + 1, ldx=2 ** 17, ldw=2 ** 17) == UNSUPPORTED
    assert forward(lib, ids(tokens=0, ids=None)) == OK


def test_refusals_of_the_losss_gradients(lib):
    for kw in (dict(x=None), dict(w=None), dict(ldw=63), dict(first=1), dict(loss=None), dict(lse=None), dict(dloss=None),
               dict(stride=2), dict(scale=OUT + 2), dict(dx=None), dict(dx=OUT + 0x100001), dict(ldd=63), dict(lddw=63),
               dict(dx=X), dict(dw=B), dict(dw=OUT + 0x100000), dict(dx=OUT), dict(dw=OUT + 8192), dict(dx=A), dict(work=X),
               dict(work=B), dict(work=OUT & ~255), dict(size=100), dict(scale=OUT + 0x100000)):
        assert backward(lib, **kw) == INVALID, kw
    assert backward(lib, ids(tokens=0, ids=None), dw=None) == OK


def test_scratch_covers_every_piece(lib):
    """A piece asks for no more than the whole, and what both directions keep between pieces is there."""
    for t, v, k in ((1, 1, 1), (1000, 5003, 1001), (8192, 32_768, 4096), (100_000, 1000, 64)):
        for flags in range(8):
            whole = lib.lct_loss_work_bytes(t, v, k, v, flags)
            piece = lib.lct_loss_work_bytes(t, v, k, max(1, v // 3), flags)
            assert 0 < piece <= whole + (2 * t * ((k + 7) // 8 * 8) + 256 if flags & 1 else 0)
            if flags & 1 and v > 10_000:    # no logits: the scratch is bounded where the vocabulary grows
                assert lib.lct_loss_work_bytes(t, 64 * v, k, 64 * v, flags) < 2 * t * 64 * v
    # the logits of this batch would be 32 GB
    assert lib.lct_loss_work_bytes(65_536, 262_144, 4096, 262_144, 3) < 4 << 30


def test_refusals_of_extents_beyond_any_memory(lib):
    """2^24 rows 2^40 float32 values apart: their bytes pass 64 bits, where every overlap would be missed."""
    wide = ids(vocab=2 ** 24)
    for ld in (2 ** 40, 2 ** 38, 2 ** 30):
        assert lookup(lib, wide, ldt=ld, dtype=1, rows=2 ** 24) == INVALID
        assert gradient(lib, wide, ldo=ld, dtype=1) == INVALID
        assert gradient(lib, wide, base=B, ldb=ld, dtype=1) == INVALID
        assert forward(lib, wide, ldw=ld, rows=2 ** 24) == INVALID
        assert backward(lib, wide, lddw=ld, rows=2 ** 24) == INVALID


def test_scratch_of_sizes_that_are_refused(lib):
    for t, v, k, rows in ((10, 100, 0, 100), (10, 100, 2 ** 16 + 1, 100), (10, 100, 2 ** 64 - 1, 100), (2 ** 24 + 1, 100, 8, 100),
                          (2 ** 64 - 1, 100, 8, 100), (10, 2 ** 24 + 1, 8, 100), (10, 2 ** 64 - 1, 8, 2 ** 64 - 1), (10, 100, 8, 101)):
        for flags in range(8):
            assert lib.lct_loss_work_bytes(t, v, k, rows, flags) == 0


def test_python_refusals(lct_lib):
    torch = pytest.importorskip("torch")
    from lossless_bf16_tensor_gb300 import vocab
    x, w, t = torch.zeros(4, 8, dtype=torch.bfloat16), torch.zeros(16, 8, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.long)
    for call in (lambda: vocab.embedding(t, w), lambda: vocab.embedding_grad(x, t, 16), lambda: vocab.cross_entropy(x, w, t),
                 lambda: vocab.linear_cross_entropy(x, w, t), lambda: vocab.linear_cross_entropy(x, w, t, "median"),
                 lambda: vocab.linear_cross_entropy(x, w[:, :4], t), lambda: vocab.embedding(t, w[0]),
                 lambda: vocab.cross_entropy_grads(x, w, t, t, t, t), lambda: vocab.embedding(None, w)):
        with pytest.raises((ValueError, AttributeError)):
            call()
