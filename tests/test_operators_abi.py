"""Host-side checks of the gradient and adapter calls (no GPU): every call here
is refused, or has nothing to do, before anything is enqueued."""
import ctypes

import pytest

OK, INVALID, UNSUPPORTED = 0, 1, 2
P = ctypes.c_void_p
U64 = ctypes.c_uint64


class Bank(ctypes.Structure):
    _fields_ = [("a", P), ("b", P), ("scale", P), ("ranks", P), ("adapters", U64), ("rank", U64), ("k", U64), ("n", U64)]


class Plan(ctypes.Structure):
    _fields_ = [("order", P), ("starts", P), ("tiles", P), ("tokens", U64), ("adapters", U64)]


A, X, Y, OUT, WORK = (0x10000000 * i for i in range(1, 6))  # addresses that nobody reads


def bank(**kw):
    d = dict(a=A, b=A + 0x100000, scale=A + 0x200000, ranks=None, adapters=3, rank=16, k=64, n=128)
    return Bank(**{**d, **kw})


def plan(**kw):
    return Plan(**{**dict(order=A + 0x300000, starts=A + 0x310000, tiles=A + 0x320000, tokens=10, adapters=3), **kw})


@pytest.fixture
def lib(lct_lib):
    lib = lct_lib.library()
    lib.lct_grad_norm.argtypes = [P, P, P, U64, P, P, P]
    lib.lct_grad_clip.argtypes = [P, P, P, P, U64, ctypes.c_float, P, P, P]
    lib.lct_adapter_plan.argtypes = [P, U64, U64, P, P, P, P]
    lib.lct_adapter_forward.argtypes = [P, P, P, U64, P, U64, P, U64, P, P]
    lib.lct_adapter_backward.argtypes = [P, P, P, U64, P, U64, P, P, U64, P, U64, P, P, P, P]
    return lib


def arrays(ptrs, n, dtype):
    return (P * len(ptrs))(*ptrs), (U64 * len(n))(*n), (ctypes.c_int32 * len(dtype))(*dtype)


def clip(lib, src, dst, n, dtype, max_norm=1.0, norm=X, work=WORK):
    s, sizes, types = arrays(src, n, dtype)
    d = (P * len(dst))(*dst)
    return lib.lct_grad_clip(s, d, sizes, types, len(src), max_norm, norm, work, None)


def test_gradient_refusals(lib):
    s, n, t = arrays([A], [8], [0])
    norm = lambda *a: lib.lct_grad_norm(*a, None)  # noqa: E731
    assert norm(s, n, t, 1, None, WORK) == INVALID
    assert norm(s, n, t, 1, X + 2, WORK) == INVALID
    assert norm(s, n, t, 1, X, None) == INVALID
    assert norm(s, n, t, 1, X, WORK + 8) == INVALID
    assert norm(None, n, t, 1, X, WORK) == INVALID
    for ptr, size, kind, want in ((None, 8, 0, INVALID), (A + 1, 8, 0, INVALID), (A + 2, 8, 1, INVALID),
                                  (A, 2 ** 40 + 1, 0, INVALID), (A, 8, 2, UNSUPPORTED), (A, 8, -1, UNSUPPORTED)):
        s, n, t = arrays([ptr], [size], [kind])
        assert norm(s, n, t, 1, X, WORK) == want
        assert clip(lib, [ptr], [OUT], [size], [kind]) == want
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert clip(lib, [A], [A], [8], [0], bad) == INVALID
    # outputs over one another, over another gradient, half over their own
    assert clip(lib, [A, A + 64], [OUT, OUT + 8], [8, 8], [0, 0]) == INVALID
    assert clip(lib, [A, A + 64], [A + 64, OUT], [8, 8], [0, 0]) == INVALID
    assert clip(lib, [A], [A + 8], [8], [0]) == INVALID
    assert clip(lib, [A, A], [A, A], [8, 8], [0, 0]) == INVALID
    assert clip(lib, [A + 512, A], [OUT + 512, A + 520], [8, 8], [0, 0]) == INVALID
    assert clip(lib, [A], [None], [8], [0]) == INVALID


def forward(lib, b=None, p=None, x=X, ldx=64, y=Y, ldy=128, out=OUT, ldo=128, xa=None):
    b, p = b or bank(), p or plan()
    return lib.lct_adapter_forward(ctypes.addressof(b), ctypes.addressof(p), x, ldx, y, ldy, out, ldo, xa, None)


def backward(lib, b=None, p=None, dy=Y, ldy=128, x=X, ldx=64, xa=X + 0x100000, dx=OUT, ldd=64, out=OUT, ldo=64,
             da=OUT + 0x100000, db=OUT + 0x200000, work=WORK):
    b, p = b or bank(), p or plan()
    return lib.lct_adapter_backward(ctypes.addressof(b), ctypes.addressof(p), dy, ldy, x, ldx, xa, dx, ldd, out, ldo, da,
                                    db, work, None)


@pytest.mark.parametrize("call", [forward, backward])
def test_bank_and_plan_refusals(lib, call):
    for kw in (dict(a=None), dict(b=None), dict(scale=None), dict(a=A + 1), dict(scale=A + 2), dict(ranks=A + 2),
               dict(adapters=0), dict(rank=0), dict(k=0), dict(n=0), dict(adapters=4)):
        assert call(lib, b=bank(**kw)) == INVALID, kw
    for kw in (dict(rank=129), dict(k=2 ** 20 + 1), dict(n=2 ** 20 + 1)):
        assert call(lib, b=bank(**kw)) == UNSUPPORTED, kw
    assert call(lib, b=bank(adapters=16_385), p=plan(adapters=16_385)) == UNSUPPORTED
    for kw in (dict(order=None), dict(starts=None), dict(tiles=None), dict(tiles=A + 0x320008), dict(order=A + 2),
               dict(adapters=2)):
        assert call(lib, p=plan(**kw)) == INVALID, kw
    assert call(lib, p=plan(tokens=2 ** 24 + 1)) == UNSUPPORTED
    assert lib.lct_adapter_forward(None, None, X, 64, Y, 128, OUT, 128, None, None) == INVALID


def test_forward_refusals(lib):
    for kw in (dict(x=None), dict(y=None), dict(out=None), dict(x=X + 1), dict(ldx=63), dict(ldy=127), dict(ldo=127),
               dict(xa=OUT + 0x100002),
               dict(out=X), dict(out=Y + 2), dict(out=Y, ldo=256), dict(out=A), dict(out=A + 0x300000),
               dict(xa=X), dict(xa=OUT), dict(xa=A + 0x320000)):
        assert forward(lib, **kw) == INVALID, kw
    assert forward(lib, p=plan(tokens=0, order=None)) == OK


def test_backward_refusals(lib):
    for kw in (dict(dy=None), dict(x=None), dict(xa=None), dict(dx=None), dict(work=None), dict(work=WORK + 8),
               dict(da=None), dict(db=None), dict(da=None, db=None, out=None), dict(ldy=100), dict(ldo=63),
               dict(out=X), dict(out=Y), dict(out=OUT + 2), dict(da=Y), dict(db=OUT + 0x100000), dict(work=OUT),
               dict(da=A), dict(work=X + 0x100000), dict(out=X + 0x100000)):
        assert backward(lib, **kw) == INVALID, kw


def test_plan_refusals(lib):
    good = [X, 10, 3, Y, Y + 0x1000, OUT, None]
    for at, value, want in ((0, None, INVALID), (3, None, INVALID), (4, None, INVALID), (5, None, INVALID),
                            (0, X + 2, INVALID), (5, OUT + 8, INVALID), (2, 0, INVALID), (2, 16_385, UNSUPPORTED),
                            (1, 2 ** 24 + 1, UNSUPPORTED), (3, X, INVALID), (4, Y + 8, INVALID), (5, X, INVALID)):
        args = list(good)
        args[at] = value
        assert lib.lct_adapter_plan(*args) == want, (at, value)
