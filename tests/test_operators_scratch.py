"""Host-side checks (no GPU): the norm and the scratch of the gradient calls lie
apart from each other and from every gradient and output.  Every call here is
refused before anything is enqueued."""
import ctypes

import pytest
from test_operators_abi import INVALID, U64, P

WORK_BYTES = 4896
G, OUT, NORM, WORK = (0x10000000 * i for i in range(1, 5))  # addresses that nobody reads


@pytest.fixture
def lib(lct_lib):
    lib = lct_lib.library()
    lib.lct_grad_norm.argtypes = [P, P, P, U64, P, P, P]
    lib.lct_grad_clip.argtypes = [P, P, P, P, U64, ctypes.c_float, P, P, P]
    return lib


def call(lib, src, n, dtype, norm, work, dst=None):
    def arr(kind, v):
        return (kind * len(v))(*v)
    args = [arr(U64, n), arr(ctypes.c_int32, dtype), len(src)]
    if dst is None:
        return lib.lct_grad_norm(arr(P, src), *args, norm, work, None)
    return lib.lct_grad_clip(arr(P, src), arr(P, dst), *args, 1.0, norm, work, None)


@pytest.mark.parametrize("dtype,size", [(0, 2), (1, 4)])
def test_scratch_and_norm_over_tensors(lib, dtype, size):
    n = 1000
    for norm, work in ((G, WORK), (G + n * size - 4, WORK), (G + 400, WORK), (NORM, G), (NORM, G - WORK_BYTES + 16),
                       (NORM, G + 16), (WORK, WORK), (WORK + WORK_BYTES - 4, WORK)):
        assert call(lib, [G], [n], [dtype], norm, work) == INVALID
        assert call(lib, [G], [n], [dtype], norm, work, dst=[G]) == INVALID
        # behind a tensor that is fine, and a tensor of no values, whose address says nothing
        assert call(lib, [G + 0x1000000, 0, G], [8, 0, n], [dtype] * 3, norm, work) == INVALID
    for norm, work in ((OUT, WORK), (OUT + n * size - 4, WORK), (NORM, OUT + 32), (NORM, OUT - 16)):
        assert call(lib, [G], [n], [dtype], norm, work, dst=[OUT]) == INVALID
