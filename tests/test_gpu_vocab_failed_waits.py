"""What a backward pass of the loss leaves after a wait that ran out (made by kernels whose product warps do nothing):
neither gradient may pass for one."""
import ctypes

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_vocab import BF16, loss_bounds, loss_case, within  # noqa: E402
from test_vocab_abi import Ids  # noqa: E402

P, U = ctypes.c_void_p, ctypes.c_uint64


@pytest.fixture(scope="module")
def vocab():
    from lossless_bf16_tensor_gb300 import vocab
    return vocab


def backward(name, case, first, rows, loss, lse, dx, dw, work):
    """lct_loss_backward, or its form whose waits run out, for rows first .. first + rows of the weight."""
    from lossless_bf16_tensor_gb300 import binding as B
    x, w, ids, c = case
    call = getattr(B.library(), name)
    call.argtypes = [P, P, U, U, P, U, U, U, P, P, P, U, P, P, U, P, U, P, U, P]
    arg = Ids(ids.data_ptr(), 1, x.shape[0], w.shape[0])
    piece, out = w[first:first + rows], dw[first:first + rows]
    assert call(ctypes.addressof(arg), x.data_ptr(), x.stride(0), x.shape[1], piece.data_ptr(), w.stride(0), first, rows,
                loss.data_ptr(), lse.data_ptr(), c.data_ptr(), 1, None, dx.data_ptr(), dx.stride(0), out.data_ptr(),
                dw.stride(0), work.data_ptr(), work.numel(), torch.cuda.current_stream().cuda_stream) == B.LCT_OK


GOOD, STALLED = "lct_loss_backward", "lct_debug_loss_backward_timeout"


@pytest.mark.parametrize("t,v,k,pad", [(300, 600, 128, 8), (300, 600, 100, 3), (40, 2000, 64, 8), (2, 300, 72, 0)])
def test_both_gradients_tell(vocab, t, v, k, pad):
    """Tiles written by boxes and by lanes, several a pair of blocks, and what lies beside them."""
    case = loss_case(t, v, k, seed=40)
    x, w, ids, c = case
    loss, lse = vocab.cross_entropy(x, w, ids)
    work = torch.empty(vocab.calls.loss_work_bytes(t, v, k, v, 7), dtype=torch.uint8, device="cuda")
    dx = torch.full((t, k + pad), 2.0, device="cuda", dtype=BF16)
    dw = torch.full((v + 1, k + pad), 2.0, device="cuda", dtype=BF16)
    backward(STALLED, case, 0, v, loss, lse, dx[:, :k], dw[:v, :k], work)
    torch.cuda.synchronize()
    assert dx[:, :k].isnan().all() and dw[:v, :k].isnan().all()
    assert (dx[:, k:] == 2).all() and (dw[:, k:] == 2).all() and (dw[v] == 2).all()
    backward(GOOD, case, 0, v, loss, lse, dx[:, :k], dw[:v, :k], work)        # the next call works
    bounds = loss_bounds(x, w, ids, c)
    within(dx[:, :k], bounds[2], "dx")
    within(dw[:v, :k], bounds[3], "dw")


@pytest.mark.parametrize("bad", [0, 1])
def test_pieces(vocab, bad):
    """A wait that ran out in one of two pieces: dx, and dW from that piece on."""
    t, v, k, half = 300, 1000, 128, 600
    case = loss_case(t, v, k, seed=41)
    x, w, ids, c = case
    loss, lse = vocab.cross_entropy(x, w, ids)
    work = torch.empty(vocab.calls.loss_work_bytes(t, v, k, half, 3), dtype=torch.uint8, device="cuda")
    dx, dw = torch.zeros_like(x), torch.zeros_like(w)
    backward(STALLED if bad == 0 else GOOD, case, 0, half, loss, lse, dx, dw, work)
    backward(STALLED if bad == 1 else GOOD, case, half, v - half, loss, lse, dx, dw, work)
    torch.cuda.synchronize()
    assert dx.isnan().all() and dw[half:].isnan().all()
    if bad == 0:
        assert dw[:half].isnan().all()
    else:
        want, off = loss_bounds(x, w, ids, c)[3]
        within(dw[:half], (want[:half], off[:half]), "dw")
