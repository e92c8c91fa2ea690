"""Calls of several host threads at once, each on its own stream and operands: kernels whose shared memory goes by the
call's sizes."""
import ctypes
import threading

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_vocab_abi import P, U64, Ids  # noqa: E402

ROUNDS = 1500


def together(bodies):
    """Runs each body in a thread of its own, ROUNDS times; the statuses that they returned."""
    gate, seen = threading.Barrier(len(bodies)), [set() for _ in bodies]

    def run(i):
        gate.wait()
        for _ in range(ROUNDS):
            seen[i].add(bodies[i]())

    threads = [threading.Thread(target=run, args=(i,)) for i in range(len(bodies))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    return seen


def test_losses_of_one_token_of_several_widths(lct_lib):
    """x is held in shared memory: 40 KB and 96 KB of it."""
    lib = lct_lib.library()
    lib.lct_loss_work_bytes.argtypes = [U64, U64, U64, U64, ctypes.c_int32]
    lib.lct_loss_work_bytes.restype = U64
    lib.lct_loss_forward.argtypes = [P, P, U64, U64, P, U64, U64, U64, P, P, P, P, U64, P]
    from lossless_bf16_tensor_gb300 import vocab
    gen = torch.Generator(device="cuda").manual_seed(1)
    bodies, results = [], []
    for k in (20_480, 49_152):
        x, w = (torch.randn(n, k, generator=gen, device="cuda").to(torch.bfloat16) for n in (1, 16))
        ids = torch.tensor([3], device="cuda")
        size = lib.lct_loss_work_bytes(1, 16, k, 16, 0)
        work, out = torch.empty(size, dtype=torch.uint8, device="cuda"), torch.zeros(2, 64, device="cuda")
        arg, stream = Ids(ids.data_ptr(), 1, 1, 16), torch.cuda.Stream()
        results.append((out, vocab.cross_entropy(x, w, ids), (x, w, ids, work, arg, stream)))

        def body(k=k, x=x, w=w, work=work, size=size, out=out, arg=arg, stream=stream):
            return lib.lct_loss_forward(ctypes.addressof(arg), x.data_ptr(), k, k, w.data_ptr(), k, 0, 16, out[0].data_ptr(),
                                        out[1].data_ptr(), None, work.data_ptr(), size, stream.cuda_stream)
        bodies.append(body)
    torch.cuda.synchronize()
    assert together(bodies) == [{0}, {0}]
    for out, (loss, lse), _ in results:
        assert torch.equal(out[0, :1], loss) and torch.equal(out[1, :1], lse)


def test_sorting_for_tables_of_several_sizes(lct_lib):
    """Digits of 8 and of 9 bits: counters of 33 KB and of 66 KB."""
    lib = lct_lib.library()
    lib.lct_embedding_grad.argtypes = [P, P, U64, ctypes.c_int32, U64, ctypes.c_float, P, U64, P, U64, P, P]
    from lossless_bf16_tensor_gb300 import vocab
    gen = torch.Generator(device="cuda").manual_seed(2)
    t, k, bodies, results = 9000, 8, [], []
    for v in (60_000, 200_000):
        ids = torch.randint(0, v, (t,), generator=gen, device="cuda")
        dy = torch.randn(t, k, generator=gen, device="cuda").to(torch.bfloat16)
        out = torch.zeros(v, k, device="cuda", dtype=torch.bfloat16)
        chunks, part = (t + 31) // 32, (k + 14) // 8 * 8
        work = torch.empty(16 + 64 * ((t + 3) // 4) + 8 * chunks * part, dtype=torch.uint8, device="cuda")
        arg, stream = Ids(ids.data_ptr(), 1, t, v), torch.cuda.Stream()
        results.append((out, vocab.embedding_grad(dy, ids, v), (dy, ids, work, arg, stream)))

        def body(dy=dy, out=out, work=work, arg=arg, stream=stream):
            return lib.lct_embedding_grad(ctypes.addressof(arg), dy.data_ptr(), k, 0, k, 1.0, None, k, out.data_ptr(), k,
                                          work.data_ptr(), stream.cuda_stream)
        bodies.append(body)
    torch.cuda.synchronize()
    assert together(bodies) == [{0}, {0}]
    for out, want, _ in results:
        assert torch.equal(out, want)
