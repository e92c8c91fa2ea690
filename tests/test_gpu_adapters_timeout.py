"""Waits that run out in the adapters' kernels: product warps that do nothing, so
that every wait for a product gives up after about a second.  The kernels end,
the plan's status says so, and the next call works."""
import ctypes

import pytest
import torch

from lossless_bf16_tensor_gb300 import binding as B
from lossless_bf16_tensor_gb300.adapters import adapter_plan
from test_gpu_adapters import Case, both
from test_operators_abi import U64, Bank, P, Plan

pytestmark = pytest.mark.gpu


def operands(c):
    bank = Bank(c.a.data_ptr(), c.b.data_ptr(), c.scale.data_ptr(), None, c.n, c.r, c.k, c.m)
    plan = Plan(c.plan.order.data_ptr(), c.plan.starts.data_ptr(), c.plan.tiles.data_ptr(), c.t, c.n)
    return bank, plan


# one tile and clusters; several tiles a cluster; rows at 16-byte boundaries and at others; above rank 64
@pytest.mark.parametrize("t,n,r,k,m", [(300, 2, 16, 1024, 512), (300, 2, 16, 1001, 515), (200, 1, 72, 512, 512),
                                       (9000, 2, 8, 64, 128)])
def test_waits_that_run_out(t, n, r, k, m):
    c = Case(t, n, r, k, m, seed=t, index=[i % n for i in range(t)])
    both(c)
    lib = B.library()
    stream = torch.cuda.current_stream().cuda_stream
    bank, plan = operands(c)
    out, xa = torch.empty_like(c.y), torch.empty(t, r, device="cuda")
    call = lib.lct_debug_adapter_forward_timeout
    call.argtypes = [P, P, P, U64, P, U64, P, U64, P, P]
    assert call(ctypes.addressof(bank), ctypes.addressof(plan), c.x.data_ptr(), k, c.y.data_ptr(), m, out.data_ptr(), m,
                xa.data_ptr(), stream) == B.LCT_OK
    torch.cuda.synchronize()
    assert c.plan.status() == B.LCT_ERR_TIMEOUT

    c.plan = adapter_plan(c.index, n)
    bank, plan = operands(c)
    xa.zero_()
    dx, da, db = torch.empty_like(c.dx), torch.empty_like(c.a), torch.empty_like(c.b)
    work = torch.empty(8 * t * ((r + 15) // 16 * 16), dtype=torch.uint8, device="cuda")
    call = lib.lct_debug_adapter_backward_timeout
    call.argtypes = [P, P, P, U64, P, U64, P, P, U64, P, U64, P, P, P, P]
    assert call(ctypes.addressof(bank), ctypes.addressof(plan), c.dy.data_ptr(), m, c.x.data_ptr(), k, xa.data_ptr(),
                c.dx.data_ptr(), k, dx.data_ptr(), k, da.data_ptr(), db.data_ptr(), work.data_ptr(), stream) == B.LCT_OK
    torch.cuda.synchronize()
    assert c.plan.status() == B.LCT_ERR_TIMEOUT

    c.plan = adapter_plan(c.index, n)
    both(c)
