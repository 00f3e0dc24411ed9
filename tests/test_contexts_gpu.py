"""Calls from a thread whose current context is its own, not the device's
primary one: the library works in it and leaves it current."""
import ctypes
import threading

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    m.fa_debug_set(0, 0)
    torch.zeros(1, device="cuda")
    return m


def in_own_context(body):
    """body(driver, context) in a thread of its own, in a context made for it; its exception comes out here."""
    drv = ctypes.CDLL("libcuda.so.1")
    failed = []

    def run():
        try:
            ctx = ctypes.c_void_p()
            assert drv.cuCtxCreate_v2(ctypes.byref(ctx), 0, 0) == 0
            try:
                body(drv, ctx.value)
            finally:
                drv.cuCtxDestroy_v2(ctx)
        except BaseException as e:  # noqa: BLE001 (handed to the test's own thread)
            failed.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    if failed:
        raise failed[0]


def current(drv):
    c = ctypes.c_void_p()
    assert drv.cuCtxGetCurrent(ctypes.byref(c)) == 0
    return c.value


P16 = 1 << 20  # never touched: there is nothing to do


def test_a_callers_context_stays_current(fa):
    def body(drv, ctx):
        assert fa.fa_fwd_varlen(0, P16, P16, 0, 0, P16, P16, 1, 2, 2, 0, 8, 64, 128, 128, 128, 0.1, -1, -1, stream=0) == 0
        assert current(drv) == ctx
        assert fa.fa_cache_append(0, 0, P16, P16, P16, P16, P16, 1, 2, 0, 4, 16, 1, 64, 128, 128, stream=0) == 0
        assert current(drv) == ctx
        assert fa.fa_get_status(0) == 0
        assert current(drv) == ctx

    in_own_context(body)


def test_a_thread_without_a_context(fa):
    # its first CUDA call is the library's: the tensors' context becomes current
    q = torch.randn(40, 2, 64, device="cuda").to(torch.bfloat16)
    cu = torch.tensor([0, 40], dtype=torch.int32, device="cuda")
    o, lse = torch.zeros_like(q), torch.zeros(2, 40, device="cuda")
    want = fa.forward_varlen(q, q, q, cu, cu)
    torch.cuda.synchronize()
    got = []
    t = threading.Thread(target=lambda: got.append(
        (fa.fa_fwd_varlen(q, q, q, o, lse, cu, cu, 1, 2, 2, 40, 40, 64, 128, 128, 128, 64 ** -0.5, -1, -1, stream=0),
         fa.fa_get_status(0))))
    t.start()
    t.join()
    assert got == [(0, 0)]
    assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
