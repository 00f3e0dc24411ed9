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


def test_each_context_has_its_own_status_word(fa):
    # appending and a small forward in a context of the caller's, with memory of that context;
    # a wrong length there is reported there
    torch.manual_seed(1)
    hk, d, page, n = 2, 64, 16, 5
    k, v, q = (torch.randn(n, h, d).to(torch.bfloat16) for h in (hk, hk, 4))
    want = fa.forward_varlen(*(x.cuda() for x in (q, k, v)), *[torch.tensor([0, n], dtype=torch.int32, device="cuda")] * 2)
    want = [x.cpu() for x in want]
    assert fa.fa_get_status() == 0

    def body(drv, ctx):
        drv.cuMemAlloc_v2.argtypes = [ctypes.c_void_p, ctypes.c_size_t]
        drv.cuMemcpyHtoD_v2.argtypes = [ctypes.c_uint64, ctypes.c_void_p, ctypes.c_size_t]
        drv.cuMemcpyDtoH_v2.argtypes = [ctypes.c_void_p, ctypes.c_uint64, ctypes.c_size_t]

        def put(t):
            p = ctypes.c_uint64()
            assert drv.cuMemAlloc_v2(ctypes.byref(p), t.numel() * t.element_size()) == 0
            assert drv.cuMemcpyHtoD_v2(p.value, t.data_ptr(), t.numel() * t.element_size()) == 0
            return p.value

        def get(p, like):
            t = torch.empty_like(like)
            assert drv.cuMemcpyDtoH_v2(t.data_ptr(), p, t.numel() * t.element_size()) == 0
            return t

        pages = torch.full((3, page, hk, d), 7.0, dtype=torch.bfloat16)
        dq, dk, dv, kp, vp, o = (put(x) for x in (q, k, v, pages, pages, torch.zeros_like(q)))
        lse, cu = put(torch.zeros(4, n)), put(torch.tensor([0, n], dtype=torch.int32))
        table, good, bad = (put(torch.tensor(x, dtype=torch.int32)) for x in ([2], [n], [n - 1]))

        def append(lens):
            return fa.fa_cache_append(dk, dv, kp, vp, cu, lens, table, 1, hk, n, 3, page, 1, d, hk * d, hk * d, stream=0)

        assert append(bad) == 0 and fa.fa_get_status(0) == 1
        assert torch.equal(get(kp, pages), pages)
        assert append(good) == 0 and fa.fa_get_status(0) == 0
        got = get(kp, pages)
        assert torch.equal(got[2, :n], k) and (got[:2] == 7).all() and (got[2, n:] == 7).all()
        assert fa.fa_fwd_varlen(dq, dk, dv, o, lse, cu, cu, 1, 4, hk, n, n, d, 4 * d, hk * d, hk * d, d ** -0.5, -1, -1,
                                stream=0) == 0
        assert fa.fa_get_status(0) == 0 and current(drv) == ctx
        assert torch.equal(get(o, want[0]), want[0]) and torch.equal(get(lse, want[1]), want[1])

    in_own_context(body)
    assert fa.fa_get_status() == 0
