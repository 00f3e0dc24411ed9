"""Calls on sequences of different lengths at the edges of what fa.h allows."""
import math

import pytest
import torch

from tests import seq_util as su
from tests.test_varlen_gpu import case

pytestmark = pytest.mark.gpu

FA_ERR_INVALID_ARG, FA_ERR_TIMEOUT = 1, 5


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.fa_debug_set(0, 0)
    return m


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("hq,hk,d", [(16, 8, 128), (24, 8, 64)])
def test_items_without_keys_between_others(fa, hq, hk, d):
    # more rows than keys: a CTA's items with key tiles and without follow one another
    g = torch.Generator().manual_seed(d)
    nk = torch.randint(0, 260, (30,), generator=g).tolist()
    nq = [n + int(m) for n, m in zip(nk, torch.randint(0, 500, (30,), generator=g))]
    (q, k, v), cq, ck, seqs = case(nq, nk, hq, hk, d, 40)
    want = su.reference(seqs, d ** -0.5, True)
    c = cq.cuda(), ck.cuda()
    o, lse = fa.forward_varlen(q, k, v, *c, causal=True)
    su.check_forward(o, lse, want, cq)
    for _ in range(20):
        again = fa.forward_varlen(q, k, v, *c, causal=True)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse)
    assert fa.fa_get_status() == 0


def test_a_stream_handle_of_zero_is_the_default_stream(fa, monkeypatch):
    # the default stream's handle is 0: the call has to be made on it, and not on one of the pool's
    (q, k, v), cu, _, _ = case([70, 9], [70, 9], 4, 2, 64, 41)
    c = cu.cuda()
    pages, table, lens = torch.zeros((9, 16, 2, 64), dtype=torch.bfloat16, device="cuda"), i32(0, 1, 2, 3, 4, 5, 6, 7).view(2, 4), i32(64, 9)
    side = torch.cuda.Stream()
    real, seen = fa.lib(), []

    class Recorder:  # the library's calls, each with its stream (the last argument) noted; nothing runs
        def __getattr__(self, name):
            return lambda *args: seen.append((name, args[-1] or 0)) or 0

    def calls(stream):
        o, lse = fa.forward_varlen(q, k, v, c, c, stream=stream)
        fa.backward_varlen(q, k, v, o, lse, q.contiguous(), c, c, stream=stream)
        fa.forward_paged(q, pages, pages, c, lens, table, stream=stream)
        fa.cache_append(k, v, pages, pages, c, lens, table, stream=stream)

    monkeypatch.setattr(fa, "lib", lambda: Recorder())
    for current in (torch.cuda.default_stream(), side):
        with torch.cuda.stream(current):
            for given in (0, torch.cuda.default_stream(), side.cuda_stream, side):
                seen.clear()
                calls(given)
                want = given if isinstance(given, int) else given.cuda_stream
                assert [h for _, h in seen] == [want] * 4, (current, given, seen)
                assert torch.cuda.current_stream() == current
    monkeypatch.setattr(fa, "lib", lambda: real)
    want = fa.forward_varlen(q, k, v, c, c)
    got = fa.forward_varlen(q, k, v, c, c, stream=0)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and fa.fa_get_status() == 0


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("new,keys,left", [([1] * 5, [900, 300, 131, 40, 1], 100), ([1, 200, 33], [3000, 1500, 640], 257),
                                           ([1], [20011], 1000), ([5, 0, 300], [4, 700, 301], 0)])
@pytest.mark.parametrize("freed", [-1, "nan"])
def test_pages_behind_the_window_may_be_gone(fa, page, new, keys, left, freed):
    # pages that the window hides whole from all new tokens: their entries name no page, or one of NaN
    hq, hk, d = 8, 2, 64
    g = su.gen(42)
    ks, vs = ([su.normal((n, hk, d), g) for n in keys] for _ in range(2))
    c = su.Cache(ks, vs, page, 43)
    spare = c.ids[-1]
    assert torch.isnan(c.k[spare].float()).all()
    for b, (n, m) in enumerate(zip(new, keys)):
        first = m - n - left if n else m
        for p in range(max(0, first) // page):
            c.k[c.table[b, p]] = c.v[c.table[b, p]] = math.nan
            c.table[b, p] = -1 if freed == -1 else spare
    c.cuda()
    q, cu = su.normal((sum(new), hq, d), g), su.starts(new)
    o, lse = fa.forward_paged(q.cuda(), c.k, c.v, cu.cuda(), c.lens, c.table, window=(left, 0))
    assert fa.fa_get_status() == 0
    seqs = [(q[cu[b]:cu[b + 1]], ks[b], vs[b]) for b in range(len(new))]
    su.check_forward(o, lse, su.reference(seqs, d ** -0.5, True, (left, 0)), cu)
