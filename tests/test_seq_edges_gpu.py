"""Calls on sequences of different lengths at the edges of what fa.h allows."""
import math
import random

import pytest
import torch

from tests import seq_util as su
from tests import test_varlen_bwd_gpu as backward
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


def long_units(B, top, seed):
    """B sequences of one token over 1030 to `top` key tiles each, their pages taken from one small pool."""
    rng = random.Random(seed)
    tiles = [rng.randint(1030, top) for _ in range(B)]
    g = torch.Generator(device="cuda").manual_seed(seed)
    kp, vp = (torch.randn(64, 256, 1, 64, device="cuda", generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(B, 4, 64, device="cuda", generator=g).to(torch.bfloat16)
    table = torch.randint(0, 64, (B, top // 2 + 1), device="cuda", generator=g).to(torch.int32)
    return q, kp, vp, su.starts([1] * B).cuda(), i32(*(128 * n - 5 for n in tiles)), table


@pytest.mark.parametrize("B,top", [(456, 1400), (700, 1400), (1300, 1200)])
def test_same_bits_where_units_are_longer_than_the_sort_tells_apart(fa, B, top):
    # The plan sorts its units by their tiles, in a table of 1024 lengths. Whole or divided is decided by the
    # sorted order's busiest worker, and here that lies at the border: any change of order among
    # the longest would decide otherwise now and then, and divided units round otherwise.
    # (1300 units are more than the plan keeps in shared memory.)
    a = long_units(B, top, B * 7 + top)
    o, lse = fa.forward_paged(*a)
    q, kp, vp, cu, lens, table = a
    for b in (0, B // 2, B - 1):
        keys = table[b].long()
        seq = [q[b:b + 1].cpu()] + [x[keys].reshape(-1, 1, 64)[:int(lens[b])].cpu() for x in (kp, vp)]
        # (a stage's row sum takes an add to each of its 700 tiles and some 32 within one: below 2^-14)
        su.check_forward(o[b:b + 1], lse[:, b:b + 1], su.reference([seq], 64 ** -0.5, True), [0, 1])
    junk = torch.empty(1 << 26, device="cuda")
    for i in range(60):
        if i % 3 == 0:
            junk.zero_()  # other lines in the caches, other times of arrival
        again = fa.forward_paged(*a)
        assert torch.equal(again[0], o) and torch.equal(again[1], lse), i
    assert fa.fa_get_status() == 0


def test_gradients_of_more_row_tiles_than_the_sort_tells_apart(fa):
    # 128 query heads to a kv head: a token is a row tile
    a, b = (backward.run(fa, [1100], [300], 128, 1, 64, seed=44, causal=False) for _ in range(2))
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])


def test_append_reports_every_wrong_length(fa):
    # also those that no token's own sequence shows: offsets out of order, a sequence without new tokens
    hk, d, page, total, B = 2, 64, 16, 8, 600
    g = su.gen(45)
    k, v = (su.normal((total, hk, d), g).cuda() for _ in range(2))
    start = su.normal((3, page, hk, d), g).cuda()
    table = i32(0, 1, 2).view(3, 1)

    def run(cu, lens, table):
        kp, vp = start.clone(), start.clone()
        fa.cache_append(k, v, kp, vp, cu, lens, table)
        return fa.fa_get_status(), kp, vp

    for cu, lens in ((i32(0, 5, 3, 8), i32(5, 5, 5)), (i32(0, 0, 8, 8), i32(-1, 8, 3)), (i32(0, 8, 8, 8), i32(8, 4, 17)),
                     (i32(0, 8, 8, 9), i32(8, 4, 4)), (i32(-2, 0, 8, 8), i32(2, 8, 4))):
        st, kp, vp = run(cu, lens, table)
        assert st == FA_ERR_INVALID_ARG, (cu, lens)
    # the right sequence among them is written, and nothing else
    st, kp, vp = run(i32(0, 0, 8, 8), i32(-1, 8, 3), table)
    for got, x in ((kp, k), (vp, v)):
        want = start.clone()
        want[1, :8] = x
        assert torch.equal(got, want)
    # more sequences than a block looks over
    many = torch.zeros((B, 1), dtype=torch.int32, device="cuda")
    cu, lens = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.full((B,), 3, dtype=torch.int32, device="cuda")
    cu[1:], lens[0] = total, total
    assert run(cu, lens, many)[0] == 0
    for at in (1, 223, 224, 255, 256, 448, B - 1):
        bad = lens.clone()
        bad[at] = page + 1
        assert run(cu, bad, many)[0] == FA_ERR_INVALID_ARG, at
    assert run(cu, lens, many)[0] == 0


@pytest.mark.parametrize("lens,hq,hk,d", [([300], 2, 1, 128), ([40, 700, 0, 129], 16, 8, 64)])
def test_a_wait_of_the_backward_that_runs_out_is_reported(fa, lens, hq, hk, d):
    # the producer never delivers a tile of Q: every wait is bounded, the call ends with a status,
    # and the next one is as ever
    run = lambda: backward.run(fa, lens, lens, hq, hk, d, seed=46)  # noqa: E731
    a = run()
    (q, k, v), cu, _, _ = case(lens, lens, hq, hk, d, 46)
    c = cu.cuda()
    o, lse = fa.forward_varlen(q, k, v, c, c, causal=True)
    assert fa.fa_get_status() == 0
    assert fa.fa_debug_set(20_000_000, 1) == 0
    try:
        fa.backward_varlen(q, k, v, o, lse, o, c, c, causal=True)
        assert fa.fa_get_status() == FA_ERR_TIMEOUT
    finally:
        fa.fa_debug_set(0, 0)
    b = run()
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
