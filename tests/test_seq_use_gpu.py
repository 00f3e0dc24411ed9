"""The packed and paged calls as programs use them: a serving loop, captured
graphs, several streams, other sequences' bits, lengths and pages that are
wrong, offsets past 32 bits, a wait that runs out."""
import math
import threading

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


def test_serving_loop_as_the_whole_prompt(fa):
    # two prompts go into the cache in chunks, then token by token; at every
    # step the new rows are those of the causal attention of the whole
    hq, hk, d, page, total = 8, 2, 128, 32, [230, 75]
    g = su.gen(1)
    q, k, v = ([su.normal((n, h, d), g) for n in total] for h in (hq, hk, hk))
    want = su.reference(list(zip(q, k, v)), d ** -0.5, True)
    kp = torch.full((20, page, hk, d), math.nan, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    table = torch.randperm(20, generator=g).to(torch.int32)[:16].view(2, 8).cuda()
    done = [0, 0]
    for new in ([100, 70], [125, 0], [1, 1], [1, 1], [1, 1], [2, 1], [0, 1]):
        cu = su.starts(new)
        rows = [(b, done[b], done[b] + n) for b, n in enumerate(new)]
        part = [torch.cat([x[b][s:e] for b, s, e in rows]).cuda() for x in (q, k, v)]
        done = [e for _, _, e in rows]
        lens = i32(*done)
        fa.cache_append(part[1], part[2], kp, vp, cu.cuda(), lens, table)
        o, lse = fa.forward_paged(part[0], kp, vp, cu.cuda(), lens, table)
        assert fa.fa_get_status() == 0
        su.check_forward(o, lse, [(want[b][0][s:e], want[b][1][:, s:e], want[b][2][s:e]) for b, s, e in rows], cu)
    assert done == total


def test_other_sequences_bits_do_not_matter(fa):
    # a sequence of NaN and infinities between two others: theirs are unchanged, bit for bit
    n, hq, hk, d = [200, 90, 333], 4, 2, 128
    (q, k, v), cu, _, _ = case(n, n, hq, hk, d, 2)
    do = su.normal((sum(n), hq, d), su.gen(3)).cuda()
    c = cu.cuda()

    def run():
        o, lse = fa.forward_varlen(q, k, v, c, c, causal=True)
        return (o, lse) + tuple(fa.backward_varlen(q, k, v, o, lse, do, c, c, causal=True))

    clean = run()
    for t in (q, k, v, do):
        t[200:290] = math.nan
        t[200:290:3] = math.inf
    dirty = run()
    assert fa.fa_get_status() == 0
    keep = torch.cat([torch.arange(200), torch.arange(290, sum(n))]).cuda()
    for name, a, b in zip(("o", "lse", "dq", "dk", "dv"), clean, dirty):
        a, b = (x[:, keep] if name == "lse" else x[keep] for x in (a, b))
        if name == "dq":  # its additions are not ordered: at most a few bf16 steps apart
            a, b = a.double(), b.double()
            assert torch.isfinite(b).all() and ((a - b).abs() <= 2.0 ** -6 * a.abs() + 2.0 ** -10 * a.abs().max()).all()
        else:
            assert torch.equal(a, b), name


def test_same_call_same_bits(fa):
    for nq, nk in (([64], [5000]), ([300, 1, 40], [3000, 900, 40])):  # keys divided between CTAs
        (q, k, v), cq, ck, _ = case(nq, nk, 4, 1, 128, 4)
        a, b = (fa.forward_varlen(q, k, v, cq.cuda(), ck.cuda(), causal=True) for _ in range(2))
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_replays_with_other_lengths(fa):
    # captured once; the lengths, offsets and pages of each replay are its own
    hq, hk, d, page, B, total = 8, 2, 64, 16, 4, 600
    g = su.gen(5)
    q, k, v, do = (su.normal((total, h, d), g).cuda() for h in (hq, hk, hk, hq))
    kp, vp = (su.normal((200, page, hk, d), g).cuda() for _ in range(2))
    table = torch.randperm(200, generator=g).to(torch.int32)[:B * 45].view(B, 45).cuda()
    cu, lens = su.starts([100, 200, 1, 250]).cuda(), i32(100, 300, 700, 250)
    outs = [torch.zeros(s, device="cuda", dtype=torch.bfloat16) for s in (q.shape, q.shape, q.shape, k.shape, k.shape)]
    lses = [torch.zeros((hq, total), device="cuda") for _ in range(2)]

    def step():
        fa.cache_append(k, v, kp, vp, cu, lens, table)
        fa.forward_paged(q, kp, vp, cu, lens, table, out=(outs[0], lses[0]))
        fa.forward_varlen(q, k, v, cu, cu, causal=True, out=(outs[1], lses[1]))
        fa.backward_varlen(q, k, v, outs[1], lses[1], do, cu, cu, causal=True, out=outs[2:])

    step()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    pages = kp.clone(), vp.clone()
    for new, keys in (([100, 200, 1, 250], [100, 300, 700, 250]), ([1, 1, 1, 1], [5, 640, 17, 300]),
                      ([0, 600, 0, 0], [10, 600, 0, 9])):
        cu.copy_(su.starts(new))
        lens.copy_(i32(*keys))
        got = []
        for run in (graph.replay, step):
            kp.copy_(pages[0])
            vp.copy_(pages[1])
            for t in outs + lses:
                t.fill_(5.0)
            run()
            assert fa.fa_get_status() == 0
            got.append([t.clone() for t in outs + lses + [kp, vp]])
        for i, (a, b) in enumerate(zip(*got)):
            if i == 2:  # dQ
                assert ((a.double() - b.double()).abs() <= 2.0 ** -6 * b.double().abs() + 2.0 ** -10 * 5).all()
            else:
                assert torch.equal(a, b), i


def test_two_graphs_and_two_threads_at_once(fa):
    # calls on two streams at once, captured and eager: each has a workspace of its own
    cases = []
    for seed, nq, nk in ((6, [300, 50], [3000, 4000]), (7, [40, 500], [5000, 500])):
        (q, k, v), cq, ck, _ = case(nq, nk, 4, 1, 128, seed)
        cases.append((q, k, v, cq.cuda(), ck.cuda()))
    want = [fa.forward_varlen(*c, causal=True) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    graphs, outs = [], []
    for c, s in zip(cases, streams):
        out = (torch.zeros_like(c[0]), torch.zeros((4, c[0].shape[0]), device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                fa.forward_varlen(*c, causal=True, out=out)
        graphs.append(g)
        outs.append(out)
    torch.cuda.synchronize()
    for _ in range(20):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for out, w in zip(outs, want):
        assert torch.equal(out[0], w[0]) and torch.equal(out[1], w[1])
    bad, rounds = [], []

    def loop(c, s, w):  # (a thread's first CUDA call may be the library's)
        for _ in range(30):
            o, lse = fa.forward_varlen(*c, causal=True, stream=s)
            s.synchronize()
            rounds.append(1)
            if not (torch.equal(o, w[0]) and torch.equal(lse, w[1])):
                bad.append(s)

    threads = [threading.Thread(target=loop, args=a) for a in zip(cases, streams, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad and len(rounds) == 60 and fa.fa_get_status() == 0


def test_stream_handles(fa):
    (q, k, v), cu, _, _ = case([70, 9], [70, 9], 4, 2, 64, 8)
    c = cu.cuda()
    want = fa.forward_varlen(q, k, v, c, c)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        o, lse = fa.forward_varlen(q, k, v, c, c, stream=handle)
        s.synchronize()
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("many", [False, True])
def test_wrong_lengths_change_nothing(fa, many):
    # (many: more sequences than the self-planned path takes)
    n = [30] * (200 if many else 3)
    (q, k, v), cu, _, _ = case(n, n, 4, 2, 64, 9)
    good = cu.cuda()
    bad = []
    for at, value in ((1, -1), (2, 29), (len(n), sum(n) + 1), (0, -5)):
        x = cu.clone()
        x[at] = value
        bad.append((x.cuda(), good))
        bad.append((good, x.cuda()))
    twice = torch.tensor([0, sum(n)] * len(n), dtype=torch.int32)[:len(n) + 1]  # overlapping: 0, T, 0, T, ...
    bad.append((twice.cuda(), good))
    o, lse = torch.full_like(q, 3.0), torch.full((4, q.shape[0]), 3.0, device="cuda")
    grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
    assert fa.fa_get_status() == 0
    for cq, ck in bad:
        fa.forward_varlen(q, k, v, cq, ck, out=(o, lse))
        assert fa.fa_get_status() == FA_ERR_INVALID_ARG
        fa.backward_varlen(q, k, v, o, lse, q, cq, ck, out=grads)
        assert fa.fa_get_status() == FA_ERR_INVALID_ARG
    for t in (o, lse, *grads):
        assert (t == 3.0).all()
    assert fa.fa_get_status() == 0


def test_wrong_lengths_of_a_large_batch_change_nothing(fa):
    n = [5] * 300
    (q, k, v), cu, _, _ = case(n, n, 2, 2, 64, 19)
    o, lse = torch.full_like(q, 3.0), torch.full((2, q.shape[0]), 3.0, device="cuda")
    grads = [torch.full_like(t, 3.0) for t in (q, k, v)]
    assert fa.fa_get_status() == 0
    for at, value in ((299, 2), (300, sum(n) + 1), (0, -1)):
        bad = cu.clone()
        bad[at] = value
        for cq, ck in ((bad.cuda(), cu.cuda()), (cu.cuda(), bad.cuda())):
            fa.forward_varlen(q, k, v, cq, ck, out=(o, lse))
            assert fa.fa_get_status() == FA_ERR_INVALID_ARG
            fa.backward_varlen(q, k, v, o, lse, q, cq, ck, out=grads)
            assert fa.fa_get_status() == FA_ERR_INVALID_ARG
    for t in (o, lse, *grads):
        assert (t == 3.0).all()


def test_wrong_pages_and_cache_lengths(fa):
    hq, hk, d, page = 4, 2, 64, 16
    g = su.gen(10)
    ks = [su.normal((n, hk, d), g) for n in (40, 100)]
    c = su.Cache(ks, ks, page, 10).cuda()
    q = su.normal((2, hq, d), g).cuda()
    cu = i32(0, 1, 2)
    o, lse = torch.full_like(q, 3.0), torch.full((hq, 2), 3.0, device="cuda")
    for lens in (i32(40, -1), i32(40, c.table.shape[1] * page + 1)):
        fa.forward_paged(q, c.k, c.v, cu, lens, c.table, out=(o, lse))
        assert fa.fa_get_status() == FA_ERR_INVALID_ARG
        assert (o == 3.0).all() and (lse == 3.0).all()
    keep = c.k.clone(), c.v.clone()
    for lens in (i32(0, 100), i32(-3, 100)):  # fewer keys than new tokens, for the first: the second is written
        new = su.normal((2, hk, d), g).cuda()
        fa.cache_append(new, new, c.k, c.v, cu, lens, c.table)
        assert fa.fa_get_status() == FA_ERR_INVALID_ARG
        p, r = int(c.table[1, 99 // page]), 99 % page
        for t, was in ((c.k, keep[0]), (c.v, keep[1])):
            assert torch.equal(t[p, r], new[1])
            t[p, r] = was[p, r]
            assert torch.equal(t.view(torch.int16), was.view(torch.int16))
    # a page outside the pool is neither read nor written; the other sequence is as before
    want = fa.forward_paged(q, c.k, c.v, cu, c.lens, c.table)
    for page_id in (-1, c.k.shape[0], 2 ** 31 - 1, -2 ** 31):
        table = c.table.clone()
        table[0, 2] = page_id  # of places 32 .. 39
        o, lse = fa.forward_paged(q, c.k, c.v, cu, c.lens, table)
        assert fa.fa_get_status() == FA_ERR_INVALID_ARG
        assert torch.isfinite(o).all() and torch.equal(o[1], want[0][1]) and torch.equal(lse[:, 1], want[1][:, 1])
        k, v = c.k.clone(), c.v.clone()
        fa.cache_append(new, new, k, v, cu, i32(40, 100), table)  # (place 39 is on the bad page)
        assert fa.fa_get_status() == FA_ERR_INVALID_ARG
        p, r = int(c.table[1, 99 // page]), 99 % page
        for t, was in ((k, c.k), (v, c.v)):
            assert torch.equal(t[p, r], new[1])
            t[p, r] = was[p, r]
            assert torch.equal(t.view(torch.int16), was.view(torch.int16))
    assert fa.fa_get_status() == 0


def test_shared_prefix_pages(fa):
    # two sequences whose first pages are the same
    hq, hk, d, page = 4, 1, 128, 64
    g = su.gen(11)
    ks, vs = ([su.normal((n, hk, d), g) for n in (300, 256 + 20)] for _ in range(2))
    ks[1][:256], vs[1][:256] = ks[0][:256], vs[0][:256]
    c = su.Cache(ks, vs, page, 11)
    c.table[1, :4] = c.table[0, :4]
    c.cuda()
    q, cu = su.normal((6, hq, d), g), su.starts([1, 5])
    o, lse = fa.forward_paged(q.cuda(), c.k, c.v, cu.cuda(), c.lens, c.table)
    assert fa.fa_get_status() == 0
    su.check_forward(o, lse, su.reference([(q[:1], ks[0], vs[0]), (q[1:], ks[1], vs[1])], d ** -0.5, True), cu)


def test_pages_past_32_bits(fa):
    # 70000 pages of 64 x 8 x 128 values: the last ones begin past 2^32 elements
    hq, hk, d, page, pages = 32, 8, 128, 64, 70000
    kp, vp = (torch.empty((pages, page, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = su.gen(12)
    k, v, q = su.normal((150, hk, d), g), su.normal((150, hk, d), g), su.normal((150, hq, d), g)
    table, cu, lens = i32(pages - 1, 5, pages - 7).view(1, 3), i32(0, 150), i32(150)
    fa.cache_append(k.cuda(), v.cuda(), kp, vp, cu, lens, table)
    o, lse = fa.forward_paged(q.cuda(), kp, vp, cu, lens, table)
    assert fa.fa_get_status() == 0
    assert torch.equal(kp[pages - 7, :22].cpu(), k[128:])
    su.check_forward(o, lse, su.reference([(q, k, v)], d ** -0.5, True), cu)


def test_tokens_past_32_bits(fa):
    # the sequence's q, o and gradients begin past 2^31 elements
    hq, hk, d, total, n = 32, 2, 128, 600000, 200
    g = su.gen(13)
    q, k, v, do = (su.normal((n, h, d), g) for h in (hq, hk, hk, hq))
    Q, DO = (torch.empty((total, hq, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    K, V = (torch.empty((total, hk, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for t, x in ((Q, q), (K, k), (V, v), (DO, do)):
        t[total - n:] = x.cuda()
    cu = i32(total - n, total)
    o, lse = fa.forward_varlen(Q, K, V, cu, cu, causal=True)
    dq, dk, dv = fa.backward_varlen(Q, K, V, o, lse, DO, cu, cu, causal=True)
    assert fa.fa_get_status() == 0
    last = slice(total - n, total)
    su.check_forward(o[last], lse[:, last], su.reference([(q, k, v)], d ** -0.5, True), su.starts([n]))
    want = su.reference_backward([(q, k, v)], [do], [o[last].cpu()], d ** -0.5, True)
    su.check_backward([t[last] for t in (dq, dk, dv)], want, su.starts([n]), su.starts([n]))


def test_a_wait_that_runs_out_is_reported(fa):
    # the producer never delivers a tile: every wait is bounded, the call ends with a status
    (q, k, v), cu, _, seqs = case([300], [300], 2, 1, 128, 14)
    ks = [su.normal((200, 2, 64), su.gen(15))]
    c = su.Cache(ks, ks, 16, 15).cuda()
    pq = su.normal((1, 4, 64), su.gen(16)).cuda()
    assert fa.fa_get_status() == 0
    assert fa.fa_debug_set(20_000_000, 1) == 0
    try:
        fa.forward_varlen(q, k, v, cu.cuda(), cu.cuda())
        assert fa.fa_get_status() == FA_ERR_TIMEOUT
        fa.forward_paged(pq, c.k, c.v, i32(0, 1), c.lens, c.table)
        assert fa.fa_get_status() == FA_ERR_TIMEOUT
    finally:
        fa.fa_debug_set(0, 0)
    o, lse = fa.forward_varlen(q, k, v, cu.cuda(), cu.cuda(), causal=True)
    assert fa.fa_get_status() == 0
    su.check_forward(o, lse, su.reference(seqs, 128 ** -0.5, True), cu)


def test_nothing_to_do(fa):
    z = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    k = su.normal((5, 2, 64), su.gen(17)).cuda()
    cu0, cu5 = i32(0, 0), i32(0, 5)
    o, lse = fa.forward_varlen(z, k, k, cu0, cu5)
    assert o.shape == z.shape and lse.shape == (4, 0)
    dq, dk, dv = fa.backward_varlen(z, k, k, o, lse, z, cu0, cu5)
    assert (dk == 0).all() and (dv == 0).all() and dq.shape == z.shape
    q = su.normal((5, 4, 64), su.gen(18)).cuda()
    z2 = z[:, :2].contiguous()
    o, lse = fa.forward_varlen(q, z2, z2, cu5, cu0)
    assert (o == 0).all() and (lse == -math.inf).all()
    dq, dk, dv = fa.backward_varlen(q, z2, z2, o, lse, q, cu5, cu0)
    assert (dq == 0).all() and dk.shape == z2.shape
    assert fa.fa_get_status() == 0


def test_refusals(fa):
    q, k = (su.normal((6, h, 64), su.gen(19)).cuda() for h in (4, 2))
    cu, pages, table, lens = i32(0, 6), torch.zeros((2, 16, 2, 64), dtype=torch.bfloat16, device="cuda"), i32(0).view(1, 1), i32(6)
    ok = dict(q=q, k=k, v=k, cu_q=cu, cu_k=cu)
    for bad in (dict(q=q.float()), dict(q=q[0]), dict(k=k[:5]), dict(v=k[:, :1]), dict(q=q.transpose(0, 1)),
                dict(cu_q=cu.long()), dict(cu_k=i32(0, 3, 6)), dict(cu_q=cu.cpu()), dict(cu_q=i32(0), cu_k=i32(0)),
                dict(k=k.cpu()), dict(q=q[:, :, ::2]), dict(out=(q.float(), q)), dict(out=(torch.empty_like(q), q))):
        with pytest.raises(ValueError):
            fa.forward_varlen(**{**ok, **bad})
    with pytest.raises(fa.FAError):  # 3 query heads over 2 kv heads
        fa.forward_varlen(q[:, :3], k, k, cu, cu)
    ok = dict(q=q, k_pages=pages, v_pages=pages, cu_q=cu, lens_k=lens, page_table=table)
    for bad in (dict(k_pages=pages[0]), dict(v_pages=pages[:1]), dict(k_pages=pages[:, ::2], v_pages=pages[:, ::2]),
                dict(lens_k=i32(6, 6)), dict(page_table=table.view(-1)), dict(page_table=table.float())):
        with pytest.raises(ValueError):
            fa.forward_paged(**{**ok, **bad})
    with pytest.raises(fa.FAError):  # pages of 8
        fa.forward_paged(**{**ok, "k_pages": pages.view(4, 8, 2, 64), "v_pages": pages.view(4, 8, 2, 64)})
    assert fa.fa_get_status() == 0
