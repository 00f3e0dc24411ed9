"""Rotary positions, the 8-bit cache and its attention as programs use them: a
serving loop, a training step, captured graphs, several streams, shared pages,
offsets past 32 bits, a wait that runs out, refusals."""
import math
import threading

import numpy as np
import pytest
import torch

from tests import cache8_util as cu8
from tests import seq_util as su
from tests.test_rotary_gpu import check, turned

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


def test_serving_loop(fa):
    # Prompts go into the cache in chunks, then token by token, from one fused
    # projection: q and k turned in place, k and v appended, q over the cache. Each
    # step's rows are the attention over what the cache stands for.
    hq, hk, d, page, steps = 8, 2, 128, 32, ([100, 70], [125, 0], [1, 1], [1, 1], [17, 1], [1, 1], [0, 1])
    g = su.gen(1)
    f, m = fa.rotary_frequencies(d, scaling="yarn", factor=4.0, original_length=64)
    f64, dev_f = f.double().numpy(), f.cuda()
    c = cu8.Cache8([sum(s[b] for s in steps) for b in range(2)], hk, d, page, seed=1)
    pages, table = c.cuda()
    for new in steps:
        first = np.concatenate([np.arange(n) + c.lens[b] for b, n in enumerate(new)])
        wide = su.normal((sum(new), hq + 2 * hk, d), g)
        dev, cu = wide.cuda(), su.starts(new)
        q, k, v = dev[:, :hq], dev[:, hq:hq + hk], dev[:, hq + hk:]
        lens = i32(*(c.lens[b] + n for b, n in enumerate(new)))
        fa.rotary(q, k, dev_f, cu.cuda(), lens, mscale=m, out=(q, k))
        fa.cache_append_fp8(k, v, *pages, cu.cuda(), lens, table)
        o, lse = fa.forward_paged_fp8(q, *pages, cu.cuda(), lens, table)
        assert fa.fa_get_status() == 0
        for x, y in ((wide[:, :hq], q), (wide[:, hq:hq + hk], k)):
            check(y, *turned(su.n64(x), first, f64, False, m))
        at = [slice(int(cu[b]), int(cu[b + 1])) for b in range(2)]
        kc, vc, qc = k.cpu(), v.cpu(), q.cpu()
        c.append([kc[s] for s in at], [vc[s] for s in at])
        seqs = [(qc[s], *c.values(b)) for b, s in enumerate(at)]
        cu8.check_forward(o, lse, su.reference(seqs, d ** -0.5, True), seqs, cu)


def test_training_step(fa):
    # turned q and k through the packed attention and back: each stage against its formula in 64 bits
    n, hq, hk, d = [130, 1, 77], 4, 2, 64
    g = su.gen(2)
    q, k, v, do = (su.normal((sum(n), h, d), g) for h in (hq, hk, hk, hq))
    f, m = fa.rotary_frequencies(32)
    cu = su.starts(n)
    dev, dev_f = cu.cuda(), f.cuda()
    tq, tk = fa.rotary(q.cuda(), k.cuda(), dev_f, dev, interleaved=True)
    o, lse = fa.forward_varlen(tq, tk, v.cuda(), dev, dev, causal=True)
    dtq, dtk, dv = fa.backward_varlen(tq, tk, v.cuda(), o, lse, do.cuda(), dev, dev, causal=True)
    dq, dk = fa.rotary_backward(dtq, dtk, dev_f, dev, interleaved=True)
    assert fa.fa_get_status() == 0
    at = [slice(int(cu[b]), int(cu[b + 1])) for b in range(len(n))]
    place = np.concatenate([np.arange(x) for x in n])
    for x, y, back in ((q, tq, False), (k, tk, False), (dtq, dq, True), (dtk, dk, True)):
        check(y, *turned(su.n64(x), place, f.double().numpy(), True, m, back=back))
    want = su.reference_backward([(tq[s].cpu(), tk[s].cpu(), v[s]) for s in at], [do[s] for s in at], [o[s].cpu() for s in at],
                                 d ** -0.5, True)
    su.check_backward((dtq, dtk, dv), want, cu, cu)


@pytest.mark.parametrize("many", [False, True])
def test_graph_replays_with_other_lengths(fa, many):
    # captured once (for few rows to a kv head, or for many); the lengths, offsets and pages of each replay are its own
    hq, hk, d, page, B, total = 8, 2, 64, 16, 6, (600 if many else 12)
    g = su.gen(3)
    q, k, v = (su.normal((total, h, d), g).cuda() for h in (hq, hk, hk))
    f = fa.rotary_frequencies(d)[0].cuda()
    c = cu8.filled([700] * B, hk, d, page, 3)
    pages, table = c.cuda()
    start = [x.clone() for x in pages]
    first = [total - 5, 1, 1, 1, 1, 1]
    cu, lens = su.starts(first).cuda(), i32(*(min(700, n + 30) for n in first))
    outs = [torch.zeros(s, dtype=torch.bfloat16, device="cuda") for s in (q.shape, k.shape, q.shape)]
    lse = torch.zeros((hq, total), device="cuda")

    def step():
        fa.rotary(q, k, f, cu, lens, out=(outs[0], outs[1]))
        fa.cache_append_fp8(outs[1], v, *pages, cu, lens, table)
        fa.forward_paged_fp8(outs[0], *pages, cu, lens, table, out=(outs[2], lse))

    step()
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        with torch.cuda.graph(graph, stream=s):
            step()
    torch.cuda.current_stream().wait_stream(s)
    for new, keys in ((first, [min(700, n + 30) for n in first]), ([1, 1, 1, 1, 1, 1], [5, 640, 17, 300, 1, 33]),
                      ([0, total, 0, 0, 0, 0], [10, 600 if many else 690, 0, 9, 0, 1])):
        cu.copy_(su.starts(new))
        lens.copy_(i32(*keys))
        got = []
        for run in (graph.replay, step):
            for x, y in zip(pages, start):
                x.copy_(y)
            for t in outs + [lse]:
                t.fill_(5.0)
            run()
            assert fa.fa_get_status() == 0
            got.append([t.clone().view(torch.uint8) for t in outs + [lse] + pages])
        for i, (a, b) in enumerate(zip(*got)):
            assert torch.equal(a, b), i


@pytest.mark.parametrize("new", [[1, 2], [300, 50]])
def test_two_graphs_and_two_threads_at_once(fa, new):
    # calls on two streams at once, captured and eager: each has a workspace of its own
    cases = []
    for seed in (4, 5):
        c = cu8.filled([3000 + 500 * seed, 2000], 2, 128, 64, seed)
        pages, table = c.cuda()
        q = su.normal((sum(new), 8, 128), su.gen(seed)).cuda()
        cases.append((q, *pages, su.starts(new).cuda(), c.lens_k().cuda(), table))
    want = [fa.forward_paged_fp8(*c) for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    graphs, outs = [], []
    for c, s in zip(cases, streams):
        out = (torch.zeros_like(c[0]), torch.zeros((8, c[0].shape[0]), device="cuda"))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.stream(s):
            with torch.cuda.graph(g, stream=s):
                fa.forward_paged_fp8(*c, out=out)
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

    def loop(c, s, w):
        for _ in range(30):
            o, lse = fa.forward_paged_fp8(*c, stream=s)
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
    x = su.normal((70, 4, 64), su.gen(6)).cuda()
    f, cu, lens = fa.rotary_frequencies(64)[0].cuda(), i32(0, 70), i32(80)
    c = cu8.filled([80], 4, 64, 16, 6)
    pages, table = c.cuda()
    want = fa.rotary(x, None, f, cu, lens)[0], fa.forward_paged_fp8(x, *pages, cu, lens, table)[0]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for handle in (s, s.cuda_stream):
        got = fa.rotary(x, None, f, cu, lens, stream=handle)[0], fa.forward_paged_fp8(x, *pages, cu, lens, table, stream=handle)[0]
        s.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_items_without_keys_between_others(fa):
    # more rows than keys, many sequences: items with key tiles and without follow one another
    for new, hq in ((1, 8), (40, 8)):
        g = torch.Generator().manual_seed(new)
        keys = [0 if i % 5 else int(n) for i, n in enumerate(torch.randint(0, 900, (300 if new == 1 else 60,), generator=g))]
        c = cu8.filled(keys, 1, 128, 16, 7)
        pages, table = c.cuda()
        n = [new] * len(keys)
        q, cu = su.normal((sum(n), hq, 128), su.gen(7)), su.starts(n)
        args = (q.cuda(), *pages, cu.cuda(), c.lens_k().cuda(), table)
        o, lse = fa.forward_paged_fp8(*args)
        assert fa.fa_get_status() == 0
        seqs = [(q[cu[b]:cu[b + 1]], *c.values(b)) for b in range(len(n))]
        cu8.check_forward(o, lse, su.reference(seqs, 128 ** -0.5, True), seqs, cu)
        for _ in range(10):
            again = fa.forward_paged_fp8(*args)
            assert torch.equal(again[0], o) and torch.equal(again[1], lse)


def test_one_long_sequence_among_empty_ones(fa):
    # a batch of slots of which few are taken: the mean says single tokens
    n = [0] * 200
    n[77], n[150] = 90, 3
    keys = [x + 100 if x else i % 3 for i, x in enumerate(n)]
    c = cu8.filled(keys, 2, 64, 16, 8)
    pages, table = c.cuda()
    q, cu = su.normal((sum(n), 8, 64), su.gen(8)), su.starts(n)
    o, lse = fa.forward_paged_fp8(q.cuda(), *pages, cu.cuda(), c.lens_k().cuda(), table)
    assert fa.fa_get_status() == 0
    seqs = [(q[cu[b]:cu[b + 1]], *c.values(b)) for b in range(len(n))]
    cu8.check_forward(o, lse, su.reference(seqs, 0.125, True), seqs, cu)


@pytest.mark.parametrize("new", [[1, 1], [1, 60]])
def test_pages_hidden_by_the_window_are_not_looked_up(fa, new):
    # a server may have given them to other sequences: their entries are bad, or their codes NaN
    keys, window = [900, 1000], (100, 0)
    c = cu8.filled(keys, 2, 64, 16, 9)
    q, cu = su.normal((sum(new), 4, 64), su.gen(9)), su.starts(new)
    seqs = [(q[cu[b]:cu[b + 1]], *c.values(b)) for b in range(2)]
    for b in range(2):
        c.table[b, :(keys[b] - new[b] - 100) // 16] = -5
    pages, table = c.cuda()
    o, lse = fa.forward_paged_fp8(q.cuda(), *pages, cu.cuda(), c.lens_k().cuda(), table, window=window)
    assert fa.fa_get_status() == 0
    cu8.check_forward(o, lse, su.reference(seqs, 0.125, True, window), seqs, cu)


def test_shared_prefix_pages(fa):
    hq, hk, d, page = 4, 1, 128, 64
    c = cu8.filled([300, 276], hk, d, page, 11)
    c.table[1, :4] = c.table[0, :4]
    pages, table = c.cuda()
    q, cu = su.normal((6, hq, d), su.gen(11)), su.starts([1, 5])
    o, lse = fa.forward_paged_fp8(q.cuda(), *pages, cu.cuda(), c.lens_k().cuda(), table)
    assert fa.fa_get_status() == 0
    seqs = [(q[:1], *c.values(0)), (q[1:], *c.values(1))]
    cu8.check_forward(o, lse, su.reference(seqs, d ** -0.5, True), seqs, cu)


@pytest.mark.parametrize("new", [1, 150])
def test_pages_past_32_bits(fa, new):
    # 140000 pages of 64 x 8 x 128 codes: the last ones begin past 2^33 bytes
    hq, hk, d, page, pages = 32, 8, 128, 64, 140000
    kp, vp = (torch.empty((pages, page, hk, d), dtype=torch.uint8, device="cuda").view(cu8.E4M3) for _ in range(2))
    ks, vs = (torch.empty((pages, page // 16, hk), device="cuda") for _ in range(2))
    g = su.gen(12)
    k, v, q = su.normal((150, hk, d), g), su.normal((150, hk, d), g), su.normal((150, hq, d), g)[150 - new:]
    table, lens = i32(pages - 1, 5, pages - 7).view(1, 3), i32(150)
    fa.cache_append_fp8(k.cuda(), v.cuda(), kp, vp, ks, vs, i32(0, 150), lens, table)
    o, lse = fa.forward_paged_fp8(q.cuda(), kp, vp, ks, vs, i32(0, new), lens, table)
    assert fa.fa_get_status() == 0
    c = cu8.Cache8([150], hk, d, page, 12)
    c.append([k], [v])
    seqs = [(q, *c.values(0))]
    assert torch.equal(kp[pages - 7, :22].cpu().view(torch.uint8), c.codes[0][int(c.table[0, 2]), :22].view(torch.uint8))
    cu8.check_forward(o, lse, su.reference(seqs, d ** -0.5, True), seqs, su.starts([new]))


@pytest.mark.parametrize("hk,d", [(3, 64), (200, 64), (1, 128)])
def test_head_counts(fa, hk, d):
    run_new, keys = [1, 40], [200, 40]
    c = cu8.Cache8(keys, hk, d, 16, 13)
    g = su.gen(13)
    ks, vs = ([su.normal((n, hk, d), g) for n in keys] for _ in range(2))
    c.append(ks, vs)
    pages, table = c.cuda()
    q, cu = su.normal((41, hk, d), g), su.starts(run_new)
    o, lse = fa.forward_paged_fp8(q.cuda(), *pages, cu.cuda(), c.lens_k().cuda(), table)
    assert fa.fa_get_status() == 0
    seqs = [(q[:1], *c.values(0)), (q[1:], *c.values(1))]
    cu8.check_forward(o, lse, su.reference(seqs, d ** -0.5, True), seqs, cu)


@pytest.mark.parametrize("new", [1, 100])
def test_a_wait_that_runs_out_is_reported(fa, new):
    c = cu8.filled([300], 2, 64, 16, 14)
    pages, table = c.cuda()
    q = su.normal((new, 4, 64), su.gen(14)).cuda()
    args = (q, *pages, i32(0, new), c.lens_k().cuda(), table)
    want = fa.forward_paged_fp8(*args)
    assert fa.fa_get_status() == 0
    assert fa.fa_debug_set(20_000_000, 1) == 0
    try:
        fa.forward_paged_fp8(*args)
        assert fa.fa_get_status() == FA_ERR_TIMEOUT
    finally:
        fa.fa_debug_set(0, 0)
    got = fa.forward_paged_fp8(*args)
    assert fa.fa_get_status() == 0
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_nothing_to_do(fa):
    z = torch.empty((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    c = cu8.filled([20], 4, 64, 16, 15)
    pages, table = c.cuda()
    o, lse = fa.forward_paged_fp8(z, *pages, i32(0, 0), i32(20), table)
    assert o.shape == z.shape and lse.shape == (4, 0)
    fa.cache_append_fp8(z, z, *pages, i32(0, 0), i32(20), table)
    y, none = fa.rotary(z, None, fa.rotary_frequencies(64)[0].cuda(), i32(0, 0))
    assert y.shape == z.shape and none is None and fa.fa_get_status() == 0


def test_refusals(fa):
    q, k = (su.normal((6, h, 64), su.gen(16)).cuda() for h in (4, 2))
    c = cu8.filled([6], 2, 64, 16, 16)
    (kp, vp, ks, vs), table = c.cuda()
    cu, lens = i32(0, 6), i32(6)
    ok = dict(q=q, k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, cu_q=cu, lens_k=lens, page_table=table)
    for bad in (dict(q=q.float()), dict(k_pages=kp.view(torch.uint8)), dict(v_pages=vp[:1]), dict(k_scales=ks.half()),
                dict(v_scales=vs[:1]), dict(k_scales=ks.transpose(0, 2).contiguous().transpose(0, 2)), dict(k_scales=ks.cpu()),
                dict(lens_k=lens.long()), dict(lens_k=i32(6, 6)), dict(page_table=table.view(-1)), dict(cu_q=cu.cpu()),
                dict(k_pages=kp[:, ::2], v_pages=vp[:, ::2])):
        with pytest.raises(ValueError):
            fa.forward_paged_fp8(**{**ok, **bad})
    ok = dict(k=k, v=k, k_pages=kp, v_pages=vp, k_scales=ks, v_scales=vs, cu_q=cu, lens_k=lens, page_table=table)
    for bad in (dict(k=k.float()), dict(v=k[:5]), dict(k_pages=kp.view(torch.uint8)), dict(v_scales=vs.double()),
                dict(v_scales=vs.view(-1))):
        with pytest.raises(ValueError):
            fa.cache_append_fp8(**{**ok, **bad})
    f = fa.rotary_frequencies(64)[0].cuda()
    ok = dict(q=q, k=k, inv_freq=f, cu=cu)
    for bad in (dict(q=q.float()), dict(k=k[:5]), dict(inv_freq=f.double()), dict(inv_freq=f.cpu()), dict(cu=cu.long()),
                dict(cu=i32(0)), dict(lens=i32(6, 6)), dict(lens=i32(6).long()), dict(out=(q, None)), dict(out=(q[:5], k)),
                dict(q=q.transpose(0, 1)), dict(inv_freq=f[None]), dict(q=None, k=None)):
        with pytest.raises(ValueError):
            fa.rotary(**{**ok, **bad})
    for bad in (dict(inv_freq=f[:5]), dict(inv_freq=torch.cat((f, f))), dict(mscale=math.nan), dict(inv_freq=f[:0])):
        with pytest.raises(fa.FAError):
            fa.rotary(**{**ok, **bad})
    assert fa.fa_get_status() == 0
