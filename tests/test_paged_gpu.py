"""fa_fwd_paged and fa_cache_append on the GPU against the 64-bit oracle."""
import math

import pytest
import torch

from tests import seq_util as su

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.fa_debug_set(0, 0)
    return m


def run(fa, new, keys, hq, hk, d, page, seed, causal=True, window=None, scale=None, fused=False):
    g = su.gen(seed)
    ks, vs = [su.normal((n, hk, d), g) for n in keys], [su.normal((n, hk, d), g) for n in keys]
    c = su.Cache(ks, vs, page, seed).cuda()
    wide = su.normal((sum(new), hq + (2 * hk if fused else 0), d), g)
    q, cu = wide[:, :hq], su.starts(new)
    scale = d ** -0.5 if scale is None else scale
    o, lse = fa.forward_paged(wide.cuda()[:, :hq], c.k, c.v, cu.cuda(), c.lens, c.table, causal=causal, window=window,
                              scale=scale)
    assert fa.fa_get_status() == 0
    seqs = [(q[cu[b]:cu[b + 1]], ks[b], vs[b]) for b in range(len(new))]
    su.check_forward(o, lse, su.reference(seqs, scale, causal, window), cu)
    return o, lse


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256, 384])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(fa, page, d):
    run(fa, [1, 5, 100], [1, 300, 700], 8, 2, d, page, seed=page)


@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (6, 2), (7, 1), (32, 8), (16, 1)])
def test_single_tokens(fa, hq, hk):
    run(fa, [1] * 6, [1, 2, 127, 128, 129, 1000], hq, hk, 128, 16, seed=hq, fused=True)


@pytest.mark.parametrize("keys", [1, 16, 17, 128, 255, 256, 257, 2000, 9000])
def test_one_token(fa, keys):
    run(fa, [1], [keys], 4, 1, 128, 32, seed=keys)


def test_mixed_chunks(fa):
    run(fa, [1, 33, 1, 200, 0, 64, 1, 300], [900, 33, 4000, 200, 50, 640, 1, 1111], 8, 2, 64, 16, seed=11, fused=True)


@pytest.mark.parametrize("hq,hk,d", [(16, 8, 128), (32, 8, 64)])
def test_many_items_per_cta(fa, hq, hk, d):
    # chunks and single tokens, several work items to a CTA
    g = torch.Generator().manual_seed(hq)
    new = [1 if i % 3 else int(n) for i, n in enumerate(torch.randint(1, 300, (48,), generator=g))]
    keys = [n + int(m) for n, m in zip(new, torch.randint(0, 500, (48,), generator=g))]
    run(fa, new, keys, hq, hk, d, 16, seed=hq)


@pytest.mark.parametrize("causal,window", [(True, (100, 0)), (False, (40, 7)), (False, None), (True, (0, 0))])
def test_masks(fa, causal, window):
    run(fa, [1, 70, 9, 5], [500, 333, 9, 2], 4, 2, 128, 64, seed=12, causal=causal, window=window)


def test_more_tokens_than_keys(fa):
    # the first rows see nothing
    run(fa, [10, 300, 4], [4, 129, 0], 4, 2, 64, 16, seed=13)


def test_many_sequences(fa):
    g = torch.Generator().manual_seed(14)
    keys = torch.randint(0, 200, (1200,), generator=g).tolist()
    run(fa, [1] * 1200, keys, 2, 1, 64, 16, seed=14)


@pytest.mark.parametrize("new,keys,window", [([1], [20011], None), ([3, 0, 1], [9000, 5, 1], None), ([64], [5000], None),
                                             ([40], [7000], (2000, 0)), ([1], [20011], (300, 0)), ([17], [12], None)])
@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (3, 1, 64)])
def test_few_rows_in_many_parts(fa, new, keys, window, hq, hk, d):
    run(fa, new, keys, hq, hk, d, 32, seed=63, window=window)


def test_many_empty_sequences(fa):
    new, keys = [0] * 4000, [5] * 4000
    new[7], new[2000], new[3999] = 40, 3, 1
    keys[7], keys[3999] = 300, 900
    run(fa, new, keys, 4, 2, 128, 16, seed=62)


def test_append_then_attend(fa):
    hq, hk, d, page = 8, 2, 128, 16
    old, new = [0, 100, 31, 500], [40, 1, 17, 250]
    g = su.gen(15)
    ks, vs = [[su.normal((a + b, hk, d), g) for a, b in zip(old, new)] for _ in range(2)]
    c = su.Cache(ks, vs, page, 15)
    want_k, want_v = c.k.clone(), c.v.clone()
    for b, (a, n) in enumerate(zip(old, new)):  # the new tokens are not there yet
        for t in range(a, a + n):
            c.k[c.table[b, t // page], t % page] = math.nan
            c.v[c.table[b, t // page], t % page] = math.nan
    c.cuda()
    cu = su.starts(new)
    k, v = (torch.cat([x[a:] for x, a in zip(xs, old)]) for xs in (ks, vs))
    fused = torch.cat([su.normal((sum(new), hq, d), g), k, v], 1).cuda()
    q, fk, fv = fused[:, :hq], fused[:, hq:hq + hk], fused[:, hq + hk:]
    fa.cache_append(fk, fv, c.k, c.v, cu.cuda(), c.lens, c.table)
    o, lse = fa.forward_paged(q, c.k, c.v, cu.cuda(), c.lens, c.table)
    assert fa.fa_get_status() == 0
    for got, want in ((c.k, want_k), (c.v, want_v)):
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
    qc = q.cpu()
    seqs = [(qc[cu[b]:cu[b + 1]], ks[b], vs[b]) for b in range(4)]
    su.check_forward(o, lse, su.reference(seqs, d ** -0.5, True), cu)


@pytest.mark.parametrize("hk,d,page,new,old", [(1, 64, 16, [1], [0]), (8, 128, 64, [3, 0, 500, 1], [61, 5, 0, 63]),
                                               (3, 64, 48, [100] * 9, [7] * 9), (2, 128, 256, [1] * 300, [5] * 300)])
def test_append(fa, hk, d, page, new, old):
    g = su.gen(16)
    ks, vs = [[su.normal((a + b, hk, d), g) for a, b in zip(old, new)] for _ in range(2)]
    c = su.Cache(ks, vs, page, 16)
    want_k, want_v = c.k.clone(), c.v.clone()
    for b, (a, n) in enumerate(zip(old, new)):
        for t in range(a, a + n):
            c.k[c.table[b, t // page], t % page] = 1.0
            c.v[c.table[b, t // page], t % page] = 1.0
    c.cuda()
    k, v = (torch.cat([x[a:] for x, a in zip(xs, old)] + [su.normal((3, hk, d), g)]).cuda() for xs in (ks, vs))
    fa.cache_append(k, v, c.k, c.v, su.starts(new).cuda(), c.lens, c.table)  # (3 rows behind the last sequence)
    assert fa.fa_get_status() == 0
    for got, want in ((c.k, want_k), (c.v, want_v)):
        assert torch.equal(got.cpu().view(torch.int16), want.view(torch.int16))
