"""fa_fwd_paged_fp8 on the GPU against the 64-bit attention of the values that the cache stands for."""
import math

import pytest
import torch

from tests import cache8_util as cu8
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


def run(fa, new, keys, hq, hk, d, page, seed, causal=True, window=None, scale=None, fused=False, sigma=None, edit=None,
        q_edit=None):
    c = cu8.filled(keys, hk, d, page, seed, sigma)
    if edit:
        edit(c)
    g = su.gen(seed)
    wide = su.normal((sum(new), hq + (2 * hk if fused else 0), d), g)
    if q_edit:
        q_edit(wide)
    q, cu = wide[:, :hq], su.starts(new)
    scale = d ** -0.5 if scale is None else scale
    pages, table = c.cuda()
    o, lse = fa.forward_paged_fp8(wide.cuda()[:, :hq], *pages, cu.cuda(), c.lens_k().cuda(), table, causal=causal,
                                  window=window, scale=scale)
    assert fa.fa_get_status() == 0
    seqs = [(q[cu[b]:cu[b + 1]], *c.values(b)) for b in range(len(new))]
    cu8.check_forward(o, lse, su.reference(seqs, scale, causal, window), seqs, cu)
    return o, lse


@pytest.mark.parametrize("page", [16, 32, 48, 64, 80, 128, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_page_sizes(fa, page, d):
    run(fa, [1, 5, 100], [1, 300, 700], 8, 2, d, page, seed=page)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 4), (6, 2), (7, 1), (32, 8), (16, 1), (10, 1), (40, 1), (128, 1)])
def test_single_tokens(fa, hq, hk, d):
    run(fa, [1] * 6, [1, 2, 127, 128, 129, 1000], hq, hk, d, 16, seed=hq, fused=True)


@pytest.mark.parametrize("keys", [1, 15, 16, 17, 128, 255, 256, 257, 2000, 9000])
def test_one_token(fa, keys):
    run(fa, [1], [keys], 4, 1, 128, 32, seed=keys)


@pytest.mark.parametrize("new", [1, 2, 3, 8, 17, 64, 130, 300])
@pytest.mark.parametrize("d", [64, 128])
def test_chunks(fa, new, d):
    run(fa, [new], [new + 200], 4, 1, d, 16, seed=new)


@pytest.mark.parametrize("window", [None, (5, 0), (300, 2)])
@pytest.mark.parametrize("new,keys", [([4, 1, 3], [300, 2000, 77]), ([10, 1, 1], [12, 900, 3000]), ([16], [4000]),
                                      ([0, 9, 0, 3, 1], [50, 700, 0, 1500, 1]),
                                      ([4] * 30 + [1], [5 + 40 * i for i in range(30)] + [3])])
@pytest.mark.parametrize("d", [64, 128])
def test_few_tokens_of_few_sequences(fa, new, keys, d, window):
    run(fa, new, keys, 8, 2, d, 32, window=window, seed=len(new))


@pytest.mark.parametrize("new", [[200, 260], [128, 64], [513]])
def test_prompts_of_their_own(fa, new):
    # every key is new
    run(fa, new, new, 8, 2, 128, 64, seed=sum(new), fused=True)


def test_mixed_chunks(fa):
    run(fa, [1, 33, 1, 200, 0, 64, 1, 300], [900, 33, 4000, 200, 50, 640, 1, 1111], 8, 2, 64, 16, seed=11, fused=True)


def test_mixed_chunks_128(fa):
    run(fa, [1, 33, 1, 200, 0, 64, 1, 300], [900, 33, 2000, 200, 50, 640, 1, 1111], 8, 2, 128, 48, seed=12, fused=True)


@pytest.mark.parametrize("hq,hk,d", [(16, 8, 128), (32, 8, 64), (16, 2, 64), (8, 1, 128)])
def test_many_items_per_cta(fa, hq, hk, d):
    # chunks of one row tile and of two in any order, several work items to a CTA
    g = torch.Generator().manual_seed(hq)
    new = [1 + i % 5 if i % 3 else int(n) for i, n in enumerate(torch.randint(1, 300, (48,), generator=g))]
    keys = [n + int(m) for n, m in zip(new, torch.randint(0, 900, (48,), generator=g))]
    run(fa, new, keys, hq, hk, d, 16, seed=hq)


@pytest.mark.parametrize("window", [None, (70, 0)])
@pytest.mark.parametrize("hq,hk,d", [(8, 1, 64), (8, 2, 128)])
def test_more_units_than_a_cta_plans_for_itself(fa, hq, hk, d, window):
    g = torch.Generator().manual_seed(d)
    new = torch.randint(0, 21, (400,), generator=g).tolist()
    keys = [n + int(m) for n, m in zip(new, torch.randint(0, 300, (400,), generator=g))]
    run(fa, new, keys, hq, hk, d, 32, seed=d, window=window)


def test_long_prompt(fa):
    run(fa, [3100, 700], [3100, 2000], 2, 1, 64, 64, seed=3)


@pytest.mark.parametrize("causal,window", [(True, (100, 0)), (False, (40, 7)), (False, None), (True, (0, 0))])
@pytest.mark.parametrize("d", [64, 128])
def test_masks(fa, causal, window, d):
    run(fa, [1, 70, 9, 5], [500, 333, 9, 2], 4, 2, d, 64, seed=13, causal=causal, window=window)


def test_more_tokens_than_keys(fa):
    # the first rows see nothing
    run(fa, [10, 300, 4, 1], [4, 129, 0, 0], 4, 2, 64, 16, seed=14)


@pytest.mark.parametrize("where", ["ends", "gaps"])
def test_slots_without_a_sequence(fa, where):
    # a captured call's unused places, more than a warp looks at in one go
    n, keys = [0] * 700, [0] * 700
    for b in [0, 1, 2, 40, 41] if where == "ends" else [33, 66, 69, 300, 699]:
        n[b], keys[b] = 1 + b % 2, 500 + 3 * b
    keys[450] = 90  # keys, but no new tokens
    run(fa, n, keys, 8, 2, 64, 16, seed=29)


def test_many_sequences(fa):
    g = torch.Generator().manual_seed(15)
    keys = torch.randint(0, 200, (1200,), generator=g).tolist()
    run(fa, [1] * 1200, keys, 2, 1, 64, 16, seed=15)


def test_values_of_very_different_blocks(fa):
    # V from 1e-6 to 1e5 from block to block, both ways round: P weighs by the scales in the exponent
    run(fa, [1, 40], [1500, 700], 4, 2, 128, 16, seed=16, sigma=(1e-6, 1.0, 1e5, 1e-3))


@pytest.mark.parametrize("new", [[1, 3], [1, 20]])
@pytest.mark.parametrize("size", [1e-30, 1e-4, 300.0, 1e20])
def test_queries_of_any_size(fa, size, new):
    def edit(w):
        w *= size
        w[0, 0] = 0.0
    run(fa, new, [300, 200], 4, 2, 64, 16, seed=17, scale=0.1 / size, q_edit=edit)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.5])
def test_scales(fa, scale):
    if scale == 1.5:
        # sharper: scores up to 1.5 sum |q k| < 2^8, so their error is 2^4 times that of unit scores
        def q_edit(w):
            w *= 0.0625
    else:
        q_edit = None
    run(fa, [1, 20, 150], [300, 200, 150], 4, 2, 64, 16, seed=18, scale=scale, q_edit=q_edit)


def test_any_scales_of_blocks(fa):
    # not powers of two: a cache that was filled by something else
    def edit(c):
        g = su.gen(19)
        for s in c.scales:
            s *= torch.rand(s.shape, generator=g) + 0.5
    run(fa, [1, 90], [700, 200], 4, 2, 128, 16, seed=19, edit=edit)


@pytest.mark.parametrize("new", [[1, 3], [70, 20]])
@pytest.mark.parametrize("low,high", [(2.0 ** -80, 2.0 ** -80),
                                      (2.0 ** 100, 2.0 ** 100), (2.0 ** -70, 2.0 ** 25), (2.0 ** 10, 2.0 ** 100)])
def test_scales_of_far_apart_sizes(fa, new, low, high):
    # V's blocks in turn: the row sum is over all of them, whatever V's size
    def edit(c):
        c.scales[1][:, 0::2] *= low
        c.scales[1][:, 1::2] *= high
    run(fa, new, [700, 200], 4, 2, 128, 64, seed=27, edit=edit)


@pytest.mark.parametrize("new", [1, 90])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_are_all_minus_infinity(fa, new, d):
    c = cu8.filled([300], 1, d, 16, seed=28)
    c.codes[0].view(torch.uint8)[..., 3] = 0xB8  # -1
    pages, table = c.cuda()
    q = su.normal((new, 2, d), su.gen(28))
    q[0, 1, 3] = math.inf
    o, _ = fa.forward_paged_fp8(q.cuda(), *pages, su.starts([new]).cuda(), c.lens_k().cuda(), table)
    bad = o.float().isnan().all(2).cpu()
    assert bad[0, 1] and o.float().isnan().any(2).sum() == 1


def test_nan_stays_in_its_rows(fa):
    c = cu8.filled([300, 64], 1, 64, 16, seed=20)
    pages, table = c.cuda()
    page = int(c.table[0, 299 // 16])
    pages[0].view(torch.uint8)[page, 299 % 16] = 0x7F  # K of the last key
    q = su.normal((42, 2, 64), su.gen(20)).cuda()
    cu = su.starts([40, 2])
    o, _ = fa.forward_paged_fp8(q, *pages, cu.cuda(), c.lens_k().cuda(), table)
    assert fa.fa_get_status() == 0
    bad = o.float().isnan().flatten(1).any(1).cpu()
    assert bad[39] and not bad[:39].any() and not bad[40:].any()


@pytest.mark.parametrize("new", [3, 60])
def test_queries_that_are_not_finite(fa, new):
    c = cu8.filled([300], 1, 64, 16, seed=25)
    pages, table = c.cuda()
    q = su.normal((new, 2, 64), su.gen(25))
    q[0, 0, 3] = math.inf
    q[1, 1, 0] = math.nan
    o, _ = fa.forward_paged_fp8(q.cuda(), *pages, su.starts([new]).cuda(), c.lens_k().cuda(), table)
    bad = o.float().isnan().any(2).cpu()
    assert bad[0, 0] and bad[1, 1] and bad.sum() == 2


@pytest.mark.parametrize("new", [2, 90])
def test_queries_with_an_outlier(fa, new):
    # One channel of 30: scores up to 30 * 4 * scale 0.02 and the rounding of q in
    # two e4m3 parts: 2^-17 of 30 in each channel, times sum |k| < 120 and 0.02: 2^-11
    # at worst, all of one sign; of random signs (120 -> 11) it is 2^-14.6, within what
    # the bounds have for the scores.
    def q_edit(w):
        w[:, :, 5] = 30.0
    run(fa, [new], [400], 4, 2, 128, 16, seed=26, scale=0.02, q_edit=q_edit)


def test_rows_outside_the_sequences(fa):
    c = cu8.filled([300, 64], 2, 64, 16, seed=21)
    pages, table = c.cuda()
    q = su.normal((50, 4, 64), su.gen(21)).cuda()
    o = torch.full((50, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((4, 50), 7.0, device="cuda")
    cu = torch.tensor([5, 30, 41], dtype=torch.int32)
    fa.forward_paged_fp8(q, *pages, cu.cuda(), c.lens_k().cuda(), table, out=(o, lse))
    assert fa.fa_get_status() == 0
    for a, b in ((0, 5), (41, 50)):
        assert (o[a:b] == 7.0).all() and (lse[:, a:b] == 7.0).all()
    seqs = [(q[5:30].cpu(), *c.values(0)), (q[30:41].cpu(), *c.values(1))]
    cu8.check_forward(o, lse, su.reference(seqs, 0.125, True), seqs, cu)


def test_bad_lengths_and_pages(fa):
    c = cu8.filled([64, 64], 1, 64, 16, seed=22)
    pages, table = c.cuda()
    q = su.normal((10, 2, 64), su.gen(22)).cuda()

    def call(cu, lens, table=table):
        o = torch.full((10, 2, 64), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((2, 10), 7.0, device="cuda")
        fa.forward_paged_fp8(q, *pages, torch.tensor(cu, dtype=torch.int32).cuda(),
                             torch.tensor(lens, dtype=torch.int32).cuda(), table, out=(o, lse))
        return fa.fa_get_status(), bool((o == 7.0).all())

    assert call([0, 5, 10], [64, 64]) == (0, False)
    assert call([0, 5, 11], [64, 64]) == (1, True)
    assert call([0, 5, 4], [64, 64]) == (1, True)
    assert call([0, 5, 10], [64, -1]) == (1, True)
    assert call([0, 5, 10], [64, 16 * table.shape[1] + 1]) == (1, True)
    t = table.clone()
    t[0, 1] = 10 ** 6
    st, left = call([0, 5, 10], [64, 64], t)
    assert st == 1 and not left
    assert fa.fa_get_status() == 0


def test_bad_page_reads_as_zeros(fa):
    c = cu8.filled([48], 1, 64, 16, seed=23)
    pages, table = c.cuda()
    q = su.normal((1, 2, 64), su.gen(23))
    t = table.clone()
    t[0, 1] = -1
    o, lse = fa.forward_paged_fp8(q.cuda(), *pages, su.starts([1]).cuda(), c.lens_k().cuda(), t)
    assert fa.fa_get_status() == 1
    k, v = c.values(0)
    k[16:32] = 0
    v[16:32] = 0
    seqs = [(q, k, v)]
    cu8.check_forward(o, lse, su.reference(seqs, 0.125, True), seqs, su.starts([1]))


@pytest.mark.parametrize("new,keys", [([1, 30, 200], [5000, 77, 900]), ([1, 1, 2], [5000, 77, 900]), ([30] * 300, [200] * 300)])
def test_repeatable(fa, new, keys):
    c = cu8.filled(keys, 2, 128, 16, seed=24)
    pages, table = c.cuda()
    q = su.normal((sum(new), 8, 128), su.gen(24)).cuda()
    args = (q, *pages, su.starts(new).cuda(), c.lens_k().cuda(), table)
    o, lse = fa.forward_paged_fp8(*args)
    for _ in range(5):
        o2, lse2 = fa.forward_paged_fp8(*args)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
