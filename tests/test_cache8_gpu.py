"""fa_cache_append_fp8 on the GPU: codes and scales are those of the definition, bit for bit."""
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


def same(c, pages):
    for x, y in zip(c.codes, pages[:2]):
        a, b = x.view(torch.uint8), y.cpu().view(torch.uint8)
        # a NaN code may have either sign
        assert torch.equal(torch.where((a & 0x7F) == 0x7F, 0x7F, a), torch.where((b & 0x7F) == 0x7F, 0x7F, b))
    for x, y in zip(c.scales, pages[2:]):
        assert torch.equal(x.nan_to_num(-1.0), y.cpu().nan_to_num(-1.0))


def steps(fa, rounds, hk, d, page, seed, fused=False, sigma=(1.0,), edit=None):
    """rounds: per call the new tokens of each sequence."""
    g = su.gen(seed)
    B = len(rounds[0])
    c = cu8.Cache8([sum(r[b] for r in rounds) for b in range(B)], hk, d, page, seed)
    pages, table = c.cuda()
    for i, new in enumerate(rounds):
        total = sum(new)
        wide = (torch.randn((total, 3 * hk if fused else 2 * hk, d), generator=g) * sigma[i % len(sigma)]).to(torch.bfloat16)
        if edit:
            edit(i, wide)
        dev = wide.cuda()
        k, v = wide[:, :hk], wide[:, hk:2 * hk]
        cu = su.starts(new)
        c.append([k[cu[b]:cu[b + 1]] for b in range(B)], [v[cu[b]:cu[b + 1]] for b in range(B)])
        fa.cache_append_fp8(dev[:, :hk], dev[:, hk:2 * hk], *pages, cu.cuda(), c.lens_k().cuda(), table)
        assert fa.fa_get_status() == 0
        same(c, pages)
    return c, pages


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("d", [64, 128])
def test_prompts(fa, page, d):
    steps(fa, [[1, 15, 16, 17, 0, 200, 333]], 2, d, page, seed=page + d, fused=True)


@pytest.mark.parametrize("hk", [1, 3, 8])
def test_single_tokens_after_prompts(fa, hk):
    # each step's rows are larger or smaller than those held, so that scales rise and stay
    steps(fa, [[5, 16, 31, 0]] + [[1, 1, 1, 1]] * 20, hk, 128, 16, seed=hk, sigma=(1.0, 0.01, 3.0, 1.0, 300.0, 2.0))


@pytest.mark.parametrize("d", [64, 128])
def test_few_tokens_at_a_time(fa, d):
    # every size about an access's rows, at many places of a block
    steps(fa, [[1, 2, 3, 4, 5, 6, 0]] * 9, 3, d, 16, seed=10 + d, sigma=(1.0, 0.1, 7.0, 300.0))


def test_chunks_that_end_inside_blocks(fa):
    steps(fa, [[3, 40, 0], [20, 1, 7], [0, 0, 10], [9, 70, 1]], 2, 64, 32, seed=4, sigma=(1.0, 8.0, 1e-3, 30.0))


def test_extreme_values(fa):
    def edit(i, w):
        w[0] = 0.0                   # zeros only
        w[1] = 1e-38                 # far below the smallest scale's codes
        w[2] = 3.3e38                # near bf16's largest
        w[3, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 5.0])
        w[4] = math.nan
        w[5] = 448.0
        w[6] = 450.0                 # the next bf16 value above 448
        w[7] = 1e-20
    steps(fa, [[8], [8], [1], [1]] + [[1]] * 0, 2, 64, 16, seed=5, edit=lambda i, w: edit(i, w) if w.shape[0] == 8 else None)


@pytest.mark.parametrize("which", range(8))
def test_each_extreme_in_a_block_of_its_own(fa, which):
    vals = [0.0, 1e-38, 3.3e38, math.inf, math.nan, 448.0, 450.0, 1e-20]

    def edit(i, w):
        w[0] = vals[which]
    steps(fa, [[1], [1], [14], [1]], 1, 128, 16, seed=6, edit=lambda i, w: edit(i, w) if i == 0 else None)


def test_many_sequences(fa):
    g = su.gen(7)
    n = torch.randint(0, 3, (1500,), generator=g).tolist()
    steps(fa, [n, n[::-1]], 1, 64, 16, seed=7, sigma=(1.0, 20.0))


def test_rows_outside_the_sequences_are_left_out(fa):
    c = cu8.Cache8([20, 20], 2, 64, 16, seed=8)
    pages, table = c.cuda()
    k, v = su.normal((50, 2, 64), su.gen(8)), su.normal((50, 2, 64), su.gen(9))
    cu = torch.tensor([7, 20, 31], dtype=torch.int32)
    c.append([k[7:20], k[20:31]], [v[7:20], v[20:31]])
    fa.cache_append_fp8(k.cuda(), v.cuda(), *pages, cu.cuda(), c.lens_k().cuda(), table)
    assert fa.fa_get_status() == 0
    same(c, pages)


def test_bad_lengths_and_pages(fa):
    k = su.normal((10, 1, 64), su.gen(10)).cuda()

    def call(cu, lens, table, codes=None):
        c = cu8.Cache8([64, 64], 1, 64, 16, seed=10)
        pages, _ = c.cuda()
        before = [x.clone() for x in pages]
        fa.cache_append_fp8(k, k, *pages, torch.tensor(cu, dtype=torch.int32).cuda(),
                            torch.tensor(lens, dtype=torch.int32).cuda(), torch.tensor(table, dtype=torch.int32).cuda())
        st = fa.fa_get_status()
        changed = [not torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(before, pages)]
        return st, any(changed)

    assert call([0, 5, 10], [5, 5], [[0], [1]]) == (0, True)
    assert call([0, 0, 10], [0, 5], [[0], [1]]) == (1, False)    # more new tokens than the sequence has
    assert call([0, 0, 11], [0, 11], [[0], [1]]) == (1, False)   # more than there are
    assert call([0, 0, 10], [0, 17], [[0], [1]]) == (1, False)   # more than the table holds
    assert call([0, 0, 10], [0, 10], [[0], [99]]) == (1, False)  # no such page
    assert call([0, 0, 10], [-1, 10], [[0], [1]])[0] == 1        # told, though no token leads there
    assert fa.fa_get_status() == 0
