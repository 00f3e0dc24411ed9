"""NaN codes of V in a cache of 8 bits: they reach the rows that see their keys, in
their columns, and no others.

The reference takes them as zeros, so the bounds are cache8_util's, and sets NaN where
a visible key has one.
"""
import math

import numpy as np
import pytest
import torch

from oracle import attn_ref
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


def run(fa, new, keys, hq, hk, d, page, seed, places, causal=True, window=None):
    """places: per sequence the keys (from the end if negative) that have NaN codes, each in
    columns and a head of its own."""
    c = cu8.filled(keys, hk, d, page, seed)
    codes = c.codes[1].view(torch.uint8)
    cu = su.starts(new)
    bad = torch.zeros((sum(new), hq, d), dtype=torch.bool)
    for b, ks in enumerate(places):
        see = attn_ref.visible_mask(np.arange(new[b]), new[b], keys[b], causal, window) if new[b] else np.zeros((0, keys[b]))
        for i, k in enumerate(ks):
            k %= keys[b]
            head, cols = i % hk, [(7 * i) % d, (7 * i + 33) % d, d - 1 - i]
            page_of, row = int(c.table[b, k // page]), k % page
            codes[page_of, row, head, cols] = 0x7F if i % 2 else 0xFF
            group = hq // hk
            for r in np.flatnonzero(see[:, k]):
                bad[int(cu[b]) + r, head * group:(head + 1) * group, cols] = True
    pages, table = c.cuda()
    q = su.normal((sum(new), hq, d), su.gen(seed))
    o, lse = fa.forward_paged_fp8(q.cuda(), *pages, cu.cuda(), c.lens_k().cuda(), table, causal=causal, window=window)
    assert fa.fa_get_status() == 0
    codes[(codes & 0x7F) == 0x7F] = 0
    seqs = [(q[cu[b]:cu[b + 1]], *c.values(b)) for b in range(len(new))]
    want = su.reference(seqs, d ** -0.5, causal, window)
    assert torch.equal(o.cpu().isnan(), bad)
    ref = torch.from_numpy(np.concatenate([w[0] for w in want]))
    cu8.check_forward(torch.where(bad, ref, o.cpu().double()), lse, want, seqs, cu)
    return bad


# new tokens, keys, query heads, kv heads, places, window: few rows to a kv head
FEW = [
    ([4], [300], 4, 1, [[-1, -2, 100]], None),               # a chunk's own last tokens
    ([2], [290], 4, 1, [[-1]], None),
    ([4], [300], 8, 2, [[-1, -3, -4, 5, 299, 0]], None),
    ([1, 3], [700, 33], 4, 1, [[0, 350, -1], [-1, -2, 1]], None),
    ([10], [4], 1, 1, [[0, 1, 3]], None),                    # rows that see nothing
    ([4], [9000], 4, 1, [[-1, 17, 5000, -3]], None),         # keys divided
    ([4], [9000], 4, 1, [[-1, 17, 8979, 8980, 8981]], (16, 0)),  # behind the window, in a block with keys in it
    ([3, 1], [500, 400], 4, 1, [[480, 470, 499, 0], [399, 398, 380, 371]], (20, 0)),
    ([3], [500], 2, 1, [[-1, 489, 400]], (10, 1)),
    ([1] * 9, [40 * i + 1 for i in range(9)], 16, 1, [[-1, -17]] * 9, (16, 0)),
]


@pytest.mark.parametrize("new,keys,hq,hk,places,window", FEW)
@pytest.mark.parametrize("d", [64, 128])
def test_few_rows(fa, new, keys, hq, hk, places, window, d):
    bad = run(fa, new, keys, hq, hk, d, 16, 31, places, window=window)
    assert bad.any() and not bad.flatten(1).all()


def test_few_rows_without_a_mask(fa):
    run(fa, [3], [300], 4, 1, 128, 32, 32, [[0, -1]], causal=False)


def test_few_rows_in_larger_pages(fa):
    run(fa, [4, 2], [600, 129], 4, 2, 64, 64, 33, [[-1, -2, 128], [-1, 128]], window=(128, 0))


# many rows
MANY = [
    ([200], [333], 4, 1, [[-1, -2, -100, 50, 332, 133, 127, 128]], None),
    ([513], [513], 4, 2, [[-1, 0, 250, 511, 300, 7]], None),          # a whole prompt
    ([300], [129], 4, 1, [[0, 64, -1]], None),                         # rows that see nothing
    ([20], [6000], 4, 1, [[-1, -5, 30, 4000, -20]], None),            # keys divided, one tile of rows
    ([40], [6000], 4, 1, [[-1, 5944, 5900, 5855, 3, -39]], (100, 0)),  # divided, behind the window
    ([100, 1, 0, 70], [900, 333, 20, 70], 8, 2, [[-1, 799, 700, 860], [-1, 300, 331], [0], [-1, 0, 69, 35]], (64, 0)),
    ([200], [333], 2, 1, [[-1, 100, 140, 240, 2]], (20, 1)),
    ([1, 260], [400, 500], 32, 1, [[-1, 100, 380], [-1, 240, 499, 370]], (300, 0)),
    ([60, 200, 33], [700, 333, 33], 20, 4, [[-1, 600, 640, 5], [-1, -40, 199, 150], [-1, 3]], None),
]


@pytest.mark.parametrize("new,keys,hq,hk,places,window", MANY)
@pytest.mark.parametrize("d", [64, 128])
def test_many_rows(fa, new, keys, hq, hk, places, window, d):
    bad = run(fa, new, keys, hq, hk, d, 16, 34, places, window=window)
    assert bad.any() and not bad.flatten(1).all()


@pytest.mark.parametrize("d", [64, 128])
def test_many_rows_many_items_per_cta(fa, d):
    g = torch.Generator().manual_seed(d)
    new = [1 + i % 5 if i % 3 else int(n) for i, n in enumerate(torch.randint(1, 200, (40,), generator=g))]
    keys = [n + int(m) for n, m in zip(new, torch.randint(0, 500, (40,), generator=g))]
    places = [[-1, keys[b] // 2, keys[b] - new[b] // 2 - 1] if b % 4 == 0 else [] for b in range(40)]
    run(fa, new, keys, 16, 8, d, 16, 35, places)
    run(fa, new, keys, 16, 8, d, 32, 36, places, window=(50, 0))


def test_many_rows_without_a_mask(fa):
    run(fa, [90], [300], 4, 1, 128, 48, 37, [[0, -1, 150]], causal=False)
