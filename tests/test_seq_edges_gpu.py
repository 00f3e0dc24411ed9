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
