"""fa_fwd_varlen on the GPU: packed sequences of different lengths against
the 64-bit oracle, one sequence at a time."""
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


def case(nq, nk, hq, hk, d, seed, fused=False, before=0, behind=0):
    """Packed q, k, v (bits that no sequence owns are NaN), offsets, per-sequence views."""
    g = su.gen(seed)
    tq, tk = before + sum(nq) + behind, before + sum(nk) + behind
    cq, ck = su.starts(nq, before), su.starts(nk, before)
    if fused:
        assert nq == nk
        x = su.normal((tq, hq + 2 * hk, d), g)
        q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    else:
        q, k, v = su.normal((tq, hq, d), g), su.normal((tk, hk, d), g), su.normal((tk, hk, d), g)
    for t, cu in ((q, cq), (k, ck), (v, ck)):
        t[:before] = math.nan
        t[cu[-1]:] = math.nan
    seqs = [(q[cq[b]:cq[b + 1]], k[ck[b]:ck[b + 1]], v[ck[b]:ck[b + 1]]) for b in range(len(nq))]
    if fused:
        x = x.cuda()
        dev = (x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:])
    else:
        dev = (q.cuda(), k.cuda(), v.cuda())
    return dev, cq, ck, seqs


def run(fa, nq, nk, hq, hk, d, seed, causal=True, window=None, scale=None, fused=False, before=0, behind=0):
    (q, k, v), cq, ck, seqs = case(nq, nk, hq, hk, d, seed, fused, before, behind)
    scale = d ** -0.5 if scale is None else scale
    o = torch.full((q.shape[0], hq, d), 7.0, device="cuda", dtype=torch.bfloat16)
    lse = torch.full((hq, q.shape[0]), 7.0, device="cuda")
    fa.forward_varlen(q, k, v, cq.cuda(), ck.cuda(), causal=causal, window=window, scale=scale, out=(o, lse))
    assert fa.fa_get_status() == 0
    su.check_forward(o, lse, su.reference(seqs, scale, causal, window), cq)
    # rows of no sequence keep what they had
    for t in (o[:before], o[cq[-1]:], lse[:, :before], lse[:, cq[-1]:]):
        assert (t == 7.0).all()
    return o, lse


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 2), (6, 2), (5, 1), (7, 1), (8, 1)])
def test_heads(fa, hq, hk, d):
    n = [1, 130, 0, 37, 257]
    run(fa, n, n, hq, hk, d, seed=1)


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 127, 128, 129, 255, 256, 257, 640])
@pytest.mark.parametrize("causal", [False, True])
def test_lengths(fa, n, causal):
    run(fa, [n], [n], 4, 2, 128, seed=n, causal=causal)


@pytest.mark.parametrize("nq,nk", [([5, 300], [300, 5]), ([1, 1, 1], [1000, 0, 129]), ([64, 0, 200], [0, 50, 513]),
                                   ([0, 0], [10, 0]), ([400], [700])])
@pytest.mark.parametrize("causal,window", [(True, None), (False, None), (False, (20, 5)), (True, (64, 0)), (False, (0, 0)),
                                           (False, (-1, 3)), (False, (3, -1))])
def test_masks_and_empty_rows(fa, nq, nk, causal, window):
    run(fa, nq, nk, 4, 2, 64, seed=3, causal=causal, window=window)


@pytest.mark.parametrize("hq,hk,d", [(8, 2, 128), (3, 1, 64)])
def test_fused_projection_and_rows_around(fa, hq, hk, d):
    n = [200, 1, 77]
    run(fa, n, n, hq, hk, d, seed=4, fused=True, before=3, behind=9)


@pytest.mark.parametrize("scale", [0.0, -0.1, 0.5])
def test_scales(fa, scale):
    run(fa, [150, 40], [150, 40], 2, 2, 128, seed=5, scale=scale)


def test_many_sequences(fa):
    rng = torch.Generator().manual_seed(6)
    n = torch.randint(0, 9, (1500,), generator=rng).tolist()
    run(fa, n, n, 2, 1, 64, seed=6)


def test_many_empty_sequences(fa):
    n = [0] * 4000
    n[7], n[2000], n[3999] = 40, 3, 300
    run(fa, n, n, 4, 2, 128, seed=61)


@pytest.mark.parametrize("hq,hk,d", [(16, 8, 128), (24, 8, 64), (20, 20, 128)])
def test_many_items_per_cta(fa, hq, hk, d):
    # long and short units mixed, several to a CTA
    rng = torch.Generator().manual_seed(hq)
    n = torch.randint(0, 420, (36,), generator=rng).tolist()
    run(fa, n, n, hq, hk, d, seed=hq)


def test_group_of_128(fa):
    run(fa, [5, 3], [300, 3], 128, 1, 64, seed=7)


def test_whole_keys_divided_between_ctas(fa):
    # one row block, many key tiles: the keys are divided and joined again
    run(fa, [256], [5000], 1, 1, 128, seed=8, causal=False)
    run(fa, [300, 20], [3000, 4000], 2, 1, 64, seed=9)


def test_as_the_dense_call(fa):
    # a batch of equal lengths gives what fa_fwd gives, up to the order of additions
    B, N, hq, hk, d = 3, 384, 4, 2, 128
    (q, k, v), cq, _, seqs = case([N] * B, [N] * B, hq, hk, d, 10)
    o, lse = fa.forward_varlen(q, k, v, cq.cuda(), cq.cuda(), causal=True)
    do, dl = fa.forward(q.view(B, N, hq, d), k.view(B, N, hk, d), v.view(B, N, hk, d), causal=True)
    want = su.reference(seqs, d ** -0.5, True)
    su.check_forward(o, lse, want, cq)
    su.check_forward(do.view(-1, hq, d), dl.permute(1, 0, 2).reshape(hq, -1), want, cq)
