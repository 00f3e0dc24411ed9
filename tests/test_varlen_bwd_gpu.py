"""fa_bwd_varlen on the GPU: gradients of packed sequences against the 64-bit
formulas and against differences of the 64-bit forward."""
import math

import numpy as np
import pytest
import torch

from oracle import attn_ref
from tests import seq_util as su
from tests.test_varlen_gpu import case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.fa_debug_set(0, 0)
    return m


def run(fa, nq, nk, hq, hk, d, seed, causal=True, window=None, scale=None, fused=False, before=0, behind=0):
    (q, k, v), cq, ck, seqs = case(nq, nk, hq, hk, d, seed, fused, before, behind)
    scale = d ** -0.5 if scale is None else scale
    dout = su.normal((q.shape[0], hq, d), su.gen(seed + 1000))
    dout[:before] = math.nan
    dout[cq[-1]:] = math.nan
    kw = dict(causal=causal, window=window, scale=scale)
    cqd, ckd = cq.cuda(), ck.cuda()
    o, lse = fa.forward_varlen(q, k, v, cqd, ckd, **kw)
    got = [torch.full(s, 7.0, device="cuda", dtype=torch.bfloat16)
           for s in ((q.shape[0], hq, d), (k.shape[0], hk, d), (k.shape[0], hk, d))]
    fa.backward_varlen(q, k, v, o, lse, dout.cuda(), cqd, ckd, out=got, **kw)
    assert fa.fa_get_status() == 0
    douts = [dout[cq[b]:cq[b + 1]] for b in range(len(nq))]
    outs = [o[int(cq[b]):int(cq[b + 1])].cpu() for b in range(len(nq))]
    su.check_backward(got, su.reference_backward(seqs, douts, outs, scale, causal, window), cq, ck)
    for t, cu in zip(got, (cq, ck, ck)):  # rows of no sequence keep what they had
        assert (t[:before] == 7.0).all() and (t[int(cu[-1]):] == 7.0).all()
    return got


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (4, 2), (6, 2), (5, 1), (7, 1), (8, 1)])
def test_heads(fa, hq, hk, d):
    n = [1, 130, 0, 37, 257]
    run(fa, n, n, hq, hk, d, seed=1)


@pytest.mark.parametrize("n", [1, 2, 31, 33, 127, 128, 129, 256, 300, 640])
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
    n = torch.randint(0, 9, (700,), generator=rng).tolist()
    run(fa, n, n, 2, 1, 64, seed=6)


@pytest.mark.parametrize("B", [31, 32, 33, 255, 256, 257])
def test_numbers_of_sequences(fa, B):
    rng = torch.Generator().manual_seed(B)
    n = torch.randint(0, 70, (B,), generator=rng).tolist()
    run(fa, n, n, 3, 1, 64, seed=B)


def test_many_empty_sequences(fa):
    n = [0] * 4000
    n[7], n[2000], n[3999] = 40, 3, 300
    run(fa, n, n, 4, 2, 128, seed=61)


@pytest.mark.parametrize("hq,hk,d", [(16, 8, 128), (24, 8, 64)])
def test_many_items_per_cta(fa, hq, hk, d):
    rng = torch.Generator().manual_seed(hq)
    n = torch.randint(0, 420, (40,), generator=rng).tolist()
    run(fa, n, n, hq, hk, d, seed=hq)


def test_group_of_128(fa):
    run(fa, [5, 3], [300, 3], 128, 1, 64, seed=7)


def test_long_sequences_in_whole_units_and_divided(fa):
    run(fa, [1200], [1200], 2, 1, 128, seed=8)                    # few key tiles: divided
    run(fa, [300, 300, 290], [300, 300, 290], 16, 16, 64, seed=9)  # many: whole


def test_against_differences(fa):
    # the directional derivative of L = sum(dO O) along each gradient, by central
    # differences of the 64-bit forward: relative error of the difference h^2,
    # of the bf16 gradients 2^-8 each way (they are the direction too, so their
    # own rounding moves the norm by at most 2 * 2^-7)
    n, hq, hk, d = [60, 33], 2, 1, 64
    (q, k, v), cq, _, seqs = case(n, n, hq, hk, d, 12)
    dout = su.normal((sum(n), hq, d), su.gen(13))
    c = cq.cuda()
    o, lse = fa.forward_varlen(q, k, v, c, c, causal=True)
    grads = fa.backward_varlen(q, k, v, o, lse, dout.cuda(), c, c, causal=True)
    base = [su.n64(t) for t in (q, k, v)]
    do = su.n64(dout)

    def loss(x):
        t = 0.0
        for b in range(2):
            r = slice(int(cq[b]), int(cq[b + 1]))
            t += (attn_ref.forward(x[0][None, r], x[1][None, r], x[2][None, r], d ** -0.5, True)[0][0] * do[r]).sum()
        return t

    for i in range(3):
        g = su.n64(grads[i])
        norm = np.sqrt((g * g).sum())
        h = 1e-4
        hi, lo = list(base), list(base)
        hi[i], lo[i] = base[i] + h * g / norm, base[i] - h * g / norm
        assert abs((loss(hi) - loss(lo)) / (2 * h) - norm) <= 2.0 ** -6 * norm, i


def test_same_inputs_same_dk_dv(fa):
    a = run(fa, [700, 90], [700, 90], 8, 2, 128, seed=14)
    b = run(fa, [700, 90], [700, 90], 8, 2, 128, seed=14)
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
