"""fa_rotary on the GPU against the formula in 64 bits.

Bound, for a pair (a, b) and factor m: the angle is off by at most 2^-25 half turns
(its rounding to fp32) and 2^-31 (its cut to 32 bits), together below 2^-23
radians; sincospif by 2 ulp (2^-23), the product with m by 2^-24, the two
products and their sum by 2^-24 each of their terms: below 2^-20 m (|a| + |b|)
in all; and the result is rounded to bf16, 2^-8 of itself and of that."""
import math

import numpy as np
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


def pairs(d, rot, interleaved):
    j = np.arange(rot // 2)
    return (2 * j, 2 * j + 1) if interleaved else (j, j + rot // 2)


def turned(x, place, inv_freq, interleaved, m, back=False):
    """x [n, heads, d] (fp64); returns it turned and the bound."""
    rot = 2 * len(inv_freq)
    t = np.outer(place.astype(np.float64), inv_freq) * (-1.0 if back else 1.0)
    ia, ib = pairs(x.shape[2], rot, interleaved)
    a, b = x[:, :, ia], x[:, :, ib]
    co, si = m * np.cos(t)[:, None], m * np.sin(t)[:, None]
    y, e = x.copy(), np.zeros_like(x)
    y[:, :, ia], y[:, :, ib] = a * co - b * si, b * co + a * si
    # numpy's own reduction of t: exact to 2^-53 of t
    err = (2.0 ** -20 + 2.0 ** -52 * np.abs(t)[:, None]) * abs(m) * (np.abs(a) + np.abs(b))
    e[:, :, ia] = e[:, :, ib] = err
    out = np.zeros(x.shape, bool)
    out[:, :, ia] = out[:, :, ib] = True
    return y, np.where(out, 2.0 ** -8 * (np.abs(y) + e) + e, 0.0)


def check(got, want, bound):
    off = np.abs(su.n64(got) - want) - bound
    assert off.size == 0 or (off <= 0).all(), f"{off.max():.3e} beyond the bound at {np.unravel_index(off.argmax(), off.shape)}"


def run(fa, new, ctx, hq, hk, d, rot, interleaved, seed, m=1.0, fused=False, in_place=False, base=10000.0, lens=True):
    g = su.gen(seed)
    total = sum(new)
    wide = su.normal((total, hq + (2 if fused else 1) * hk, d), g)
    dev = wide.cuda()
    q, k = wide[:, :hq], wide[:, hq:hq + hk]
    dq, dk = dev[:, :hq], dev[:, hq:hq + hk]
    f, _ = fa.rotary_frequencies(rot, base)
    cu = su.starts(new).cuda()
    ln = torch.tensor([n + c for n, c in zip(new, ctx)], dtype=torch.int32).cuda() if lens else None
    place = np.concatenate([np.arange(n) + (c if lens else 0) for n, c in zip(new, ctx)]).astype(np.int64)
    kw = dict(interleaved=interleaved, mscale=m, out=(dq, dk) if in_place else None)
    yq, yk = fa.rotary(dq, dk, f.cuda(), cu, ln, **kw)
    assert fa.fa_get_status() == 0
    f64 = f.double().numpy()
    for x, y in ((q, yq), (k, yk)):
        check(y, *turned(su.n64(x), place, f64, interleaved, m))
    # outside q and k nothing is written
    if in_place and fused:
        assert torch.equal(dev[:, hq + hk:].cpu(), wide[:, hq + hk:])
    if not in_place:
        assert torch.equal(dev.cpu(), wide)
        gq, gk = fa.rotary_backward(yq, yk, f.cuda(), cu, ln, interleaved=interleaved, mscale=m)
        for x, y in ((yq, gq), (yk, gk)):
            check(y, *turned(su.n64(x), place, f64, interleaved, m, back=True))


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 16), (64, 48), (64, 64), (128, 16), (128, 64), (128, 80), (128, 128)])
def test_layouts(fa, d, rot, interleaved):
    run(fa, [1, 30, 0, 77], [5, 0, 9, 1000], 6, 2, d, rot, interleaved, seed=rot, m=1.25, fused=True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rot", [32, 128])
def test_in_place(fa, rot, interleaved):
    run(fa, [20, 3], [0, 100], 4, 4, 128, rot, interleaved, seed=rot, fused=True, in_place=True)


@pytest.mark.parametrize("hq,hk", [(1, 1), (32, 8), (33, 11), (200, 1)])
@pytest.mark.parametrize("n", [1, 2, 700])
def test_heads(fa, hq, hk, n):
    run(fa, [n], [17], hq, hk, 128, 128, False, seed=hq)


def test_far_places(fa):
    # (numpy's angle is exact to 2^-53 of it: 2^-30 here)
    run(fa, [3, 5, 2, 1], [100000, 1 << 20, (1 << 24) + 1, 2 ** 31 - 2], 2, 1, 64, 64, False, seed=3)


def test_places_without_lengths(fa):
    run(fa, [300, 1, 45], [0, 0, 0], 8, 2, 64, 32, True, seed=4, lens=False)


def test_many_sequences(fa):
    g = su.gen(5)
    n = torch.randint(0, 4, (3000,), generator=g).tolist()
    run(fa, n, [i % 57 for i in range(3000)], 2, 1, 64, 64, False, seed=5)


def test_long(fa):
    run(fa, [9000, 2000], [0, 4096], 8, 2, 128, 128, False, seed=6, fused=True)


@pytest.mark.parametrize("freq", [0.0, 1.0, -0.5, 3.0, 1e4, 2.0 ** 24, 2.0 ** 30, 1e-20, 1e-42, 2.0 ** -126])
def test_any_frequency(fa, freq):
    g = su.gen(7)
    x = su.normal((50, 1, 64), g)
    f = torch.full((8,), freq)
    y, none = fa.rotary(x.cuda(), None, f.cuda(), su.starts([50]).cuda())
    assert none is None and fa.fa_get_status() == 0
    f64 = f.double().numpy()
    # turns by exact integers: p f / 2 pi in 200 bits
    from fractions import Fraction
    pi = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286209, 10 ** 78)
    t = [float((Fraction(p) * Fraction(float(f64[0])) / (2 * pi)) % 1) * 2.0 * math.pi for p in range(50)]
    a, b = su.n64(x)[:, 0, :8], su.n64(x)[:, 0, 8:16]
    co, si = np.cos(t)[:, None], np.sin(t)[:, None]
    got = su.n64(y)[:, 0]
    # (the turn's fraction itself is off by p f 2^-64 at most, below 2^-20 here)
    tol = (2.0 ** -20 + 50 * abs(freq) * 2.0 ** -60) * (np.abs(a) + np.abs(b))
    for z, w in ((got[:, :8], a * co - b * si), (got[:, 8:16], b * co + a * si)):
        assert (np.abs(z - w) <= 2.0 ** -8 * (np.abs(w) + tol) + tol).all()


def test_gradient_by_differences(fa):
    # L = sum(w * rotary(x)): linear in x, so that a difference is exact up to the outputs' roundings
    g = su.gen(8)
    x, w = su.normal((6, 2, 64), g), su.normal((6, 2, 64), g)
    f, m = fa.rotary_frequencies(32, scaling="yarn", factor=4.0, original_length=64)
    cu, ln = su.starts([6]).cuda(), torch.tensor([40], dtype=torch.int32).cuda()
    grad, _ = fa.rotary_backward(w.cuda(), None, f.cuda(), cu, ln, mscale=m)
    place = np.arange(34, 40)
    for i in range(64):
        e = torch.zeros_like(x)
        e[:, :, i] = 1.0
        y = su.n64(fa.rotary(e.cuda(), None, f.cuda(), cu, ln, mscale=m)[0])
        got = su.n64(grad)[:, :, i]
        want = (su.n64(w) * y).sum(2)
        # two values of y, each rounded to bf16, and the gradient's rounding
        bound = 2.0 ** -7 * (np.abs(su.n64(w)) * np.abs(y)).sum(2) + 2.0 ** -8 * np.abs(want) + 1e-6
        assert (np.abs(got - want) <= bound).all()
    assert len(place) == 6


def test_rows_outside_and_bad_lengths(fa):
    x = su.normal((20, 2, 64), su.gen(9)).cuda()
    f = fa.rotary_frequencies(64)[0].cuda()

    def call(cu, lens):
        y = torch.full_like(x, 7.0)
        fa.rotary(x, None, f, torch.tensor(cu, dtype=torch.int32).cuda(),
                  None if lens is None else torch.tensor(lens, dtype=torch.int32).cuda(), out=(y, None))
        return fa.fa_get_status(), (y == 7.0).flatten(1).all(1).cpu().tolist()

    st, left = call([4, 9, 15], None)
    assert st == 0 and left == [not 4 <= i < 15 for i in range(20)]
    assert call([0, 21], None) == (1, [True] * 20)
    assert call([0, 5, 10], [4, 20])[0] == 1      # the first has more rows than places
    assert call([0, 5, 10], [4, 20])[1][:5] == [True] * 5
    assert call([0, 0, 5], [-3, 5])[0] == 1       # told, though no token leads there
    assert fa.fa_get_status() == 0


def test_far_apart_tokens(fa):
    # offsets past 2^32 bytes: rows 2^24 elements apart
    big = torch.empty((260 << 24) // 2, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(big, (129, 1, 64), (1 << 24, 64, 1))
    x.copy_(su.normal((129, 1, 64), su.gen(10)))
    f = fa.rotary_frequencies(64)[0].cuda()
    cu = su.starts([129]).cuda()
    y, _ = fa.rotary(x, None, f, cu)
    z, _ = fa.rotary(x.contiguous(), None, f, cu)
    assert torch.equal(y, z)
