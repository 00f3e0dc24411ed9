"""fa_rotary with any finite frequency at any place, against angles by exact integers
(test_rotary_gpu's bound: the angle below 2^-23 radians, all in all 2^-20 (|a| + |b|))."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

from tests import seq_util as su

pytestmark = pytest.mark.gpu

PI = Fraction(3141592653589793238462643383279502884197169399375105820974944592307816406286209, 10 ** 78)


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.fa_debug_set(0, 0)
    return m


@pytest.mark.parametrize("freqs", [[1.0, -1.9999999, 2.0, 2.5, -7.0, 255.0, 300.25, 4097.0],
                                   [1e5, 2.0 ** 20 + 1, -2.0 ** 24 + 1, 2.0 ** 25, 2.0 ** 26 + 8, 2.0 ** 30, 3e10, -1e13],
                                   [2.0 ** 63, 2.0 ** 64, 2.0 ** 88, -2.0 ** 89, 2.0 ** 90, 1.7e30, 3.4e38, -1e38],
                                   [1e-45, 2.0 ** -126, -1e-30, 2.0 ** -40, 1e-9, 0.1, 0.99999994, 0.0]])
@pytest.mark.parametrize("interleaved", [False, True])
def test_frequencies_at_far_places(fa, freqs, interleaved):
    # (pi above has 78 digits, 2^-258: of 2^128 * 2^31 turns 2^-99 are left)
    ends = [2 ** 31 - 1, 2 ** 31 - 7, (1 << 30) + 3, 12345678, 4, 70000]
    new = [4, 1, 3, 2, 4, 1]
    x = su.normal((sum(new), 2, 64), su.gen(1))
    f = torch.tensor(freqs)
    y, _ = fa.rotary(x.cuda(), None, f.cuda(), su.starts(new).cuda(), torch.tensor(ends, dtype=torch.int32).cuda(),
                     interleaved=interleaved)
    assert fa.fa_get_status() == 0
    places = [e - n + i for e, n in zip(ends, new) for i in range(n)]
    t = np.array([[float(Fraction(p) * Fraction(v) / (2 * PI) % 1) * 2.0 * math.pi for v in f.tolist()] for p in places])
    a, b = np.arange(8) * 2 if interleaved else np.arange(8), np.arange(8) * 2 + 1 if interleaved else np.arange(8) + 8
    xa, xb, got = su.n64(x)[:, :, a], su.n64(x)[:, :, b], su.n64(y)
    co, si = np.cos(t)[:, None], np.sin(t)[:, None]
    tol = 2.0 ** -20 * (np.abs(xa) + np.abs(xb))
    for z, w in ((got[:, :, a], xa * co - xb * si), (got[:, :, b], xb * co + xa * si)):
        off = np.abs(z - w) - (2.0 ** -8 * (np.abs(w) + tol) + tol)
        assert (off <= 0).all(), f"{off.max():.3e} beyond its bound"
