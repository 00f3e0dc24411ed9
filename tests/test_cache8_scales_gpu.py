"""fa_cache_append_fp8 into blocks whose scale is no power of two (something else filled them).

The reference takes quotients and products in fp64, which tells them from halfway between two
codes: a bf16 value over a 24-bit scale, or a code times one, that is not halfway is off it by
more than 2^-32 of itself. Values are chosen so that a scale is the fp32 number nearest to
the one that would put them halfway: where fp32 says halfway and the value is not."""
import numpy as np
import pytest
import torch

from tests import cache8_util as cu8
from tests import seq_util as su

pytestmark = pytest.mark.gpu

TABLE = torch.arange(127, dtype=torch.uint8).view(cu8.E4M3).double().numpy()  # the codes' magnitudes
HALVES = (TABLE[1:] + TABLE[:-1]) / 2


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    m.fa_debug_set(0, 0)
    return m


def nearest(y):
    """Codes (uint8) of fp64 values of magnitude 448 at most, ties to even."""
    a = np.abs(y)
    i = np.searchsorted(HALVES, a)  # the code below the half that is not below a
    up = (i < 126) & (a == HALVES[np.minimum(i, 125)]) & (i % 2 == 1)
    return ((i + up) | np.where(np.signbit(y), 0x80, 0)).astype(np.uint8)


def halfway_scale(x, rng):
    """fp32 scales with which x is near halfway between two codes, no powers of two."""
    h = rng.choice(HALVES[(HALVES > 2.0 ** -6) & (HALVES < 210)], x.shape)  # (so that the scale holds x, and stays)
    s = (x / h).astype(np.float32)
    return np.where(np.frexp(s)[0] == 0.5, s * np.float32(1.5), s)


def setup(rng, hk, d, held):
    """Pages of 16 with `held` rows of codes in each of two sequences' one block."""
    codes = [torch.from_numpy(rng.integers(0, 120, (2, 16, hk, d)).astype(np.uint8) | rng.choice([0, 0x80], (2, 16, hk, d)).astype(np.uint8))
             for _ in range(2)]
    return codes, torch.tensor([[0], [1]], dtype=torch.int32)


def run(fa, codes, scales, table, k, v, cu, lens):
    pages = [x.cuda().view(cu8.E4M3) for x in codes] + [torch.from_numpy(s).cuda() for s in scales]
    fa.cache_append_fp8(k.cuda(), v.cuda(), *pages, cu.cuda(), lens.cuda(), table.cuda())
    assert fa.fa_get_status() == 0
    return [x.view(torch.uint8).cpu().numpy() for x in pages[:2]], [x.cpu().numpy() for x in pages[2:]]


@pytest.mark.parametrize("held,new", [(1, 1), (5, 2), (3, 13), (15, 1)])
@pytest.mark.parametrize("d", [64, 128])
def test_new_rows_over_a_scale_that_stays(fa, d, held, new):
    rng, hk = np.random.default_rng(held + d), 8
    codes, table = setup(rng, hk, d, held)
    base = su.normal((2, hk), su.gen(d)).double().abs().numpy() + 0.01
    base = torch.from_numpy(base).to(torch.bfloat16).double().numpy()
    scales = [halfway_scale(base, rng)[:, None, :] for _ in range(2)]
    xs = []
    for s in scales:  # rows: the head's value and halves of it, of both signs; and any others that the scale holds
        x = np.where(rng.random((2, new, hk, d)) < 0.5, base[:, None, :, None] * rng.choice([1.0, -0.5, 0.25], (2, new, hk, d)),
                     rng.uniform(-440, 440, (2, new, hk, d)) * s[:, :, :, None])
        top = 440.0 * np.exp2(np.floor(np.log2(s)))[:, :, :, None]  # (the power of two that x wants is no larger)
        x = torch.from_numpy(np.clip(x, -top, top)).to(torch.bfloat16)
        xs.append(x)
    cu, lens = su.starts([new, new]), torch.tensor([held + new] * 2, dtype=torch.int32)
    got, got_scales = run(fa, codes, scales, table, xs[0].flatten(0, 1), xs[1].flatten(0, 1), cu, lens)
    for x, c, s, g, gs in zip(xs, codes, scales, got, got_scales):
        assert np.array_equal(gs, s)
        want = c.numpy().copy()
        want[:, held:held + new] = nearest(x.double().numpy() / s.astype(np.float64)[:, :, :, None])
        assert np.array_equal(g, want)


@pytest.mark.parametrize("held", [1, 6, 15])
@pytest.mark.parametrize("d", [64, 128])
def test_held_rows_of_a_scale_that_rises(fa, d, held):
    rng, hk = np.random.default_rng(held + d), 8
    codes, table = setup(rng, hk, d, held)
    scales = []
    for c in codes:  # the first held code of each head comes halfway in the new scale, which is 1
        first = np.maximum(TABLE[c.numpy()[:, 0, :, 0] & 0x7F], 2.0 ** -6)
        h = rng.choice(HALVES[8:40], first.shape)
        s = (h / first).astype(np.float32)
        s = np.where(s >= 1, s / np.float32(2.0) ** np.floor(np.log2(s) + 1), s).astype(np.float32)
        scales.append(np.where(np.frexp(s)[0] == 0.5, s * np.float32(0.75), s)[:, None, :])
    x = torch.full((2, hk, d), 300.0, dtype=torch.bfloat16)
    x[:, :, 1] = -448.0
    cu, lens = su.starts([1, 1]), torch.tensor([held + 1] * 2, dtype=torch.int32)
    got, got_scales = run(fa, codes, scales, table, x, x, cu, lens)
    for c, s, g, gs in zip(codes, scales, got, got_scales):
        assert (gs == 1.0).all()
        want = c.numpy().copy()
        old = want[:, :held]
        value = TABLE[old & 0x7F] * np.where(old & 0x80, -1.0, 1.0) * s.astype(np.float64)[:, :, :, None]
        want[:, :held] = nearest(value)
        want[:, held] = nearest(x.double().numpy())
        assert np.array_equal(g, want)
