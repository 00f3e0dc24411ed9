"""Host-only checks of the rotary and 8-bit cache calls: bad arguments are
refused before any device work, and the frequencies' formulas."""
import math

import pytest
import torch

from tests.test_seq_abi import APPEND, OF_KV, OF_PAGES, OF_Q, P16, PAGED, SHARED


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    m.lib()
    return m


def with_scales(base, after):
    out = {}
    for n, v in base.items():
        out[n] = v
        if n == after:
            out["k_scales"] = out["v_scales"] = P16
    return out


ROTARY = dict(q=P16, k=P16, q_out=P16, k_out=P16, inv_freq=P16, cu_q=P16, lens=P16, B=2, Hq=4, Hk=2, total=50, d=128, rot=64,
              q_stride=512, k_stride=256, q_out_stride=512, k_out_stride=256, mscale=1.0, interleaved=0, transposed=0)
CALLS = {"fa_fwd_paged_fp8": with_scales(PAGED, "v_pages"), "fa_cache_append_fp8": with_scales(APPEND, "v_pages"),
         "fa_rotary": ROTARY}
FOUR = ("cu_q", "lens_k", "lens", "page_table", "k_scales", "v_scales", "inv_freq")


def call(fa, name, **kw):
    a = dict(CALLS[name])
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(fa, name)(*a.values(), 0)


BAD = ([("fa_fwd_paged_fp8", b, c) for b, c in SHARED + OF_Q + OF_PAGES]
       + [("fa_cache_append_fp8", b, c) for b, c in SHARED + OF_KV + OF_PAGES]
       + [("fa_rotary", b, c) for b, c in [
           (dict(B=0), 1), (dict(Hq=-1), 1), (dict(Hk=-1), 1), (dict(Hq=0, Hk=0), 1), (dict(total=-1), 1), (dict(d=0), 1),
           (dict(d=96), 2), (dict(d=256, rot=256), 2), (dict(rot=0), 2), (dict(rot=8), 2), (dict(rot=24), 2),
           (dict(rot=-16), 1), (dict(rot=144), 1), (dict(total=1 << 29), 2), (dict(B=1 << 29), 2),
           (dict(q_stride=504), 1), (dict(k_stride=255), 1), (dict(q_out_stride=500), 1), (dict(k_out_stride=248), 1),
           (dict(k_stride=1 << 39), 2), (dict(total=1 << 26, q_out_stride=1 << 37), 2), (dict(mscale=float("nan")), 1),
           (dict(mscale=float("inf")), 1), (dict(interleaved=2), 1), (dict(transposed=-1), 1),
           (dict(q_out_stride=1024), 1),  # in place, but other rows
           (dict(Hq=1 << 23, q_stride=1 << 30), 2), (dict(total=1 << 28, Hq=8, q_stride=1024), 2)]])


@pytest.mark.parametrize("name,bad,code", BAD)
def test_bad_sizes(fa, name, bad, code):
    assert call(fa, name, **bad) == code


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_pointers(fa, name):
    for arg, v in CALLS[name].items():
        if v == P16:
            if arg != "lens":  # (may be null)
                assert call(fa, name, **{arg: 0}) == 1, arg
            assert call(fa, name, **{arg: P16 + 2}) == 1, arg
            if arg not in FOUR:
                assert call(fa, name, **{arg: P16 + 8}) == 1, arg


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
@pytest.mark.parametrize("name", list(CALLS))
def test_good_arguments_reach_the_device_check(fa, name):
    assert call(fa, name) == 6
    total = "total" if name == "fa_rotary" else "total_q"
    assert call(fa, name, **{total: 0}) == 6
    if name == "fa_rotary":
        assert call(fa, name, lens=0) == 6
        assert call(fa, name, Hq=0, q=0, q_out=0, q_stride=0, q_out_stride=0) == 6
        assert call(fa, name, Hk=0, k=0, k_out=0, k_stride=0, k_out_stride=0) == 6
        assert call(fa, name, q_out=P16 + 4096, q_out_stride=1024) == 6


def test_python_checks(fa):
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    p, s = torch.zeros(1, 16, 2, 64, dtype=torch.uint8).view(torch.float8_e4m3fn), torch.zeros(1, 1, 2)
    with pytest.raises(ValueError):  # not on a GPU
        fa.forward_paged_fp8(t, p, p, s, s, i, i[:1], i[None])
    with pytest.raises(ValueError):
        fa.cache_append_fp8(t, t, p, p, s, s, i, i[:1], i[None])
    with pytest.raises(ValueError):
        fa.rotary(t, t, torch.zeros(16), i)
    with pytest.raises(ValueError):
        fa.rotary(None, None, torch.zeros(16), i)


def test_frequencies(fa):
    f, m = fa.rotary_frequencies(64, 10000.0)
    want = [10000.0 ** (-2 * j / 64) for j in range(32)]
    assert m == 1.0 and f.dtype == torch.float32 and f.tolist() == torch.tensor(want, dtype=torch.float64).float().tolist()
    lin, m = fa.rotary_frequencies(64, scaling="linear", factor=4.0)
    assert m == 1.0 and torch.equal(lin, f / 4.0)
    # ntk: the fastest pair as it was, the slowest 1 / factor
    ntk, m = fa.rotary_frequencies(64, scaling="ntk", factor=8.0)
    assert m == 1.0 and ntk[0] == 1.0 and abs(float(ntk[-1] * 8.0 / f[-1]) - 1.0) < 1e-6
    # yarn: as they were from beta_fast turns on, 1 / factor up to beta_slow, falling between
    y, m = fa.rotary_frequencies(128, scaling="yarn", factor=16.0, original_length=4096)
    f = fa.rotary_frequencies(128)[0]
    turns = 4096 * f.double() / (2 * math.pi)
    r = (y / f).double()
    assert abs(m - (0.1 * math.log(16.0) + 1.0)) < 1e-12
    assert (r[turns > 40] == 1.0).all() and ((r[turns < 0.8] * 16 - 1.0).abs() < 1e-6).all()
    assert (r[1:] <= r[:-1] + 1e-6).all() and ((r > 1 / 16.001) & (r <= 1.0)).all()


@pytest.mark.parametrize("kw", [dict(dim=3), dict(dim=0), dict(dim=64, base=1.0), dict(dim=64, base=math.inf),
                                dict(dim=64, scaling="other"), dict(dim=64, scaling="linear", factor=0.5),
                                dict(dim=64, scaling="yarn", factor=2.0), dict(dim=64, factor=math.nan),
                                dict(dim=64, scaling="yarn", factor=2.0, original_length=0)])
def test_frequencies_refuse(fa, kw):
    with pytest.raises(ValueError):
        fa.rotary_frequencies(**kw)
