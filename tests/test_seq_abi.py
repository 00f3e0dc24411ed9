"""Host-only checks of the calls on sequences of different lengths: bad
arguments are refused before any device work."""
import pytest
import torch

P16 = 1 << 20  # any aligned non-null address: validation fails before it is touched


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    m.lib()
    return m


VARLEN = dict(q=P16, k=P16, v=P16, o=P16, lse=P16, cu_q=P16, cu_k=P16, B=2, Hq=4, Hkv=2, total_q=50, total_k=60, d=128,
              q_stride=512, k_stride=256, v_stride=256, scale=0.1, window_left=-1, window_right=0)
PAGED = dict(q=P16, k_pages=P16, v_pages=P16, o=P16, lse=P16, cu_q=P16, lens_k=P16, page_table=P16, B=2, Hq=4, Hkv=2,
             total_q=50, num_pages=9, page_size=16, max_pages=4, d=128, q_stride=512, scale=0.1, window_left=-1,
             window_right=0)
APPEND = dict(k=P16, v=P16, k_pages=P16, v_pages=P16, cu_q=P16, lens_k=P16, page_table=P16, B=2, Hkv=2, total_q=50,
              num_pages=9, page_size=16, max_pages=4, d=128, k_stride=256, v_stride=256)
BWD = dict(q=P16, k=P16, v=P16, o=P16, lse=P16, dout=P16, dq=P16, dk=P16, dv=P16)
BWD.update({n: VARLEN[n] for n in VARLEN if n not in BWD})
CALLS = {"fa_bwd_varlen": BWD, "fa_fwd_varlen": VARLEN, "fa_fwd_paged": PAGED, "fa_cache_append": APPEND}


def call(fa, name, **kw):
    a = dict(CALLS[name])
    assert set(kw) <= set(a)
    a.update(kw)
    return getattr(fa, name)(*a.values(), 0)


SHARED = [(dict(B=0), 1), (dict(Hkv=0), 1), (dict(d=96), 2), (dict(d=0), 1), (dict(total_q=-1), 1),
          (dict(total_q=1 << 29), 2)]
OF_PAGES = [(dict(num_pages=0), 1), (dict(page_size=0), 1), (dict(page_size=8), 2), (dict(page_size=20), 2),
            (dict(max_pages=0), 1), (dict(max_pages=1 << 26), 2)]
OF_Q = [(dict(Hq=3), 1), (dict(Hq=0), 1), (dict(Hq=258, q_stride=1 << 16), 2), (dict(scale=float("nan")), 1),
        (dict(scale=float("inf")), 1), (dict(q_stride=511), 1), (dict(q_stride=504), 1), (dict(q_stride=1 << 39), 2)]
OF_KV = [(dict(k_stride=248), 1), (dict(v_stride=257), 1), (dict(v_stride=1 << 39), 2)]
BAD = ([(f, b, c) for f in ("fa_fwd_varlen", "fa_bwd_varlen") for b, c in SHARED + OF_Q + OF_KV + [(dict(total_k=-1), 1), (dict(total_k=1 << 29), 2)]]
       + [("fa_fwd_paged", b, c) for b, c in SHARED + OF_Q + OF_PAGES]
       + [("fa_cache_append", b, c) for b, c in SHARED + OF_KV + OF_PAGES])


@pytest.mark.parametrize("name,bad,code", BAD)
def test_bad_sizes(fa, name, bad, code):
    assert call(fa, name, **bad) == code


@pytest.mark.parametrize("name,total,stride", [("fa_fwd_varlen", "total_q", "q_stride"), ("fa_fwd_varlen", "total_k", "v_stride"),
                                               ("fa_bwd_varlen", "total_k", "k_stride"), ("fa_fwd_paged", "total_q", "q_stride"),
                                               ("fa_cache_append", "total_q", "k_stride")])
def test_bytes_that_pass_64_bits(fa, name, total, stride):
    assert call(fa, name, **{total: 1 << 26, stride: 1 << 37}) == 2  # 2^64 bytes


@pytest.mark.parametrize("name", list(CALLS))
def test_bad_pointers(fa, name):
    for arg, v in CALLS[name].items():
        if v == P16:
            assert call(fa, name, **{arg: 0}) == 1, arg
            assert call(fa, name, **{arg: P16 + 2}) == 1, arg
            if arg not in ("cu_q", "cu_k", "lens_k", "page_table"):
                assert call(fa, name, **{arg: P16 + 8}) == 1, arg


@pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
@pytest.mark.parametrize("name", list(CALLS))
def test_good_arguments_reach_the_device_check(fa, name):
    assert call(fa, name) == 6
    # nothing to do, and null pointers for it: still needs a device
    assert call(fa, name, total_q=0, **{a: 0 for a in ("q", "o", "lse", "dout", "dq") if a in CALLS[name]}) == 6
    if name == "fa_fwd_varlen":
        assert call(fa, name, total_k=0, k=0, v=0) == 6
    if name == "fa_bwd_varlen":
        assert call(fa, name, total_k=0, k=0, v=0, dk=0, dv=0) == 6
    if "window_left" in CALLS[name]:
        assert call(fa, name, window_left=2**31 - 1, window_right=-2**31) == 6


def test_python_checks(fa):
    t = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        fa.forward_varlen(t, t, t, i, i)
    with pytest.raises(ValueError):
        fa.forward_paged(t, t[None], t[None], i, i[:1], i[None])
    with pytest.raises(ValueError):
        fa.cache_append(t, t, t[None], t[None], i, i[:1], i[None])
