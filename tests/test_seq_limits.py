"""Limits of the calls on sequences of different lengths, checked on the host:
what the kernels' 32-bit counts cannot hold is refused."""
import pytest
import torch

from tests.test_seq_abi import call, fa  # noqa: F401 (fa: the fixture)

FA_ERR_UNSUPPORTED, FA_ERR_NO_DEVICE = 2, 6


@pytest.mark.parametrize("heads,d", [(1 << 23, 128), ((1 << 24) - 1, 128), (1 << 24, 128), (1 << 25, 64), (1 << 25, 128)])
def test_append_refuses_tokens_of_2_30_values(fa, heads, d):
    big = dict(B=1, Hkv=heads, total_q=1, d=d, num_pages=1, max_pages=1, k_stride=heads * d, v_stride=heads * d)
    assert call(fa, "fa_cache_append", **big) == FA_ERR_UNSUPPORTED


def test_backward_refuses_more_padded_rows_than_its_counts_hold(fa):
    # 2^21 sequences of 4 tokens, 16 kv heads: a tile of 128 rows to each
    assert call(fa, "fa_bwd_varlen", B=1 << 21, Hq=16, Hkv=16, total_q=1 << 23, total_k=1 << 23, d=64, q_stride=1024,
                k_stride=1024, v_stride=1024) == FA_ERR_UNSUPPORTED


@pytest.mark.skipif(torch.cuda.is_available(), reason="stops at the device check")
def test_backward_takes_many_empty_sequences(fa):
    # no more tiles than tokens, however many sequences there are
    assert call(fa, "fa_bwd_varlen", B=1 << 25, Hq=2, Hkv=1, total_q=10, total_k=10) == FA_ERR_NO_DEVICE


@pytest.mark.parametrize("window,causal,want", [((5, 7), False, (5, 7)), ((-1, -9), False, (-1, -1)), (None, True, (-1, 0)),
                                                ((4, 7), True, (4, 0)), ((4, -1), True, (4, 0)),
                                                ((2 ** 31, 2 ** 31 - 1), False, (2 ** 31 - 1, 2 ** 31 - 1)),
                                                ((2 ** 32 + 5, 2 ** 63 - 1), False, (2 ** 31 - 1, 2 ** 31 - 1)),
                                                ((-2 ** 32 + 5, -2 ** 63), False, (-1, -1))])
def test_window_bounds_past_32_bits(fa, window, causal, want):
    # (ctypes would take their low 32 bits)
    assert fa._window_args(causal, window) == want


@pytest.mark.parametrize("heads", [1 << 24, 1 << 25, 1 << 28])
def test_backward_refuses_rows_of_many_heads(fa, heads):
    # one token: a tile of 128 rows to each kv head
    assert call(fa, "fa_bwd_varlen", B=1, Hq=heads, Hkv=heads, total_q=1, total_k=1, d=64, q_stride=64 * heads,
                k_stride=64 * heads, v_stride=64 * heads) == FA_ERR_UNSUPPORTED
