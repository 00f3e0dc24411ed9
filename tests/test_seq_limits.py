"""Limits of the calls on sequences of different lengths, checked on the host:
what the kernels' 32-bit counts cannot hold is refused."""
import pytest

from tests.test_seq_abi import call, fa  # noqa: F401 (fa: the fixture)

FA_ERR_UNSUPPORTED = 2


@pytest.mark.parametrize("heads,d", [(1 << 23, 128), ((1 << 24) - 1, 128), (1 << 24, 128), (1 << 25, 64), (1 << 25, 128)])
def test_append_refuses_tokens_of_2_30_values(fa, heads, d):
    big = dict(B=1, Hkv=heads, total_q=1, d=d, num_pages=1, max_pages=1, k_stride=heads * d, v_stride=heads * d)
    assert call(fa, "fa_cache_append", **big) == FA_ERR_UNSUPPORTED
