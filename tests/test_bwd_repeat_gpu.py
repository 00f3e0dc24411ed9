"""The backward calls again and again on the same inputs: dK and dV are sums in
a fixed order, so every call has to give the first one's bits (two warps that
are not ordered where they share tensor memory would show here)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def fa():
    import __graft_entry__
    __graft_entry__.build()
    import exact_attention_99_gb300 as m
    m.fa_debug_set(0, 0)
    return m


def normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)


@pytest.mark.parametrize("B,Hq,Hkv,N,d,causal", [(2, 8, 8, 2048, 128, True), (1, 16, 4, 4096, 128, False),
                                                 (2, 8, 8, 2048, 64, True), (4, 6, 2, 1000, 64, False)])
def test_dense(fa, B, Hq, Hkv, N, d, causal):
    g = torch.Generator(device="cuda").manual_seed(N + d)
    q, do = normal(g, B, N, Hq, d), normal(g, B, N, Hq, d)
    k, v = normal(g, B, N, Hkv, d), normal(g, B, N, Hkv, d)
    o, lse = fa.forward(q, k, v, causal=causal)
    first = fa.backward(q, k, v, o, lse, do, causal=causal)
    for _ in range(30):
        again = fa.backward(q, k, v, o, lse, do, causal=causal)
        assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])
    assert fa.fa_get_status() == 0


@pytest.mark.parametrize("lens,Hq,Hkv,d,causal", [([2000, 900, 3000, 40, 1500], 16, 8, 128, True), ([4096], 4, 1, 128, False),
                                                  ([2000, 900, 3000, 40, 1500], 16, 8, 64, True), ([700, 650], 6, 2, 64, False)])
def test_packed(fa, lens, Hq, Hkv, d, causal):
    g = torch.Generator(device="cuda").manual_seed(sum(lens) + d)
    n = sum(lens)
    q, do, k, v = normal(g, n, Hq, d), normal(g, n, Hq, d), normal(g, n, Hkv, d), normal(g, n, Hkv, d)
    cu = torch.tensor([0] + lens, device="cuda").cumsum(0).to(torch.int32)
    o, lse = fa.forward_varlen(q, k, v, cu, cu, causal=causal)
    first = fa.backward_varlen(q, k, v, o, lse, do, cu, cu, causal=causal)
    for _ in range(30):
        again = fa.backward_varlen(q, k, v, o, lse, do, cu, cu, causal=causal)
        assert torch.equal(again[1], first[1]) and torch.equal(again[2], first[2])
    assert fa.fa_get_status() == 0
