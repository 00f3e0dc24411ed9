"""A process's first call of the library may be one that is captured into a
graph: what the library sets up on its first call does not end the capture."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import sys
import torch
import exact_attention_99_gb300 as fa

g = torch.Generator(device="cuda").manual_seed(1)
n = [300, 40, 900]
T = sum(n)
normal = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)
q, k, v = normal(T, 8, 64), normal(T, 2, 64), normal(T, 2, 64)
o, lse, grads = torch.zeros_like(q), torch.zeros(8, T, device="cuda"), [torch.zeros_like(x) for x in (q, k, v)]
kp, vp = normal(700, 16, 2, 64), normal(700, 16, 2, 64)
i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
cu, lens, table = i32([0, 300, 340, 1240]), i32([3000, 40, 2500]), torch.randperm(700, device="cuda", generator=g)[:600].view(3, 200).to(torch.int32)


def step(which):
    if which == "dense":
        x, y = q[:1024].view(1, 1024, 8, 64), k[:1024].view(1, 1024, 2, 64)
        a, b = fa.forward(x, y, y, causal=True)
        return [a, b, *fa.backward(x, y, y, a, b, x, causal=True)[1:]]
    if which == "forward":
        return fa.forward_varlen(q, k, v, cu, cu, causal=True)
    if which == "backward":
        return fa.backward_varlen(q, k, v, o, lse, q, cu, cu, causal=True, out=grads)[1:]
    fa.cache_append(k, v, kp, vp, cu, lens, table)
    return [kp, vp, *fa.forward_paged(q, kp, vp, cu, lens, table)]


torch.cuda.synchronize()
graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
with torch.cuda.stream(s):
    with torch.cuda.graph(graph, stream=s):
        got = step(sys.argv[1])
graph.replay()
torch.cuda.synchronize()
got = [x.clone() for x in got]
want = step(sys.argv[1])
assert all(torch.equal(a, b) for a, b in zip(got, want)) and fa.fa_get_status() == 0
print("same")
"""


@pytest.mark.parametrize("which", ["dense", "forward", "backward", "paged"])
def test_the_first_call_is_captured(which):
    import __graft_entry__
    __graft_entry__.build()
    r = subprocess.run([sys.executable, "-c", CHILD, which], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "same", r.stderr[-2000:]
