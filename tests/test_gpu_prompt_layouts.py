"""Calls that the other tests of the prompt operators do not make: heads in
front of tokens, heads that overlap, a process whose first calls are captured."""
import os
import subprocess
import sys

import pytest
import torch

from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_prompt import Case

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def results(a, c):
    out, lse = c.fwd(a)
    return dict(c.bwd(a, out, lse), out=out, lse=lse)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("packed", [False, True])
def test_heads_in_front_of_tokens(attn, D, packed):  # noqa: F811
    """[heads, tokens, channels] in memory, handed over as [tokens, heads,
    channels]: a token's stride is shorter than a head's."""
    nq, nk = ([300, 41], [310, 41]) if packed else ([333], [333])
    c = Case(6, 2, D, nq, nk, packed, True, seed=D)
    want = results(attn, c)

    def turned(x):
        y = x.transpose(-3, -2).contiguous().transpose(-3, -2)
        assert y.stride(-3) == D and y.stride(-2) > D
        return y
    c.q, c.k, c.v = (turned(x) for x in (c.q, c.k, c.v))
    c.kw["gate"] = turned(c.kw["gate"])
    got = results(attn, c)
    for n in want:
        assert torch.equal(got[n], want[n]), n
    assert status() == 0


@pytest.mark.parametrize("D", [64, 256])
def test_heads_that_overlap(attn, D):  # noqa: F811
    """Key heads that share memory, eight channels apart."""
    c = Case(4, 2, D, [200], [260], False, False, seed=5)
    n = c.k.shape[1]
    base = torch.randn(1, n, D + 8, device="cuda:0").to(torch.bfloat16)
    c.k = base.as_strided((1, n, 2, D), (n * (D + 8), D + 8, 8, 1))
    got = results(attn, c)
    c.k = c.k.contiguous()
    want = results(attn, c)
    for name in want:
        assert torch.equal(got[name], want[name]), name


FIRST = """
import torch
from gated_deltanet_linear_04_gb300 import attn, gdn, spec, workloads as wl
dev, bf = "cuda", torch.bfloat16
d = wl.AttnDims(B=2, T=200, Hq=8, Hkv=2, D=%d, Drot=32)
g = torch.Generator(device=dev).manual_seed(1)
r = lambda *s: torch.randn(s, generator=g, device=dev).to(bf)
q, k, v, gate, dout = r(2, 200, 8, d.D), r(2, 200, 2, d.D), r(2, 200, 2, d.D), r(2, 200, 8, d.D), r(2, 200, 8, d.D)
w = torch.ones(d.D, device=dev)
fr = attn.rope_freqs(attn.rope_inv_freq(32), dev)
axes = attn.rope_axes([6, 5, 5], device=dev)
pos = torch.arange(200, device=dev, dtype=torch.int32).expand(3, 2, 200).contiguous()
t, u, tok = torch.softmax(torch.randn(2, 4, 999, device=dev), -1), torch.rand(2, 4, device=dev), torch.zeros(2, 3, dtype=torch.int32, device=dev)
def step():
    a, b = attn.qk_norm_rope_axes(d, q, k, w, w, fr, axes, pos)
    out, lse = attn.attn_prefill(d, a, b, v, gate=gate, return_lse=True)
    x = attn.attn_prefill_backward(d, a, b, v, out, lse, dout, gate=gate)
    y = attn.qk_norm_rope_axes_backward(d, q, k, w, w, fr, axes, pos, x["dq"], x["dk"])
    return [a, b, out, lse, *x.values(), *y.values(), *spec.verify(t, tok, u)]
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
for x, y in zip(got, step()):
    assert torch.equal(x, y)
assert gdn.gdn_device_status() == 0
print("equal")
"""


@pytest.mark.parametrize("D", [64, 128, 256])
def test_the_first_calls_of_a_process_can_be_captured(attn, D):  # noqa: F811
    """Nothing is set up by a first call that a capture does not allow."""
    r = subprocess.run([sys.executable, "-c", FIRST % D], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "equal" in r.stdout, r.stderr[-2000:]
