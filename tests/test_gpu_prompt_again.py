"""Rows that are done once more by the definition, key by key, behind the pass:
however many keys they see, no wait gives up over them, and what they are is
what the formulas give."""
import math

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _prompt_ref as R
from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_prompt import Case, near

pytestmark = pytest.mark.gpu

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
DEV = "cuda:0"


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_long_rows_beside_padding_that_is_not_finite(attn, D, bad):  # noqa: F811
    """100000 queries behind a prefix, 131067 keys of a slot of 131072; what
    lies in the last five slots meets the weights 0 of the queries of the last
    key step.  They alone are compared, with the definition."""
    nq, nk, slot, some = 100000, 131067, 131072, 160
    g = torch.Generator(device=DEV).manual_seed(D)

    def normal(*s):
        return torch.randn(s, generator=g, device=DEV).to(BF16)

    d = wl.AttnDims(B=1, T=nq, Hq=1, Hkv=1, D=D)
    q, k, v, dout = normal(1, nq, 1, D), normal(1, slot, 1, D), normal(1, slot, 1, D), normal(1, nq, 1, D)
    n_k = torch.tensor([nk], dtype=I32, device=DEV)
    k[:, nk:] = bad
    v[:, nk:] = bad
    out, lse = attn.attn_prefill(d, q, k, v, n_k=n_k, return_lse=True)
    got = attn.attn_prefill_backward(d, q, k, v, out, lse, dout, n_k=n_k)
    assert status() == 0
    assert all(torch.isfinite(x.float()).all() for x in (out, lse, *got.values()))
    # the last queries, each by itself: their outputs and dq
    tail = slice(nq - some, nq)
    rows = [x[0, tail] for x in (q, dout)]
    want, wlse, tol, ltol = R.prefill(rows[0], k[0, :nk], v[0, :nk], [(0, some, some)], [(0, nk, nk)], D ** -0.5)
    near(out[0, tail], want, tol, "out")
    near(lse[0, tail], wlse, ltol, "lse")
    w, t = R.prefill_backward(rows[0], k[0, :nk], v[0, :nk], rows[1], [(0, some, some)], [(0, nk, nk)], D ** -0.5)["dq"]
    near(got["dq"][0, tail], w, t, "dq")


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gated", [False, True])
def test_rows_of_whole_and_of_split_tiles(attn, D, gated):  # noqa: F811
    """An infinite value and an infinite gradient in one head: the other heads
    keep their bits, the head's own channels are what the formulas give."""
    c = Case(8, 4, D, [700, 300], [900, 300], True, gated, seed=D)
    out, lse = c.fwd(attn)
    k0, _, _ = c.ks[0]
    c.v[k0 + 70, 1, 9] = math.inf
    out2, lse2 = c.fwd(attn)
    assert torch.equal(lse, lse2)
    # key 70 is seen by every query of the first sequence (200 keys are before the first); key head 1: heads 2 and 3
    q0, _, nq = c.qs[0]
    seen = torch.zeros(c.rows, 8, D, dtype=torch.bool, device=DEV)
    seen[q0:q0 + nq, 2:4, 9] = True
    assert torch.equal(out2[:, [0, 1, 4, 5, 6, 7]], out[:, [0, 1, 4, 5, 6, 7]])
    assert (out2[seen] == math.inf).all()
    # the other channels of these rows are numbers, and the definition's
    assert torch.isfinite(out2.float()[~seen]).all()
    want, _, tol, _ = c.want_fwd()
    near(out2[~seen], want[~seen], tol[~seen], "out")
    c.v[k0 + 70, 1, 9] = 0.0
    c.dout[q0 + 5, 6, 3] = math.inf
    out3, lse3 = c.fwd(attn)
    again = c.bwd(attn, out3, lse3)
    base = Case(8, 4, D, [700, 300], [900, 300], True, gated, seed=D)
    base.v[k0 + 70, 1, 9] = 0.0
    grads = base.bwd(attn, out3, lse3)
    for n, heads in (("dq", [0, 1, 2, 3, 4, 5, 7]), ("dk", [0, 1, 2]), ("dv", [0, 1, 2])):
        assert torch.equal(again[n][:, heads], grads[n][:, heads]), n
    rest = torch.ones(c.rows, dtype=torch.bool, device=DEV)
    rest[q0 + 5] = False
    assert torch.equal(again["dq"][rest, 6], grads["dq"][rest, 6])
    assert not torch.isfinite(again["dq"][q0 + 5, 6].float()).any()
    # dv of the keys that the token sees: infinite in that channel, numbers in the others
    dv = again["dv"][k0:k0 + 200 + 6, 3].float()
    others = [i for i in range(D) if i != 3]
    assert torch.isfinite(dv[:, others]).all() and (dv[:, 3] == math.inf).sum() > 150
    assert status() == 0
