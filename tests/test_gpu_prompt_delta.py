"""The gradients of queries that see few keys, row by row.

dS_j = P_j sum_d dO_d (v_jd - o_d): with delta summed from P and dP themselves
every error of dO enters as dO_d e_d (v_jd - o_d), which is 0 for a query of one
key and small where one key has most of the weight.  From the rounded output it
would enter as dO_d o_d e_d, whatever the keys: for such rows many times dq.

A row's error is bounded by its norm.  Roundings to bf16 are off by e with |e|
<= 2^-8 of the value, of variance 2^-16 / 3 at most, independent of each other:
dO's (with a gate; one for all keys of the row), dS's (one a key), dq's own.
The expected square of the error's norm is their sum of squares; a single
rounding may govern a row, so six times its root is allowed.

The f32 arithmetic is added: sums of D products by 16 at a time, each of the
D / 16 additions off by 2^-23 of what has been summed so far, at most four times
the root of the products' squares or the sum itself, in the forward pass's
scores (in lse), in the backward pass's, and in dP; 2^-20 for the exponential
and its argument.
"""
import math

import pytest
import torch

from tests import _prompt_ref as R
from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_prompt import Case

pytestmark = pytest.mark.gpu

F64 = torch.float64
VAR = R.BF ** 2 / 3


def rows_of_few_keys(c, got, most):
    """Largest error of a dq row of at most `most` keys, in units of its bound."""
    flat = c.flat
    gate = c.kw.get("gate")
    G = c.q.shape[-2] // c.k.shape[-2]
    worst, checked = 0.0, 0
    for (q0, _, nq), (k0, _, nk) in zip(c.qs, c.ks):
        n = min(nq, max(0, most - (nk - nq)))
        first = max(0, nq - nk)                          # (before: no key)
        if n <= first:
            continue
        cols = nk - nq + n
        vis = R.seen(nq, nk, c.q.device)[first:n, :cols]
        for h in range(c.q.shape[-2]):
            q, do = (flat(x)[q0 + first:q0 + n, h].to(F64) for x in (c.q, c.dout))
            k, v = (flat(x)[k0:k0 + cols, h // G].to(F64) for x in (c.k, c.v))
            if gate is not None:
                do = do * torch.sigmoid(flat(gate)[q0 + first:q0 + n, h].to(F64))
            s = c.scale * q @ k.T
            z = s.masked_fill(~vis, -math.inf)
            lse = torch.logsumexp(z, -1, keepdim=True)
            p = torch.exp(z - lse)
            dp = do @ v.T
            ds = p * (dp - (p * dp).sum(-1, keepdim=True))
            dq = c.scale * ds @ k
            # E |error|^2 / scale^2
            var = VAR * (ds.square() @ k.square().sum(-1, keepdim=True))[:, 0]
            if gate is not None:
                # for each channel d of dO: | sum_j P_j (v_jd - o_d) k_j |^2
                pk = p @ k                               # sum_j P_j k_j
                pv = p @ v
                each = torch.einsum("tj,jd,je->tde", p, v, k) - pv[:, :, None] * pk[:, None, :]
                var += VAR * (do.square() * each.square().sum(-1)).sum(-1)
            var = c.scale ** 2 * var + VAR * dq.square().sum(-1)
            def summed(a, b, x):
                return q.shape[-1] / 16 * 2.0 ** -23 * (4 * (a.square() @ b.square().T).sqrt() + x.abs())

            e_s = 2 * abs(c.scale) * summed(q, k, q @ k.T) * vis + 2.0 ** -20 * (1 + lse.abs())
            e_ds = p * (2 * e_s * (dp.abs() + (p * dp.abs()).sum(-1, keepdim=True)) + summed(do, v, dp) + 2.0 ** -22 * dp.abs())
            e_ds = e_ds + p * (p * (e_s * dp.abs() + summed(do, v, dp))).sum(-1, keepdim=True) + R.TINY * (dp.abs() + 2) * vis
            f32 = (abs(c.scale) * e_ds @ k.abs()).norm(dim=-1) + R.TINY * k.shape[-1]
            err = (flat(got["dq"])[q0 + first:q0 + n, h].to(F64) - dq).norm(dim=-1)
            worst = max(worst, float((err / (6 * var.sqrt() + f32)).max()))
            checked += n - first
    assert checked > 0
    return worst


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("std", [1.0, 2.5])
@pytest.mark.parametrize("heads", [(4, 4), (3, 1), (16, 2)])
def test_rows_of_few_keys(attn, D, gated, std, heads):  # noqa: F811
    """Prompts of 64, 65 and more tokens, behind prefixes and longer than their
    keys: a row's gradient does not depend on what comes after it."""
    c = Case(*heads, D, [64, 65, 129, 700, 40], [64, 65, 129, 720, 30], True, gated, seed=7, std=std)
    out, lse = c.fwd(attn)
    got = c.bwd(attn, out, lse)
    assert rows_of_few_keys(c, got, 64) <= 1.0


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gated", [False, True])
def test_a_query_of_one_key_has_no_gradient(attn, D, gated):  # noqa: F811
    """P is 1: dq is 0 but for the f32 arithmetic, in prompts of any length.
    (Small queries and keys: their scores' errors in the worst case, not only as
    they come, are far below a rounding to bf16.)"""
    for n in (1, 64, 65, 128, 1000):
        c = Case(4, 4, D, [n], [n], False, gated, seed=n, std=0.1)
        out, lse = c.fwd(attn)
        got = c.bwd(attn, out, lse)
        q, do, v, k = (x[0, 0].double() for x in (c.q, c.dout, c.v, c.k))
        s = c.scale * (q * k).sum(-1)
        e_p = 2 * R.F32 * ((D + 4) * c.scale * (q.abs() * k.abs()).sum(-1) + 4 * s.abs()) + 2.0 ** -20 * (2 + s.abs())
        size = c.scale * (do.abs() * v.abs()).sum(-1) * (e_p + 2.0 ** -22)
        assert (got["dq"][0, 0].double().abs() <= size[:, None] * k.abs() * (1 + R.BF)).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("gated", [False, True])
def test_a_prompt_cut_short_has_the_same_first_rows(attn, D, gated):  # noqa: F811
    """64 tokens alone and the same 64 with more behind them: two kinds of tiles,
    one definition."""
    c = Case(4, 4, D, [200], [200], False, gated, seed=11, std=2.0)
    out, lse = c.fwd(attn)
    got = c.bwd(attn, out, lse)["dq"][:, :64]
    c.d = c.d.with_(T=64)
    for n in ("q", "k", "v", "dout"):
        setattr(c, n, getattr(c, n)[:, :64].contiguous())
    if gated:
        c.kw["gate"] = c.kw["gate"][:, :64].contiguous()
    c.kw.update(n_q=None, n_k=None)
    c.qs = c.ks = [(0, 64, 64)]
    alone = c.bwd(attn, out[:, :64].contiguous(), lse[:, :64].contiguous())["dq"]
    assert torch.equal(got, alone)
