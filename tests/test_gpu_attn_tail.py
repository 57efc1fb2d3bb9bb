"""attn_decode where one key outweighs each of many others, which only
together carry part of the output."""
import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _attn_ref as R
from tests.test_gpu_attn import DEV, E4M3, F64, I32, attn, gen, status, value64  # noqa: F401

pytestmark = pytest.mark.gpu


CASES = [(12.0, 0), (17.5, 0), (17.5, 30000), (18.5, 0), (18.5, 77777)]


def one_before_many(attn, nats, place, rows, fp8):  # noqa: F811
    """80000 keys of score 0 and one of `nats`: all rows read the same pages.
    One row for each SM (rows = 0) leaves each of them to one CTA, a single row
    is split over all.  The dominant key's value is zero in all channels but
    one, so that the others' sums stand alone there.  Returns the errors of
    output and log-sum-exp and the reference's bounds."""
    n, P, D = 80001, 64, 64
    B = rows or torch.cuda.get_device_properties(0).multi_processor_count
    d = wl.AttnDims(B, 1, 2, 1, D)
    g = gen(int(nats * 2) + place)
    width = -(-n // P)
    cache = attn.KVCache.empty(d, width, P, E4M3 if fp8 else torch.bfloat16, DEV)
    v = torch.rand(cache.v.shape, generator=g) + 0.5
    v[place // P, 0, place % P] = 0.0
    v[place // P, 0, place % P, 5] = 448.0
    cache.v.copy_(v.to(cache.v.dtype))
    k = torch.zeros(cache.k.shape)
    k[place // P, 0, place % P, 0] = 1.0
    cache.k.copy_(k.to(cache.k.dtype))
    if fp8:
        for s in (cache.k_scale, cache.v_scale):
            s.view(torch.uint8).fill_(127)
    table = torch.arange(width, dtype=I32)[None]
    q = torch.zeros((1, 1, 2, D))
    q[..., 0] = nats * 8                                    # exact in bf16; the score is nats
    q = q.to(torch.bfloat16)
    out, lse = attn.attn_decode(d, q.expand(B, 1, 2, D).contiguous().to(DEV), cache, table.expand(B, -1).contiguous().to(DEV),
                                torch.full((B,), n - 1, dtype=I32, device=DEV), return_lse=True)
    want, want_lse, tol, lse_tol = R.decode(q, value64(cache.k, cache.k_scale), value64(cache.v, cache.v_scale), table,
                                            P, [n - 1], None, 0.125)
    assert status() == 0
    return (out.cpu().to(F64) - want).abs(), tol, (lse.cpu().to(F64) - want_lse).abs(), lse_tol


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 0])
@pytest.mark.parametrize("nats,place", CASES)
def test_sum_of_one_key_before_many(attn, nats, place, rows, fp8):  # noqa: F811
    """The log-sum-exp: small terms on top of a large one do not drift."""
    _, _, err, tol = one_before_many(attn, nats, place, rows, fp8)
    assert torch.all(err <= tol), (float(err.max()), float(tol.max()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rows", [1, 0])
@pytest.mark.parametrize("nats,place", CASES)
def test_output_of_one_key_before_many(attn, nats, place, rows, fp8):  # noqa: F811
    """Each weight's rounding and the output's are at most half a step of bf16."""
    err, tol, _, _ = one_before_many(attn, nats, place, rows, fp8)
    assert torch.all(err <= tol), "off by %.3e more than %.3e" % (float((err - tol).max()), float(tol[..., 6].max()))
