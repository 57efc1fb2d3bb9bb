"""The relative errors that the GPU results are held to, on the CPU: results
with the kernels' roundings pass, results with a planted mistake do not."""
from types import SimpleNamespace

import pytest
import torch

from tests import _prompt_ref as R
from tests import _prompt_rms as M
from tests.test_gpu_prompt_delta import rows_of_few_keys

BF16, F64 = torch.bfloat16, torch.float64

# Hq, Hkv, D, queries, keys, gated
CASES = [
    (4, 2, 256, [300], [300], True),
    (4, 4, 128, [257], [1300], True),
    (4, 1, 64, [700, 100, 3, 90], [700, 100, 3, 90], False),
    (4, 4, 64, [400, 60], [500, 60], True),
    (6, 2, 64, [300, 20], [290, 20], False),           # queries before the first key
]


@pytest.fixture(scope="module", params=CASES, ids=str)
def case(request):
    Hq, Hkv, D, nq, nk, gated = request.param
    g = torch.Generator().manual_seed(Hq + sum(nk))

    def normal(rows, H, s):
        return (torch.randn(rows, H, D, generator=g) * s).to(BF16)

    q, k, v, dout = normal(sum(nq), Hq, 1.5), normal(sum(nk), Hkv, 1.0), normal(sum(nk), Hkv, 1.0), normal(sum(nq), Hq, 0.3)
    gate = normal(sum(nq), Hq, 1.5) if gated else None
    at = [torch.tensor([0] + n).cumsum(0) for n in (nq, nk)]
    qs, ks = (R.sequences(len(n), sum(n), a, None) for n, a in zip((nq, nk), at))
    args = (q, k, v, dout, qs, ks, D ** -0.5, gate)
    want = {n: x for n, (x, _) in R.prefill_backward(*args).items()}
    want["out"] = R.prefill(q, k, v, qs, ks, D ** -0.5, gate)[0]
    return args, want, M.restated(*args)


def rejected(got, want, name):
    with pytest.raises(AssertionError):
        M.check(got, want, name)


def test_the_kernels_roundings_pass(case):
    args, want, got = case
    assert set(got) == set(want)
    for n in want:
        M.check(got[n], want[n], n)


def test_a_factor_and_noise_are_rejected(case):
    args, want, got = case
    g = torch.Generator().manual_seed(1)
    for n in want:
        rejected(got[n] * 1.02, want[n], n)
        rejected(got[n] * 0.98, want[n], n)
        rms = want[n].square().mean().sqrt()
        rejected(got[n] + 0.01 * rms * torch.randn(got[n].shape, generator=g, dtype=F64), want[n], n)
        rejected(torch.zeros_like(got[n]), want[n], n)
        one = got[n].clone()
        one[:, -1] *= 1.02                              # one head only
        rejected(one, want[n], n)
        some = got[n].clone()
        some[64:128, 0] *= 1.02                         # one block of one head only
        rejected(some, want[n], n)


@pytest.mark.parametrize("token", [150, 255])
def test_a_query_that_is_left_out_is_rejected(case, token):
    args, want, _ = case
    got = M.restated(*args, drop_token=(0, 1, token))
    for n in ("dk", "dv"):
        rejected(got[n], want[n], n)


@pytest.mark.parametrize("first", [0, 64, 192])
def test_a_step_that_is_left_out_is_rejected(case, first):
    args, want, _ = case
    rejected(M.restated(*args, drop_step=(0, 1, first))["dq"], want["dq"], "dq")


def test_delta_from_the_output_is_rejected_for_rows_of_few_keys(case):
    """By their own bound, row by row (all rows' relative error hardly shows it)."""
    args, want, got = case
    q, k, v, dout, qs, ks, scale, gate = args
    c = SimpleNamespace(flat=lambda x: x, kw={} if gate is None else {"gate": gate}, q=q, k=k, v=v, dout=dout, qs=qs, ks=ks, scale=scale)
    if qs[0][2] <= ks[0][2] - 64:
        pytest.skip("no query of at most 64 keys")
    assert rows_of_few_keys(c, got, 64) <= 1.0
    assert rows_of_few_keys(c, M.restated(*args, delta_of_few=False), 64) > 1.0
