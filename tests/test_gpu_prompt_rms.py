"""A prompt's attention and its gradients on the GPU by their relative errors:
of tensors, heads and blocks of rows (tests/_prompt_rms.py derives the bounds)."""
import pytest

from tests import _prompt_rms as M
from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_prompt import Case

pytestmark = pytest.mark.gpu

# Hq, Hkv, D, queries, keys, packed, gated
CASES = [
    (16, 2, 256, [300], [300], False, True),
    (16, 2, 256, [1500, 77], [1500, 77], True, True),
    (4, 4, 128, [257], [1300], False, True),
    (32, 8, 128, [100, 700, 3, 0, 513], [100, 700, 3, 0, 513], True, False),
    (12, 1, 128, [100, 300, 3, 513], [103, 300, 4, 1213], True, True),
    (8, 8, 256, [900, 65], [900, 65], True, False),
    (8, 8, 64, [128, 129, 127], [128, 129, 127], True, True),
    (9, 3, 64, [77], [77], False, False),
    (13, 1, 256, [40, 600], [43, 600], True, True),
    (3, 1, 64, [2500], [3000], False, True),
    (1, 1, 128, [4000], [4000], False, False),
    (6, 2, 64, [300, 20], [290, 20], True, False),
]


@pytest.mark.parametrize("case", CASES)
def test_relative_errors(attn, case):  # noqa: F811
    Hq, Hkv, D, nq, nk, packed, gated = case
    c = Case(Hq, Hkv, D, nq, nk, packed, gated, seed=sum(nk))
    out, lse = c.fwd(attn)
    got = dict(c.bwd(attn, out, lse), out=out)
    want = {n: x for n, (x, _) in c.want_bwd().items()}
    want["out"] = c.want_fwd()[0]
    assert set(got) == set(want)
    for n in want:
        M.check(c.flat(got[n]), want[n], n)
    assert status() == 0
