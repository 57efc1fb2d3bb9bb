"""Probabilities outside [0, 1] count as their nearest value there, NaN as 0:
for whether a drafted token stands as for the token drawn after it."""
import math

import pytest
import torch

from tests import _prompt_ref as R
from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_spec import call, make, spec  # noqa: F401

pytestmark = pytest.mark.gpu

ODD = [-1.0, -0.0, -math.inf, math.nan, 2.0 ** -130, 0.25, 1.0, 1.5, 3.0, math.inf]
U = [0.0, 2.0 ** -24, 0.25, 0.5, 0.7, 1.0 - 2.0 ** -24]


def counts(x):
    return None if x is None else torch.nan_to_num(x, nan=0.0, posinf=1.0, neginf=0.0).clamp(0.0, 1.0)


def test_both_numbers_of_a_drafted_token(spec):  # noqa: F811
    """Every pair of odd values at the one drafted token, every u."""
    cases = [(p, q, u) for p in ODD for q in ODD for u in U]
    B, V = len(cases), 40
    target, draft = torch.full((B, 2, V), 1.0 / V), torch.full((B, 1, V), 0.5 / V)
    tokens = torch.tensor([[i % V] for i in range(B)], dtype=torch.int32)
    rows = torch.arange(B)
    target[rows, 0, tokens[:, 0].long()] = torch.tensor([c[0] for c in cases])
    draft[rows, 0, tokens[:, 0].long()] = torch.tensor([c[1] for c in cases])
    u = torch.tensor([[c[2], 0.375] for c in cases])
    for d in (draft, None):
        out, keep = call(spec, target, tokens, u, d)
        want, wkeep = R.verify(counts(target), tokens, u, counts(d))
        assert torch.equal(keep, wkeep) and torch.equal(out, want)
    # a token that the target does not have never stands: u q < 0 is false for every u and q
    for odd in (-1.0, math.nan, -math.inf, 0.0):
        target[rows, 0, tokens[:, 0].long()] = odd
        assert (call(spec, target, tokens, u, draft)[1] == 1).all()


@pytest.mark.parametrize("drafted", [True, False])
def test_odd_values_all_over_the_rows(spec, drafted):  # noqa: F811
    B, T, V = 60, 4, 500
    target, tokens, u, draft = make(B, T, V, 0.5, 17, drafted)
    g = torch.Generator().manual_seed(2)
    odd = torch.tensor([-1.0, -0.5, math.nan, -math.inf, 1.5, math.inf])
    for x in (target, draft):
        if x is None:
            continue
        flat = x.view(-1, V)
        # (at most 8 ones beside what the row has: sums below 16)
        at = torch.randint(0, V, (flat.shape[0], 8), generator=g)
        flat.scatter_(1, at, odd[torch.randint(0, 6, at.shape, generator=g)])
    # drafted tokens among them
    at = torch.rand(B, T, generator=g) < 0.5
    for x in (target[:, :T], draft):
        if x is not None:
            v = odd[torch.randint(0, 6, (B, T), generator=g)]
            old = x.gather(2, tokens.long()[..., None])[..., 0]
            x.scatter_(2, tokens.long()[..., None], torch.where(at, v, old)[..., None])
    out, keep = call(spec, target, tokens, u, draft)
    want, wkeep = R.verify(counts(target), tokens, u, counts(draft))
    assert torch.equal(keep, wkeep) and torch.equal(out, want)
