"""Rows of drafted tokens that are spread over a cluster of CTAs with next to
nothing to read in some of them: a CTA's sums go to CTAs that may have only
just started."""
import pytest
import torch

from tests import _prompt_ref as R
from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_spec import DEV, call, make, spec  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [0, 2])
@pytest.mark.parametrize("V", [4097, 8192, 8193, 28673, 32769])
@pytest.mark.parametrize("B", [1, 3, 37])
def test_empty_pieces(spec, B, V, T):  # noqa: F811
    """16 warps a CTA, pieces of whole batches of 256: 4097 tokens leave 15 of
    32 warps without any."""
    target, tokens, u, draft = make(B, T, V, 1.0, B + T + V)
    out, keep = call(spec, target, tokens, u, draft if T else None)
    want, wkeep = R.verify(target[:2], tokens[:2], u[:2], draft[:2] if T else None)
    assert torch.equal(out[:2], want) and torch.equal(keep[:2], wkeep)
    dev = [x.to(DEV) for x in (target, tokens, u)] + [draft.to(DEV) if T else None]
    again = [spec.verify(dev[0], dev[1], dev[2], draft=dev[3]) for _ in range(200)]
    for o, k in again:
        assert torch.equal(o.cpu(), out) and torch.equal(k.cpu(), keep)
