"""The verification of drafted tokens at the ends of its ranges."""
import pytest
import torch

from tests import _prompt_ref as R
from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_spec import DEV, call, make, spec  # noqa: F401

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.mark.parametrize("T", [31, 32, 33, 64, 1023])
def test_many_drafts(spec, T):  # noqa: F811
    """All stand, all but one, or some: runs that end at, before and behind 32."""
    B, V = 40, 24
    g = torch.Generator().manual_seed(T)
    target = torch.softmax(torch.randn(B, T + 1, V, generator=g), -1)
    tokens = torch.randint(0, V, (B, T), generator=g).to(I32)
    u = torch.zeros(B, T + 1)
    u[:, T] = torch.rand(B, generator=g)
    for b in range(B):
        if b % 4 != 0:
            u[b, min(T - 1, [0, T - 1, 32, 31, 63, T // 2][b % 6])] = 1.0 - 2.0 ** -24     # (falls: p < 1)
    n = torch.tensor([T if b % 5 else max(0, T - 1) for b in range(B)], dtype=I32)
    for draft in (None, torch.softmax(torch.randn(B, T, V, generator=g), -1)):
        out, keep = call(spec, target, tokens, u, draft, n)
        want, wkeep = R.verify(target, tokens, u, draft, n)
        assert torch.equal(keep, wkeep) and torch.equal(out, want)


@pytest.mark.parametrize("V", [(1 << 24) - 1, 1 << 24, 5000001])
@pytest.mark.parametrize("B", [1, 3])
def test_the_largest_vocabularies(spec, V, B):  # noqa: F811
    """Against whole numbers of 2^-60: probabilities that are multiples of 2^-37,
    of a sum below 8."""
    g = torch.Generator(device=DEV).manual_seed(V % 1000 + B)
    units = torch.randint(0, 1 << 13, (B, 1, V), generator=g, device=DEV)       # of 2^-37
    target = units.to(torch.float32) * 2.0 ** -37
    for top in (0.0, 2.0 ** -30, 0.25, 0.7, 1.0 - 2.0 ** -24):
        u = torch.full((B, 1), top, device=DEV)
        out, keep = spec.verify(target, torch.zeros(B, 0, dtype=I32, device=DEV), u)
        assert (keep == 1).all()
        for b in range(B):
            sums = units[b, 0].cumsum(0)                                           # (below 2^37)
            total = int(sums[-1])
            num, den = float(top).as_integer_ratio()
            # the first sum above u total
            want = int(torch.searchsorted(sums, torch.tensor([num * total // den], device=DEV), right=True))
            assert int(out[b, 0]) == want
