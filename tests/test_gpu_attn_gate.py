"""The gate of attn_decode at tokens that are not there."""
import math

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests.test_gpu_attn import DEV, I32, attn, check_decode, gen, make_cache, normal, tables  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,pos,n_new", [
    (1, 8, 2, 64, [40, 7, 0], [1, 0, 1]),
    (3, 16, 2, 256, [100, 3, 30], [2, 0, 3]),
    (2, 8, 1, 128, [50000, 20, 40000], [1, 2, 0]),            # the first row split over the length
    (8, 16, 1, 64, [900, 33, 2], [3, 8, 0]),
])
def test_gates_of_absent_tokens(attn, T, Hq, Hkv, D, pos, n_new, fp8, bad):  # noqa: F811
    """Whatever the gate holds at a token past n_new, the token gives zeros."""
    B, P = 3, 16
    d = wl.AttnDims(B, T, Hq, Hkv, D)
    g = gen(T + D)
    width = -(-(max(pos) + T) // P)
    cache = make_cache(attn, d, B * width + 1, P, fp8, g)
    table = tables(g, B, width, B * width + 1)
    q, gate = normal(g, B, T, Hq, D), normal(g, B, T, Hq, D)
    absent = torch.arange(T) >= torch.tensor(n_new)[:, None]
    spoilt = torch.where(absent[..., None, None], torch.full_like(gate, bad), gate)
    out, lse = attn.attn_decode(d, q.to(DEV), cache, table.to(DEV), torch.tensor(pos, dtype=I32, device=DEV),
                                torch.tensor(n_new, dtype=I32, device=DEV), spoilt.to(DEV), return_lse=True)
    assert torch.all(out.cpu()[absent] == 0) and torch.all(lse.cpu()[absent] == -math.inf)
    check_decode(out, lse, q, cache, table, pos, n_new, D ** -0.5, gate)
