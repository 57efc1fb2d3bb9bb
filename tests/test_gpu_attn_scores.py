"""attn_decode at scores so large that one key decides: the output is its value."""
import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests.test_gpu_attn import BF16, DEV, F64, I32, attn, gen, make_cache, normal, status, tables, value64  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("pos", [0, 500, 30000])
@pytest.mark.parametrize("top", [1e3, 1e5, 1e6, 1e7, 1e9])
def test_the_largest_score_decides(attn, top, pos, fp8):  # noqa: F811
    """Two rows, the first one split over the length when it is long: one key's
    score is about `top`, the others' are 0 and weigh e^-1000 or less.  The
    weight is 1 and the output the key's value, with any scale: 2^-20 for the
    f32 steps and half a step of bf16."""
    B, P, D = 2, 16, 64
    d = wl.AttnDims(B, 1, 4, 2, D)
    g = gen(pos + int(top))
    width = pos // P + 1
    cache = make_cache(attn, d, B * width, P, fp8, g)
    table = tables(g, B, width, B * width)
    cache.k.view(torch.uint8).zero_()
    if fp8:
        cache.v_scale.view(torch.uint8).copy_(torch.randint(80, 175, cache.v_scale.shape, generator=g).to(torch.uint8))
        cache.k_scale.view(torch.uint8).fill_(127)
    at = [pos // 3, pos // 2]
    for b in range(B):
        cache.k.view(torch.uint8 if fp8 else torch.int16)[table[b, at[b] // P], :, at[b] % P, 3] = 0x38 if fp8 else 0x3f80
    q = normal(g, B, 1, 4, D)
    q[..., 3] = top * 8
    out = attn.attn_decode(d, q.to(DEV), cache, table.to(DEV), torch.full((B,), pos, dtype=I32, device=DEV))
    v = value64(cache.v, cache.v_scale)
    want = torch.stack([v[table[b, at[b] // P], :, at[b] % P] for b in range(B)])[:, None].repeat_interleave(2, 2)
    err = (out.cpu().to(F64) - want).abs()
    assert torch.all(err <= (2.0 ** -20 + 2.0 ** -8) * want.abs()), float((err / want.abs().clamp(min=1e-300)).max())
    assert status() == 0
