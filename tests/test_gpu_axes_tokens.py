"""Single new tokens with positions on several axes into the paged cache: a
serving step of a prompt with images."""
import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _attn_ref as A
from tests.test_gpu_attn import DEV, EPS, F64, I32, attn, gen, make_cache, near_bf16, normal, tables, to_dev, weights  # noqa: F401
from tests.test_gpu_axes import turned

pytestmark = pytest.mark.gpu


# B, Hq, Hkv, D, Drot, interleaved, axes, page size
CASES = [
    (1, 16, 2, 256, 64, False, 3, 16),
    (128, 16, 2, 256, 64, False, 3, 64),
    (37, 9, 3, 64, 32, True, 2, 16),
    (5, 32, 8, 128, 128, True, 8, 32),
    (3, 8, 8, 128, 0, False, 3, 16),                     # no pair turns
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_append_of_single_tokens(attn, case, fp8):  # noqa: F811
    """Queries as the definition has them, keys and values in the cache as norm +
    rotation and the plain append leave them; rows without a new token stay."""
    B, Hq, Hkv, D, rot, inter, A_, P = case
    d = wl.AttnDims(B, 1, Hq, Hkv, D, rot, inter, EPS)
    g = gen(sum(case[:5]))
    q, k, v = normal(g, B, 1, Hq, D), normal(g, B, 1, Hkv, D), normal(g, B, 1, Hkv, D)
    w = weights(g, d)
    qg, kg, vg, wq, wk = to_dev(q, k, v, *w)
    inv = attn.rope_inv_freq(rot)
    fr = attn.rope_freqs(inv, DEV)
    n = rot // 2
    axes = attn.rope_axes([n // A_ + (i < n % A_) for i in range(A_)], cyclic=True)
    rope = torch.randint(-20, 300000, (A_, B, 1), generator=g, dtype=I32)
    width = 5
    table = tables(g, B, width, B * width + 2).to(DEV)
    start = torch.randint(0, width * P - 1, (B,), generator=g, dtype=I32)
    new = (torch.arange(B) % 4 != 1).to(I32) if B > 1 else torch.ones(1, dtype=I32)
    startg, newg, ropeg, axesg = to_dev(start, new, rope, axes)
    a, b = (make_cache(attn, d, B * width + 2, P, fp8) for _ in range(2))
    got = attn.kv_append_axes(d, qg, kg, vg, wq, wk, fr, axesg, ropeg, a, table, startg, newg)
    want = turned(None, q, w[0], rope, axes, inv, inter)
    there = (new != 0)[:, None, None, None]
    noise = 2.0 ** -20 * A.norm(q.to(F64), w[0], EPS).abs().amax(-1, keepdim=True)
    near_bf16(got, torch.where(there, want, torch.zeros_like(want)), noise, "q")
    _, kr = attn.qk_norm_rope_axes(d, qg, kg, wq, wk, fr, axesg, ropeg)
    attn.kv_append(d.with_(Drot=0), qg, kr, vg, None, None, None, b, table, startg, newg)
    view = (lambda x: x.view(torch.uint8)) if fp8 else (lambda x: x)  # noqa: E731
    assert torch.equal(view(a.v), view(b.v))
    if not fp8:
        assert torch.equal(a.k, b.k)
        return
    assert torch.equal(view(a.v_scale), view(b.v_scale))
    one = torch.ones(B, dtype=I32, device=DEV)
    x, y = (attn.kv_read(d, c, table, startg, one * newg)[0].double() for c in (a, b))
    # each e4m3 rounding: half of 2^-3 of the value or of the smallest step, 2^-9 of the scale <= amax / 224; bf16 before one
    amax = y.abs().amax(-1, keepdim=True)
    assert ((x - y).abs() <= 2.0 ** -3 * y.abs() + 2.0 ** -8 * y.abs() + 2.0 ** -9 * amax / 112).all()


def test_a_captured_step_moves_on(attn):  # noqa: F811
    """One graph of the append; positions and tokens change between replays."""
    d = wl.AttnDims(4, 1, 16, 2, 256, 64, False, EPS)
    g = gen(3)
    q, k, v = (x.to(DEV) for x in (normal(g, 4, 1, 16, 256), normal(g, 4, 1, 2, 256), normal(g, 4, 1, 2, 256)))
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    axes = attn.rope_axes([11, 11, 10], device=DEV)
    rope = torch.zeros((3, 4, 1), dtype=I32, device=DEV)
    pos = torch.zeros(4, dtype=I32, device=DEV)
    table = tables(g, 4, 2, 10).to(DEV)
    a, b = (make_cache(attn, d, 10, 16, False) for _ in range(2))
    attn.kv_append_axes(d, q, k, v, wq, wk, fr, axes, rope, a, table, pos)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attn.kv_append_axes(d, q, k, v, wq, wk, fr, axes, rope, a, table, pos)
    for t in range(20):
        for x in (q, k, v):
            x.copy_(normal(g, *x.shape).to(DEV))
        rope.copy_(torch.randint(0, 99, (3, 4, 1), generator=g, dtype=I32).to(DEV))
        pos.fill_(t)
        graph.replay()
        want = attn.kv_append_axes(d, q, k, v, wq, wk, fr, axes, rope, b, table, pos)
        assert torch.equal(out, want)
    assert torch.equal(a.k, b.k) and torch.equal(a.v, b.v)
