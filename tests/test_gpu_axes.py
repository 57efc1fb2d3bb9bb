"""Norm + rotation with positions on several axes on the GPU: against the
64-bit definition pair by pair, and one axis against the plain calls."""
import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _attn_ref as R
from tests.test_gpu_attn import DEV, EPS, F64, I32, attn, gen, make_cache, near_bf16, normal, tables, to_dev, views, weights  # noqa: F401,E501

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


def turned(y, x, w, pos, axes, inv, inter, mask=None, sign=1.0, normed=True):
    """norm_rope (or the turn alone) with each pair's own axis."""
    z = R.norm(x.to(F64), None if w is None else w.to(F64), EPS) if normed else x.to(F64)
    out = z.clone()
    half = inv.numel()
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if inter else (i, half + i)
        ang = sign * pos[int(axes[i])].to(F64)[..., None] * inv[i]
        out[..., a] = z[..., a] * torch.cos(ang) - z[..., b] * torch.sin(ang)
        out[..., b] = z[..., b] * torch.cos(ang) + z[..., a] * torch.sin(ang)
    return out if mask is None else torch.where((mask != 0)[..., None, None], out, torch.zeros_like(out))


# B, T, Hq, Hkv, D, Drot, interleaved, axes, cyclic, masked, weighted
CASES = [
    (1, 1, 1, 1, 64, 16, False, 3, False, False, True),
    (2, 3, 4, 2, 64, 64, True, 3, True, True, True),
    (3, 37, 9, 3, 128, 96, False, 2, False, True, True),
    (2, 5, 16, 2, 256, 64, False, 3, True, False, True),
    (1, 700, 16, 2, 256, 256, True, 8, True, True, False),
    (4, 9, 8, 8, 128, 0, False, 1, False, True, True),
    (1, 1500, 32, 8, 64, 32, False, 4, False, False, True),
]


def make(attn, case):  # noqa: F811
    B, T, Hq, Hkv, D, rot, inter, A, cyclic, masked, weighted = case
    d = wl.AttnDims(B, T, Hq, Hkv, D, rot, inter, EPS)
    g = gen(sum(case[:6]))
    cpu, gpu = views(g, d)
    w = weights(g, d) if weighted else [None, None]
    pos = torch.randint(-50, 100000, (A, B, T), generator=g, dtype=I32)
    n = rot // 2
    axes = attn.rope_axes([n // A + (i < n % A) for i in range(A)], cyclic)
    mask = None
    if masked:
        mask = (torch.rand((B, T), generator=g) < 0.6).to(torch.uint8)
    return d, g, cpu, gpu, w, pos, axes, mask


@pytest.mark.parametrize("case", CASES)
def test_forward(attn, case):  # noqa: F811
    d, g, (q, k, _), (qg, kg, _), w, pos, axes, mask = make(attn, case)
    inv = attn.rope_inv_freq(d.Drot)
    wq, wk, posg, axesg, maskg = to_dev(*w, pos, axes, mask)
    qo, ko = attn.qk_norm_rope_axes(d, qg, kg, wq, wk, attn.rope_freqs(inv, DEV), axesg, posg, maskg)
    for got, x, ww, what in ((qo, q, w[0], "q"), (ko, k, w[1], "k")):
        want = turned(None, x, ww, pos, axes, inv, d.interleaved, mask)
        # f32: the norm's and the rotation's few roundings, the angle to 2^-23
        near_bf16(got, want, 2.0 ** -20 * R.norm(x.to(F64), ww, EPS).abs().amax(-1, keepdim=True), what)


@pytest.mark.parametrize("case", CASES)
def test_backward(attn, case):  # noqa: F811
    d, g, (q, k, _), (qg, kg, _), w, pos, axes, mask = make(attn, case)
    inv = attn.rope_inv_freq(d.Drot)
    dqo, dko = normal(g, d.B, d.T, d.Hq, d.D, std=0.1), normal(g, d.B, d.T, d.Hkv, d.D, std=0.1)
    wq, wk, posg, axesg, maskg, a, b = to_dev(*w, pos, axes, mask, dqo, dko)
    got = attn.qk_norm_rope_axes_backward(d, qg, kg, wq, wk, attn.rope_freqs(inv, DEV), axesg, posg, a, b, maskg)
    for n, x, dy, ww in (("q", q, dqo, w[0]), ("k", k, dko, w[1])):
        dz = turned(None, dy, None, pos, axes, inv, d.interleaved, mask, -1.0, normed=False)
        x = x.to(F64)
        if ww is None:
            near_bf16(got["d" + n], dz, 2.0 ** -20 * dy.to(F64).abs().amax(-1, keepdim=True), "d" + n)
            continue
        rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS)
        xhat, gz = x * rstd, dz * ww.to(F64)
        dx = rstd * (gz - xhat * (gz * xhat).mean(-1, keepdim=True))
        noise = 2.0 ** -19 * rstd * (gz.abs().amax(-1, keepdim=True) * (1 + xhat.abs() * xhat.abs().amax(-1, keepdim=True)))
        near_bf16(got["d" + n], dx, noise, "d" + n)
        dw, size = (dz * xhat).sum((0, 1, 2)), (dz * xhat).abs().sum((0, 1, 2))
        assert ((got["dw" + n].cpu().to(F64) - dw).abs() <= 2.0 ** -19 * size + 1e-12).all()


@pytest.mark.parametrize("inter", [False, True])
def test_one_axis_gives_the_bits_of_the_plain_calls(attn, inter):  # noqa: F811
    d = wl.AttnDims(3, 50, 16, 2, 256, 64, inter, EPS)
    g = gen(4)
    _, (q, k, v) = views(g, d)
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    pos = torch.randint(0, 9999, (3, 50), generator=g, dtype=I32).to(DEV)
    axes = attn.rope_axes([32], device=DEV)
    for x, y in zip(attn.qk_norm_rope(d, q, k, wq, wk, fr, pos), attn.qk_norm_rope_axes(d, q, k, wq, wk, fr, axes, pos[None])):
        assert torch.equal(x, y)
    # axes that agree, and axis numbers past the last
    three = pos[None].expand(3, 3, 50).contiguous()
    odd = torch.arange(32, dtype=torch.uint8, device=DEV) * 8 + 7
    for x, y in zip(attn.qk_norm_rope(d, q, k, wq, wk, fr, pos), attn.qk_norm_rope_axes(d, q, k, wq, wk, fr, odd, three)):
        assert torch.equal(x, y)
    a = attn.qk_norm_rope_backward(d, q, k, wq, wk, fr, pos, q.contiguous(), k.contiguous())
    b = attn.qk_norm_rope_axes_backward(d, q, k, wq, wk, fr, axes, pos[None], q.contiguous(), k.contiguous())
    for n in a:
        assert torch.equal(a[n], b[n]), n


@pytest.mark.parametrize("fp8", [False, True])
def test_append_turns_by_the_axes_and_writes_by_the_position(attn, fp8):  # noqa: F811
    """The cache afterwards is that of norm + rotation with axes, written where
    the plain append writes."""
    d = wl.AttnDims(3, 21, 16, 2, 256, 64, False, EPS)
    g = gen(6)
    _, (q, k, v) = views(g, d)
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    axes = attn.rope_axes([11, 11, 10], cyclic=True, device=DEV)
    rope = torch.randint(0, 500, (3, 3, 21), generator=g, dtype=I32).to(DEV)
    table = tables(g, 3, 6, 40).to(DEV)
    start = torch.tensor([0, 33, 70], dtype=I32, device=DEV)
    n = torch.tensor([21, 0, 13], dtype=I32, device=DEV)
    a, b = (make_cache(attn, d, 40, 16, fp8) for _ in range(2))
    got = attn.kv_append_axes(d, q, k, v, wq, wk, fr, axes, rope, a, table, start, n)
    qr, kr = attn.qk_norm_rope_axes(d, q, k, wq, wk, fr, axes, rope)
    keep = (torch.arange(21, device=DEV) < n[:, None])[..., None, None]
    assert torch.equal(got, torch.where(keep, qr, torch.zeros_like(qr)))
    # (the plain append without norm and rotation; with e4m3 the keys were rounded to bf16 on the way)
    plain = d.with_(Drot=0)
    attn.kv_append(plain, q, kr, v, None, None, None, b, table, start, n)
    view = (lambda x: x.view(torch.uint8)) if fp8 else (lambda x: x)  # noqa: E731
    assert torch.equal(view(a.v), view(b.v))
    if not fp8:
        assert torch.equal(a.k, b.k)
        return
    assert torch.equal(view(a.v_scale), view(b.v_scale))
    x, y = (attn.kv_read(d.with_(T=96), c, table, torch.zeros(3, dtype=I32, device=DEV), start + n)[0].double() for c in (a, b))
    # each e4m3 rounding: half of 2^-3 of the value or of the smallest step, 2^-9 of the scale <= amax / 224
    amax = y.abs().amax(-1, keepdim=True)
    assert ((x - y).abs() <= 2.0 ** -3 * y.abs() + 2.0 ** -8 * y.abs() + 2.0 ** -9 * amax / 112).all()


def test_streams_and_graphs(attn):  # noqa: F811
    d = wl.AttnDims(2, 300, 8, 2, 128, 64, False, EPS)
    g = gen(8)
    _, (q, k, _) = views(g, d)
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    axes = attn.rope_axes([16, 8, 8], device=DEV)
    pos = torch.randint(0, 500, (3, 2, 300), generator=g, dtype=I32).to(DEV)
    want = attn.qk_norm_rope_axes(d, q, k, wq, wk, fr, axes, pos)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = attn.qk_norm_rope_axes(d, q, k, wq, wk, fr, axes, pos, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = attn.qk_norm_rope_axes(d, q, k, wq, wk, fr, axes, pos)
    pos.add_(17)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(attn.qk_norm_rope_axes(d, q, k, wq, wk, fr, axes, pos), out))
