"""The full-attention operators on the GPU against their 64-bit definitions
(tests/_attn_ref.py): norm + rotation and its gradients, the paged cache
written and read back, and the attention of new tokens over it."""
import math

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _attn_ref as R

pytestmark = pytest.mark.gpu

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu
DEV = "cuda:0"
EPS = 1e-6


@pytest.fixture(scope="module")
def attn():
    from gated_deltanet_linear_04_gb300.build import build_library
    build_library()
    from gated_deltanet_linear_04_gb300 import attn as a, gdn
    assert torch.cuda.is_available(), "these tests need a GPU"
    torch.cuda.set_device(0)
    gdn.gdn_device_status()
    yield a
    assert gdn.gdn_device_status() == gdn.GDN_OK


def status():
    from gated_deltanet_linear_04_gb300 import gdn
    return gdn.gdn_device_status()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g) * std).to(BF16)


def views(g, d, gated=False):
    """q, k, v as views of one packed CPU projection (q's heads twice as wide
    when gated), and the same views on the GPU."""
    wide = 2 * d.D if gated else d.D
    x = normal(g, d.B, d.T, d.Hq * wide + 2 * d.Hkv * d.D, std=2.0)

    def split(x):
        q = x[..., :d.Hq * wide].view(d.B, d.T, d.Hq, wide)[..., :d.D]
        k, v = (x[..., d.Hq * wide + i * d.Hkv * d.D:][..., :d.Hkv * d.D].view(d.B, d.T, d.Hkv, d.D) for i in (0, 1))
        return q, k, v

    return split(x), split(x.to(DEV))


def weights(g, d):
    return [(torch.rand(d.D, generator=g) + 0.5) for _ in range(2)]


def near_bf16(got, want, noise, what):
    """One bf16 rounding of a result that is `noise` (absolute) off."""
    got = got.detach().cpu().to(F64)
    assert got.shape == want.shape
    bad = ~((got - want).abs() <= 2.0 ** -8 * want.abs() + noise)
    assert not bad.any(), "%s: %d of %d off, worst %.3e at value %.3e" % (
        what, int(bad.sum()), bad.numel(), float((got - want).abs()[bad].max()), float(want[bad].abs().max()))


# ---------------------------------------------------------------------------
# norm + rotation
# ---------------------------------------------------------------------------
NORM_CASES = [
    # B, T, Hq, Hkv, D, Drot, interleaved, masked, weighted, first position
    (1, 1, 1, 1, 64, 16, False, False, True, 0),
    (2, 3, 4, 2, 64, 64, False, True, True, 5),
    (3, 7, 9, 3, 64, 32, True, True, True, 100),
    (2, 5, 16, 2, 256, 64, False, False, True, 200000),
    (1, 65, 6, 2, 128, 128, True, False, True, 10 ** 6),
    (2, 33, 12, 1, 128, 96, False, True, True, 2 ** 31 - 100),
    (1, 130, 16, 1, 256, 256, False, False, True, -50),
    (1, 4, 3, 3, 256, 48, True, False, False, 7),
    (4, 9, 8, 8, 128, 0, False, True, True, 0),
    (1, 17, 5, 5, 64, 64, False, False, False, -2 ** 31),
    (1, 700, 32, 8, 128, 64, False, True, True, 3),
]


def norm_case(case):
    B, T, Hq, Hkv, D, rot, inter, masked, weighted, first = case
    d = wl.AttnDims(B, T, Hq, Hkv, D, rot, inter, EPS)
    g = gen(sum(case[:6]))
    cpu, gpu = views(g, d, gated=Hq % 2 == 0)
    w = weights(g, d) if weighted else [None, None]
    pos = (first + torch.arange(T)[None, :] + torch.arange(B)[:, None]).to(I32)
    mask = None
    if masked:
        mask = (torch.rand((B, T), generator=g) < 0.6).to(torch.uint8)
        mask[0] = 0                                      # a row without any token
        mask[-1, 0] = 1
    return d, cpu, gpu, w, pos, mask


def to_dev(*ts):
    return [None if t is None else t.to(DEV) for t in ts]


@pytest.mark.parametrize("case", NORM_CASES)
def test_norm_rope(attn, case):
    d, (q, k, _), (qg, kg, _), w, pos, mask = norm_case(case)
    inv = attn.rope_inv_freq(d.Drot)
    wq, wk, posg, maskg = to_dev(*w, pos, mask)
    qo, ko = attn.qk_norm_rope(d, qg, kg, wq, wk, attn.rope_freqs(inv, DEV), posg, maskg)
    for got, x, ww, what in ((qo, q, w[0], "q"), (ko, k, w[1], "k")):
        want = R.norm_rope(x, ww, pos, inv, d.interleaved, EPS, mask)
        # f32: the norm's and the rotation's few roundings, the angle to 2^-23
        near_bf16(got, want, 2.0 ** -20 * R.norm(x.to(F64), ww, EPS).abs().amax(-1, keepdim=True), what)
        if mask is not None:
            assert torch.all(got.cpu()[mask == 0] == 0)


def test_norm_rope_in_place_and_empty(attn):
    d = wl.AttnDims(2, 5, 4, 2, 128, 64)
    g = gen(1)
    q, k = normal(g, 2, 5, 4, 128).to(DEV), normal(g, 2, 5, 2, 128).to(DEV)
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    pos = torch.arange(10, dtype=I32, device=DEV).view(2, 5)
    want = attn.qk_norm_rope(d, q, k, wq, wk, fr, pos)
    attn.gdn_qk_norm_rope(d, q, k, wq, wk, fr, pos, None, q, k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    e = d.with_(T=0)
    z = torch.empty((2, 0, 4, 128), dtype=BF16, device=DEV)
    qo, ko = attn.qk_norm_rope(e, z, z[:, :, :2], wq, wk, fr, pos[:, :0].contiguous())
    assert qo.shape == (2, 0, 4, 128) and ko.numel() == 0
    out = attn.qk_norm_rope_backward(e, z, z[:, :, :2], wq, wk, fr, pos[:, :0].contiguous(), qo, ko)
    assert torch.all(out["dwq"] == 0) and torch.all(out["dwk"] == 0)


@pytest.mark.parametrize("case", NORM_CASES)
def test_norm_rope_backward(attn, case):
    d, (q, k, _), (qg, kg, _), w, pos, mask = norm_case(case)
    g = gen(77)
    dq, dk = normal(g, d.B, d.T, d.Hq, d.D, std=0.1), normal(g, d.B, d.T, d.Hkv, d.D, std=0.1)
    inv = attn.rope_inv_freq(d.Drot)
    args = (d, qg, kg, *to_dev(*w), attn.rope_freqs(inv, DEV), *to_dev(pos, dq, dk, mask))
    out = attn.qk_norm_rope_backward(*args)
    again = attn.qk_norm_rope_backward(*args)
    assert set(out) == ({"dq", "dk"} if w[0] is None else {"dq", "dk", "dwq", "dwk"})
    for name in out:
        assert torch.equal(out[name], again[name]), name          # fixed summation order
    for n, x, ww, dy in (("q", q, w[0], dq), ("k", k, w[1], dk)):
        dx, dw, size = R.norm_rope_bwd(x, ww, dy, pos, inv, d.interleaved, EPS, mask)
        x64 = x.to(F64)
        rstd = 1.0 if ww is None else 1.0 / torch.sqrt((x64 * x64).mean(-1, keepdim=True) + EPS)
        top = dy.to(F64).abs().amax(-1, keepdim=True) * 2 * rstd * (1.0 if ww is None else 1.5)
        # f32: dz, the norm and the mean's sum, each term at most |w dz|max times |xhat|
        near_bf16(out["d" + n], dx, 2.0 ** -19 * top * (1 + (x64 * rstd).abs()), "d" + n)
        if mask is not None:
            assert torch.all(out["d" + n].cpu()[mask == 0] == 0)
        if ww is not None:
            # partial sums of f32 terms that are 2^-21 off
            err = (out["dw" + n].cpu().to(F64) - dw).abs()
            assert torch.all(err <= 2.0 ** -19 * size + 1e-30), float((err / size).max())


def test_norm_rope_backward_against_differences(attn):
    """The forward kernel's own outputs: f(x + h e) - f(x - h e) for a few
    directions e, f = sum dy y in f64 of the bf16 outputs.  One output's
    rounding is at most 2^-8 |y|, the step is large; the bound
    adds them all up."""
    d = wl.AttnDims(1, 2, 2, 1, 64, 32)
    g = gen(9)
    x, xk = normal(g, 1, 2, 2, 64), normal(g, 1, 2, 1, 64)
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(32), DEV)
    pos = torch.tensor([[3, 900]], dtype=I32, device=DEV)
    dy, dyk = normal(g, 1, 2, 2, 64), normal(g, 1, 2, 1, 64)
    out = attn.qk_norm_rope_backward(d, *to_dev(x, xk), wq, wk, fr, pos, *to_dev(dy, dyk))

    def f(w_):
        y, _ = attn.qk_norm_rope(d, *to_dev(x, xk), w_, wk, fr, pos)
        return (y.cpu().to(F64) * dy.to(F64)), y.cpu().to(F64)

    for i in (0, 17, 40, 63):
        e = torch.zeros(64, device=DEV)
        e[i] = 0.25
        (a, ya), (b, yb) = f(wq + e), f(wq - e)
        # f is linear in w: the quotient is exact up to the outputs' roundings
        reached = ya != yb                                  # the others round alike and cancel
        tol = 2.0 ** -8 * float(((ya.abs() + yb.abs()) * dy.to(F64).abs())[reached].sum()) / 0.5
        assert abs(float((a - b).sum()) / 0.5 - float(out["dwq"][i])) <= tol + 1e-4


# ---------------------------------------------------------------------------
# the cache
# ---------------------------------------------------------------------------
def make_cache(attn, d, n_pages, P, fp8, g=None):
    """A cache and its 64-bit values: zeros, or random rows."""
    c = attn.KVCache.empty(d, n_pages, P, E4M3 if fp8 else BF16, DEV)
    if g is not None:
        for pages, scale in ((c.k, c.k_scale), (c.v, c.v_scale)):
            x = torch.randn(pages.shape, generator=g)
            if fp8:
                pages.copy_((x * 100).clamp(-448, 448).to(E4M3))
                scale.view(torch.uint8).copy_(torch.randint(117, 122, scale.shape, generator=g).to(torch.uint8))
            else:
                pages.copy_(x.to(BF16))
    return c


def value64(pages, scale):
    x = pages.cpu().to(F64)
    return x if scale is None else x * scale.cpu().to(F64)[..., None]


def tables(g, B, width, n_pages):
    return torch.randperm(n_pages, generator=g)[:B * width].view(B, width).to(I32)


APPEND_CASES = [
    # B, T, Hq, Hkv, D, Drot, page size, fp8, positions, n_new
    (1, 1, 16, 2, 256, 64, 16, False, [0], None),
    (1, 1, 16, 2, 256, 64, 64, True, [1000], None),
    (3, 1, 4, 4, 64, 64, 32, True, [31, 32, 0], [1, 1, 0]),
    (4, 5, 9, 3, 64, 32, 16, False, [0, 14, 33, 7], [5, 2, 0, 99]),
    (2, 37, 8, 1, 128, 128, 16, True, [3, 250], [37, 20]),
    (2, 130, 6, 2, 128, 0, 256, True, [200, 1], None),
    (1, 300, 16, 2, 256, 64, 128, True, [77], [-4]),
    (1, 515, 2, 2, 64, 16, 64, False, [61], None),
]


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("case", APPEND_CASES)
def test_append_and_read(attn, case, inter):
    B, T, Hq, Hkv, D, rot, P, fp8, positions, n_new = case
    d = wl.AttnDims(B, T, Hq, Hkv, D, rot, inter, EPS)
    g = gen(D + T + P)
    (q, k, v), (qg, kg, vg) = views(g, d, gated=Hq == 16)
    w = weights(g, d)
    inv = attn.rope_inv_freq(rot)
    width = -(-(max(positions) + T) // P)
    n_pages = B * width + 2
    cache = make_cache(attn, d, n_pages, P, fp8, g)
    old = [t.cpu().clone() for t in (cache.k, cache.v)]
    table = tables(g, B, width, n_pages)
    pos = torch.tensor(positions, dtype=I32)
    nn = None if n_new is None else torch.tensor(n_new, dtype=I32)
    qo = attn.kv_append(d, qg, kg, vg, *to_dev(*w), attn.rope_freqs(inv, DEV), cache, *to_dev(table, pos, nn))
    n = [T if n_new is None else max(0, min(T, n_new[b])) for b in range(B)]
    live = torch.tensor([[t < n[b] for t in range(T)] for b in range(B)]).to(torch.uint8)
    tokens = pos[:, None].long() + torch.arange(T)
    want_q = R.norm_rope(q, w[0], tokens, inv, inter, EPS, live)
    near_bf16(qo, want_q, 2.0 ** -20 * R.norm(q.to(F64), w[0], EPS).abs().amax(-1, keepdim=True), "q")
    written = torch.zeros((n_pages, P), dtype=torch.bool)
    for x64, pages, scale, was, noise, name in (
            (R.norm_rope(k, w[1], tokens, inv, inter, EPS), cache.k, cache.k_scale, old[0], 2.0 ** -20, "k"),
            (v.to(F64), cache.v, cache.v_scale, old[1], 0.0, "v")):
        got = value64(pages, scale)
        for b in range(B):
            for t in range(n[b]):
                page, slot = R.lookup(table, n_pages, P, b, positions[b] + t)
                written[page, slot] = True
                x, y = x64[b, t], got[page, :, slot]
                off = noise * x.abs().amax(-1, keepdim=True)
                if not fp8:
                    assert torch.all((y - x).abs() <= 2.0 ** -8 * x.abs() * (noise > 0) + off), name
                    continue
                s = scale[page, :, slot].cpu().to(F64)[..., None]
                codes, e = R.e4m3(x)
                want_s = torch.ldexp(torch.ones_like(x[..., :1]), e[..., None])
                assert torch.equal(s, want_s), name
                # half a step of the code (2^-4 relative, 2^-10 at the subnormal end)
                assert torch.all((y - x).abs() <= torch.maximum(2.0 ** -4 * x.abs(), 2.0 ** -10 * s) + off), name
                # values: bits of the exact quotient's rounding; keys: away from a border
                if noise == 0.0:
                    assert torch.equal(y, codes * s), name
                else:
                    assert float((y != codes * s).double().mean()) <= 0.01
        keep = ~written
        raw = pages.view(torch.uint8) if fp8 else pages
        was = was.view(torch.uint8) if fp8 else was
        assert torch.equal(raw.cpu().transpose(1, 2)[keep], was.transpose(1, 2)[keep]), name + ": a stray write"
    # read back exactly what the cache holds
    kr, vr = attn.kv_read(d, cache, *to_dev(table, pos, nn))
    for got, pages, scale in ((kr, cache.k, cache.k_scale), (vr, cache.v, cache.v_scale)):
        held = value64(pages, scale)
        for b in range(B):
            for t in range(T):
                if t < n[b]:
                    page, slot = R.lookup(table, n_pages, P, b, positions[b] + t)
                    assert torch.equal(got[b, t].cpu().to(F64), held[page, :, slot])
                else:
                    assert torch.all(got[b, t] == 0)


def test_append_special_rows(attn):
    """Zero rows, the type's smallest and largest values, infinities and NaN."""
    d = wl.AttnDims(1, 6, 1, 1, 64, 0)
    v = torch.zeros((1, 6, 1, 64), dtype=BF16)
    v[0, 1, 0, 5] = 2.0 ** -133                   # smallest bf16
    v[0, 2, 0, :] = torch.finfo(BF16).max
    v[0, 3, 0, 7] = math.inf
    v[0, 4, 0, 9] = math.nan
    v[0, 5, 0, :3] = torch.tensor([448.0, -1.75, 2.0 ** -10])
    x = v.to(DEV)
    table = torch.zeros((1, 1), dtype=I32, device=DEV)
    pos = torch.zeros(1, dtype=I32, device=DEV)
    for fp8 in (True, False):
        cache = make_cache(attn, d, 1, 16, fp8)
        attn.kv_append(d, x, x, x, None, None, None, cache, table, pos)
        k, vv = attn.kv_read(d, cache, table, pos)
        same = torch.equal(k.view(torch.int16), vv.view(torch.int16))
        assert same                                                        # no norm, no rotation: alike
        got = vv.cpu()
        if not fp8:
            assert torch.allclose(got.to(F64), v.to(F64), rtol=0, atol=0, equal_nan=True)   # (a NaN's bits are free)
            continue
        assert cache.v_scale.view(torch.uint8).cpu()[0, 0, :6].tolist() == [0, 0, 247, 255, 255, 127]
        assert torch.all(got[0, 0] == 0)
        assert torch.all(torch.isnan(got[0, 3].float())) and torch.all(torch.isnan(got[0, 4].float()))
        # 1.9921875 * 2^127 is 254.99 * 2^120, nearest code 256: past bf16's end, an infinity when read
        assert torch.all(got[0, 2].float() == math.inf)
        assert got[0, 5, 0, :3].tolist() == [448.0, -1.75, 0.0]            # 2^-10: a tie at half the smallest code


def test_bad_pages_are_skipped_and_reported(attn):
    from gated_deltanet_linear_04_gb300 import gdn
    d = wl.AttnDims(3, 2, 2, 1, 64, 32)
    g = gen(4)
    _, (q, k, v) = views(g, d)
    w = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(32), DEV)
    # row 0: a good page then an entry past the cache; row 1: a negative entry; row 2: a position past the table
    table = torch.tensor([[1, 7], [-1, 0], [2, 0]], dtype=I32, device=DEV)
    pos = torch.tensor([15, 0, 31], dtype=I32, device=DEV)
    for fp8 in (False, True):
        cache = make_cache(attn, d, 4, 16, fp8)
        assert status() == gdn.GDN_OK
        attn.kv_append(d, q, k, v, *w, fr, cache, table, pos)
        assert status() == gdn.GDN_ERR_BAD_PAGE
        used = (value64(cache.v, cache.v_scale) != 0).any(-1)[:, 0]
        at = {(int(p), int(s)) for p, s in torch.nonzero(used)}
        assert at == {(1, 15), (0, 15)}                              # row 0 token 0, row 2 token 0
        kr, vr = attn.kv_read(d, cache, table, pos)
        assert status() == gdn.GDN_ERR_BAD_PAGE
        assert torch.all(kr[0, 1] == 0) and torch.all(vr[1] == 0) and torch.all(vr[2, 1] == 0)
        assert torch.all((vr[0, 0] != 0).any(-1)) and torch.all((vr[2, 0] != 0).any(-1))
        neg = torch.tensor([-2, 0, -1], dtype=I32, device=DEV)
        before = cache.k.view(torch.uint8).clone()
        attn.kv_append(d, q, k, v, *w, fr, cache, torch.full_like(table, -5), neg)
        assert status() == gdn.GDN_ERR_BAD_PAGE and torch.equal(before, cache.k.view(torch.uint8))
    # a decode call leaves the keys of bad pages out
    q1 = normal(g, 3, 2, 2, 64)
    cache = make_cache(attn, d, 4, 16, False, g)
    out, lse = attn.attn_decode(d, q1.to(DEV), cache, table, pos, return_lse=True)
    assert status() == gdn.GDN_ERR_BAD_PAGE
    check_decode(out, lse, q1, cache, table.cpu(), [15, 0, 31], None, 64 ** -0.5)


# ---------------------------------------------------------------------------
# attention over the cache
# ---------------------------------------------------------------------------
def check_decode(out, lse, q, cache, table, pos, n_new, scale, gate=None):
    want, want_lse, tol, lse_tol = R.decode(q, value64(cache.k, cache.k_scale), value64(cache.v, cache.v_scale), table,
                                            cache.page_size, pos, n_new, scale, gate)
    got = out.cpu().to(F64)
    bad = ~((got - want).abs() <= tol)
    assert not bad.any(), "out: %d of %d off, worst %.3e (bound %.3e there)" % (
        int(bad.sum()), bad.numel(), float((got - want).abs()[bad].max()), float(tol[bad].min()))
    if got.numel() and float(want.norm()):
        assert float((got - want).norm() / want.norm()) <= 2.0 ** -8      # the roundings are random
    if lse is not None:
        got = lse.cpu().to(F64)
        empty = want_lse == -math.inf
        assert torch.all(got[empty] == -math.inf) and torch.all(out.cpu()[empty] == 0)
        assert torch.all((got - want_lse).abs()[~empty] <= lse_tol[~empty])


DECODE_CASES = [
    # B, T, Hq, Hkv, D, page size, positions, n_new, gated
    (1, 1, 16, 2, 256, 16, [0], None, True),                             # one key
    (1, 1, 16, 2, 256, 64, [1000], None, False),
    (2, 1, 8, 8, 64, 16, [15, 16], None, False),                         # one query head per key head
    (3, 1, 9, 3, 64, 32, [0, 63, 64], [1, 0, 1], True),                  # an empty row
    (5, 1, 12, 1, 128, 128, [5, 127, 128, 129, 700], None, False),
    (2, 1, 16, 1, 128, 256, [300, 2], None, True),                       # 16 query rows
    (2, 2, 16, 2, 256, 16, [31, 100], None, False),                      # 16 rows in a window
    (3, 4, 32, 8, 128, 32, [0, 61, 515], [4, 3, 1], True),
    (2, 8, 16, 2, 256, 64, [200, 3], [8, 5], False),                     # 64 rows
    (2, 8, 16, 1, 64, 16, [77, 0], None, True),                          # 128 rows
    (1, 5, 15, 1, 256, 16, [333], None, False),                          # 75 rows
    (1, 3, 7, 1, 128, 64, [4000], None, False),                          # 21 rows
    (2, 6, 24, 4, 64, 64, [0, 129], [0, 6], False),                      # 36 rows
    (40, 1, 4, 2, 64, 16, [(37 * i) % 191 for i in range(40)], None, False),
    (300, 1, 2, 1, 64, 16, [(7 * i) % 40 for i in range(300)], [i % 5 != 0 for i in range(300)], False),
    (1, 1, 8, 1, 256, 64, [20001], None, True),                          # split over the length
]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("case", DECODE_CASES)
def test_decode(attn, case, fp8):
    B, T, Hq, Hkv, D, P, pos, n_new, gated = case
    d = wl.AttnDims(B, T, Hq, Hkv, D)
    g = gen(B + T + Hq + D + P)
    width = -(-(max(pos) + T) // P)
    n_pages = B * width + 1
    cache = make_cache(attn, d, n_pages, P, fp8, g)
    table = tables(g, B, width, n_pages)
    q = normal(g, B, T, Hq, D, std=1.5)
    gate = normal(g, B, T, Hq, 2 * D)[..., D:] if gated else None
    gg = None if gate is None else torch.cat((torch.zeros_like(gate), gate), -1).to(DEV)[..., D:]
    nn = None if n_new is None else torch.tensor([int(x) for x in n_new], dtype=I32)
    args = (d, q.to(DEV), cache, *to_dev(table, torch.tensor(pos, dtype=I32), nn), gg)
    out, lse = attn.attn_decode(*args, return_lse=True)
    check_decode(out, lse, q, cache, table, pos, nn, D ** -0.5, gate)
    again = attn.attn_decode(*args)
    assert torch.equal(out, again)                                       # fixed order of the joins
    # a table wider than needed, its further entries never looked at
    wide = torch.cat((table, torch.full((B, 3), 1 << 30, dtype=I32)), 1).to(DEV)
    more, lse = attn.attn_decode(d, args[1], cache, wide, *args[4:], return_lse=True)
    check_decode(more, lse, q, cache, table, pos, nn, D ** -0.5, gate)   # (what a table could hold chooses the tiles)


@pytest.mark.parametrize("spare", [0, 64])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D", [(32, 8, 64), (24, 8, 128), (32, 8, 256)])
def test_decode_short_rows(attn, Hq, Hkv, D, fp8, spare):
    """Many rows of few keys: lengths around every tile's end, in tables with
    and without room for more (`spare` further pages per row)."""
    B, P = 80, 16
    d = wl.AttnDims(B, 1, Hq, Hkv, D)
    g = gen(B + D + spare)
    ends = (1, 16, 63, 64, 65, 127, 128, 129, 192, 193, 255, 256, 257)
    pos = [ends[i % len(ends)] - 1 for i in range(B)]
    width = -(-max(ends) // P)
    cache = make_cache(attn, d, B * width + 1, P, fp8, g)
    table = tables(g, B, width, B * width + 1)
    q, gate = normal(g, B, 1, Hq, D, std=1.5), normal(g, B, 1, Hq, D)
    wide = torch.cat((table, torch.full((B, spare), -1, dtype=I32)), 1)
    out, lse = attn.attn_decode(d, q.to(DEV), cache, wide.to(DEV), torch.tensor(pos, dtype=I32).to(DEV),
                                gate=gate.to(DEV), return_lse=True)
    check_decode(out, lse, q, cache, table, pos, None, D ** -0.5, gate)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("Hq,Hkv,D,T", [(16, 2, 256, 1), (32, 8, 128, 4), (16, 2, 64, 3)])
def test_decode_repeats_bit_for_bit(attn, Hq, Hkv, D, T, fp8):
    """Many tiles per CTA, many calls back to back: the ring's fills land in
    any order, the results are the same."""
    d = wl.AttnDims(3, T, Hq, Hkv, D)
    P, pos = 16, [60000, 45001, 70]
    width = -(-(max(pos) + T) // P)
    cache = make_cache(attn, d.with_(B=1), width, P, fp8)
    (cache.k.view(torch.uint8) if fp8 else cache.k).random_(0, 120)
    (cache.v.view(torch.uint8) if fp8 else cache.v).random_(0, 120)
    if fp8:
        cache.k_scale.view(torch.uint8).fill_(118)
        cache.v_scale.view(torch.uint8).random_(115, 121)
    table = torch.stack([torch.randperm(width, generator=gen(i)) for i in range(3)]).to(I32).to(DEV)
    q = normal(gen(5), 3, T, Hq, D).to(DEV)
    pg = torch.tensor(pos, dtype=I32, device=DEV)
    want = attn.attn_decode(d, q, cache, table, pg)
    got = [attn.attn_decode(d, q, cache, table, pg) for _ in range(100)]
    same = [torch.equal(g, want) for g in got]
    assert all(same) and status() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_ignores_unseen_slots(attn, fp8):
    """NaN and infinities in every slot past the rows' keys, and in a draft
    token's own key and value for the tokens before it."""
    B, T, P = 2, 3, 16
    d = wl.AttnDims(B, T, 4, 2, 64)
    g = gen(6)
    pos = [20, 14]
    cache = make_cache(attn, d, 7, P, fp8, g)
    table = tables(g, B, 3, 7)
    clean_k, clean_v = value64(cache.k, cache.k_scale), value64(cache.v, cache.v_scale)
    held = torch.zeros((7, P), dtype=torch.bool)
    for b in range(B):
        for j in range(pos[b] + T):
            held[R.lookup(table, 7, P, b, j)] = True
    raw = (lambda t: t.view(torch.uint8)) if fp8 else (lambda t: t.view(torch.int16))
    bad = 0x7f if fp8 else 0x7fc0
    for t in (cache.k, cache.v):
        raw(t).transpose(1, 2)[~held.to(DEV)] = bad
    q = normal(g, B, T, 4, 64)
    qg, tg, pg = to_dev(q, table, torch.tensor(pos, dtype=I32))
    want, _, tol, _ = R.decode(q, clean_k, clean_v, table, P, pos, None, 0.125)
    out = attn.attn_decode(d, qg, cache, tg, pg)
    assert torch.all((out.cpu().to(F64) - want).abs() <= tol)
    # the second draft token's value is NaN, its key infinite (NaN in e4m3): token 0 does not see it
    for b in range(B):
        page, slot = R.lookup(table, 7, P, b, pos[b] + 1)
        raw(cache.v)[page, :, slot] = bad
        raw(cache.k)[page, :, slot] = bad if fp8 else 0x7f80
    out2 = attn.attn_decode(d, qg, cache, tg, pg)
    assert torch.equal(out2[:, 0], out[:, 0])
    assert torch.all(torch.isnan(out2[:, 1:].float()))


def test_decode_extreme_scores_and_scales(attn):
    """Scores of thousands, a negative and a zero scale, e4m3 rows whose scales
    lie 2^60 apart."""
    d = wl.AttnDims(2, 1, 4, 2, 64)
    g = gen(8)
    q = normal(g, 2, 1, 4, 64, std=30.0)
    pos = [90, 33]
    table = tables(g, 2, 6, 12)
    qg, tg, pg = to_dev(q, table, torch.tensor(pos, dtype=I32))
    for fp8 in (False, True):
        cache = make_cache(attn, d, 12, 16, fp8, g)
        for scale in (10.0, -1.0, 0.0):
            out, lse = attn.attn_decode(d, qg, cache, tg, pg, scale=scale, return_lse=True)
            check_decode(out, lse, q, cache, table, pos, None, scale)
    cache.v_scale.view(torch.uint8).copy_(torch.randint(67, 187, cache.v_scale.shape, generator=g).to(torch.uint8))
    cache.k_scale.view(torch.uint8).copy_(torch.randint(90, 122, cache.k_scale.shape, generator=g).to(torch.uint8))
    out, lse = attn.attn_decode(d, qg, cache, tg, pg, return_lse=True)
    check_decode(out, lse, q, cache, table, pos, None, 0.125)
    # all values zero so far (scale byte 0), then rows that are not
    cache.v.view(torch.uint8).zero_()
    cache.v_scale.view(torch.uint8).zero_()
    page, slot = R.lookup(table, 12, 16, 0, 90)
    cache.v.view(torch.uint8)[page, :, slot] = 0x38                      # 1.0
    cache.v_scale.view(torch.uint8)[page, :, slot] = 127
    out, lse = attn.attn_decode(d, qg, cache, tg, pg, return_lse=True)
    check_decode(out, lse, q, cache, table, pos, None, 0.125)


def test_decode_large_queries_in_e4m3(attn):
    """Query rows past fp16's range over an e4m3 cache."""
    d = wl.AttnDims(1, 1, 2, 1, 64)
    g = gen(12)
    cache = make_cache(attn, d, 3, 16, True, g)
    table = tables(g, 1, 3, 3)
    for std in (1e6, 1e-7):
        q = normal(g, 1, 1, 2, 64, std=std)
        scale = 0.125 / std
        out, lse = attn.attn_decode(d, q.to(DEV), cache, table.to(DEV), torch.tensor([40], dtype=I32, device=DEV),
                                    scale=scale, return_lse=True)
        check_decode(out, lse, q, cache, table, [40], None, scale)


def test_shared_pages_streams_and_graphs(attn):
    """Rows that share a prefix's pages; a side stream; a captured step
    replayed on new inputs."""
    B, P = 4, 16
    d = wl.AttnDims(B, 1, 8, 2, 128, 64)
    g = gen(11)
    (q, k, v), (qg, kg, vg) = views(g, d)
    wq, wk = to_dev(*weights(g, d))
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    table = torch.tensor([[0, 1, 2 + b] for b in range(B)], dtype=I32)     # two shared pages each
    pos = [33, 40, 35, 46]
    tg, pg = to_dev(table, torch.tensor(pos, dtype=I32))

    def step(cache, **kw):
        qo = attn.kv_append(d, qg, kg, vg, wq, wk, fr, cache, tg, pg, **kw)
        return qo, attn.attn_decode(d, qo, cache, tg, pg, **kw)

    cache = make_cache(attn, d, 6, P, True, gen(12))
    qo, out = step(cache)
    check_decode(out, None, qo.cpu(), cache, table, pos, None, 128 ** -0.5)
    other = make_cache(attn, d, 6, P, True, gen(12))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    qo2, out2 = step(other, stream=side)
    side.synchronize()
    assert torch.equal(out2, out) and torch.equal(qo2, qo)
    third = make_cache(attn, d, 6, P, True, gen(12))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        qo3, out3 = step(third)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out3, out) and torch.equal(third.k.view(torch.uint8), cache.k.view(torch.uint8))
    pg += 1                                                            # the next step, from the same graph
    graph.replay()
    torch.cuda.synchronize()
    check_decode(out3, None, qo3.cpu(), third, table, [p + 1 for p in pos], None, 128 ** -0.5)


@pytest.mark.parametrize("fp8", [False, True])
def test_offsets_past_32_bits(attn, fp8):
    """A cache of more than 2^32 bytes per tensor, pages at both of its ends."""
    Hkv, D, P = 2, 256, 64
    n_pages = (1 << 33) // (Hkv * D * P) if fp8 else (1 << 32) // (Hkv * D * P)
    d = wl.AttnDims(1, 2, 4, Hkv, D, 64)
    c = attn.KVCache.empty(d, n_pages, P, E4M3 if fp8 else BF16, DEV)
    assert c.k.numel() * c.k.element_size() >= 1 << 33
    g = gen(13)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 2]], dtype=I32)
    w = weights(g, d)
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    wq, wk, tg = to_dev(*w, table)
    T = 131
    (q, k, v), (qg, kg, vg) = views(g, d.with_(T=T))
    zero = torch.zeros(1, dtype=I32, device=DEV)
    attn.kv_append(d.with_(T=T), qg, kg, vg, wq, wk, fr, c, tg, zero)
    kr, vr = attn.kv_read(d.with_(T=T), c, tg, zero)
    if not fp8:
        assert torch.equal(vr.cpu(), v)
    pos = torch.tensor([T - 2], dtype=I32)
    q1 = normal(g, 1, 2, 4, D)
    out, lse = attn.attn_decode(d, q1.to(DEV), c, tg, pos.to(DEV), return_lse=True)
    # the same three pages as a small cache
    order = torch.tensor([0, 1, 2])
    pick = torch.tensor([n_pages - 1, 0, n_pages - 2], device=DEV)
    raw = [t.view(torch.uint8)[pick].view(t.dtype) for t in (c.k, c.v)]
    small = attn.KVCache(*raw, *((None, None) if not fp8 else
                                 (t.view(torch.uint8)[pick].view(E8M0) for t in (c.k_scale, c.v_scale))))
    check_decode(out, lse, q1, small, order.to(I32)[None], [T - 2], None, D ** -0.5)


def test_binding_device_checks(attn):
    d = wl.AttnDims(1, 1, 2, 1, 64, 0)
    cache = make_cache(attn, d, 2, 16, False)
    q = torch.zeros((1, 1, 2, 64), dtype=BF16, device=DEV)
    table = torch.zeros((1, 1), dtype=I32, device=DEV)
    pos = torch.zeros(1, dtype=I32, device=DEV)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        attn.attn_decode(d, q.cpu(), cache, table, pos, workspace=torch.zeros(1 << 20, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="page_table"):
        attn.attn_decode(d, q, cache, table[0], pos)
    with pytest.raises(ValueError, match="heads of"):
        attn.attn_decode(d.with_(Hkv=2), q, cache, table, pos)
    with pytest.raises(ValueError, match="pos must have shape"):
        attn.attn_decode(d, q, cache, table, torch.zeros(2, dtype=I32, device=DEV))
    with pytest.raises(TypeError, match="pos must be"):
        attn.attn_decode(d, q, cache, table, pos.long())
