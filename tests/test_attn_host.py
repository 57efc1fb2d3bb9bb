"""The full-attention operators without a GPU: refusals of the C ABI and of
the binding, workspace sizes, the rotation's frequency table, and the 64-bit
reference of the GPU tests against differences and exact values."""
import ctypes
import math
from fractions import Fraction

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _attn_ref as R

BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def lib():
    from gated_deltanet_linear_04_gb300.build import build_library
    build_library()
    from gated_deltanet_linear_04_gb300 import gdn
    return gdn.lib()


@pytest.fixture(scope="module")
def attn(lib):
    from gated_deltanet_linear_04_gb300 import attn as a
    return a


def dims(**kw):
    base = dict(B=2, T=3, Hq=4, Hkv=2, D=64, Drot=32)
    base.update(kw)
    return wl.AttnDims(**base)


BUF = ctypes.create_string_buffer(1 << 16)
P = (ctypes.addressof(BUF) + 255) // 256 * 256


def cache_struct(attn, **kw):
    base = dict(k=P, v=P, k_scale=None, v_scale=None, n_pages=4, page_size=16, format=0)
    base.update(kw)
    return attn.GdnKvCache(**base)


def abi_calls(lib, attn, d, heads=(P, 256, 64), cache=None, table=P, width=2, idx=P, ptr=P, wq=P, wk=P, freqs=P,
              ws_bytes=1 << 30, scale=0.125, only=("norm", "bwd", "append", "read", "decode")):
    """The entry points with the given arguments -> {name: status}.  The
    addresses are host memory: every call made here has to be refused (or be
    empty), so that nothing is launched."""
    c = ctypes.byref(cache if cache is not None else cache_struct(attn))
    r = ctypes.byref(attn.make_attn_dims(d))
    calls = {
        "norm": lambda: lib.gdn_qk_norm_rope(r, *heads, *heads, wq, wk, freqs, idx, None, ptr, ptr, None),
        "bwd": lambda: lib.gdn_qk_norm_rope_backward(r, *heads, *heads, wq, wk, freqs, idx, None, ptr, ptr, ptr, ptr,
                                             None if wq is None else ptr, None if wk is None else ptr, ptr, ws_bytes,
                                             None),
        "append": lambda: lib.gdn_kv_append(r, *heads, *heads, *heads, wq, wk, freqs, c, table, width, idx, None, ptr, None),
        "read": lambda: lib.gdn_kv_read(r, c, table, width, idx, None, ptr, ptr, None),
        "decode": lambda: lib.gdn_attn_decode(r, ptr, c, table, width, idx, None, None, 0, 0, scale, ptr, None, ptr, ws_bytes,
                                      None),
    }
    return {name: calls[name]() for name in only}


@pytest.mark.parametrize("kw,status", [
    ({"B": -1}, 1), ({"T": -1}, 1), ({"Hq": 0}, 1), ({"Hkv": 0}, 1), ({"Hq": 5}, 1), ({"Drot": 80}, 1),
    ({"Drot": -16}, 1), ({"eps": -1.0}, 1), ({"eps": math.nan}, 1), ({"D": 0}, 1),
    ({"D": 96, "Drot": 0}, 2), ({"D": 512}, 2), ({"Drot": 8}, 2), ({"Drot": 40}, 2), ({"Hq": 34}, 2),
    ({"B": 65536}, 2), ({"Hq": 2048, "Hkv": 2048}, 2),
])
def test_bad_dims_are_refused_everywhere(lib, attn, kw, status):
    assert set(abi_calls(lib, attn, dims(**kw)).values()) == {status}
    assert attn.gdn_attn_decode_workspace_size(dims(**kw)) == 0
    assert attn.gdn_qk_norm_rope_backward_workspace_size(dims(**kw)) == 0


def test_null_and_misaligned_pointers(lib, attn):
    d = dims()
    assert set(abi_calls(lib, attn, d, ptr=None).values()) == {1}
    assert set(abi_calls(lib, attn, d, ptr=P + 2).values()) == {1}
    assert set(abi_calls(lib, attn, d, idx=None).values()) == {1}
    assert set(abi_calls(lib, attn, d, idx=P + 2).values()) == {1}


@pytest.mark.parametrize("heads", [(None, 256, 64), (P + 8, 256, 64), (P, 252, 64), (P, 256, 60), (P, -256, 64),
                                   (P, 256, -64)])
def test_bad_head_views(lib, attn, heads):
    got = abi_calls(lib, attn, dims(), heads=heads, cache=cache_struct(attn, n_pages=-1))
    assert got["norm"] == got["bwd"] == 1
    got = abi_calls(lib, attn, dims(), heads=heads, ptr=None)
    assert got["append"] == 1


@pytest.mark.parametrize("kw,status", [
    ({"page_size": 8}, 2), ({"page_size": 48}, 2), ({"page_size": 512}, 2), ({"format": 2}, 2), ({"n_pages": -1}, 1),
    ({"k": None}, 1), ({"v": P + 8}, 1), ({"k_scale": P}, 1), ({"format": 1}, 1), ({"format": 1, "k_scale": P}, 1),
    ({"n_pages": 1 << 31}, 2), ({"n_pages": 1 << 26}, 2),
])
def test_bad_caches(lib, attn, kw, status):
    got = abi_calls(lib, attn, dims(), cache=cache_struct(attn, **kw), ptr=None)
    assert {got[n] for n in ("append", "read", "decode")} == {status}


def test_bad_tables_weights_workspaces_and_scales(lib, attn):
    d = dims()
    serving = ("append", "read", "decode")
    assert {abi_calls(lib, attn, d, table=None, ptr=None)[n] for n in serving} == {1}
    assert {abi_calls(lib, attn, d, width=-1, only=[n])[n] for n in serving} == {1}
    for kw in ({"wq": None}, {"wk": None}, {"wq": P + 4}, {"freqs": None}):
        got = abi_calls(lib, attn, d, **kw, only=("norm", "bwd", "append"))
        assert set(got.values()) == {1}, kw
    need = attn.gdn_attn_decode_workspace_size(d)
    assert need > 0 and abi_calls(lib, attn, dims(T=1, D=96, Drot=0))["decode"] == 2
    r = ctypes.byref(attn.make_attn_dims(d))
    c = ctypes.byref(cache_struct(attn))

    def decode(scale=0.1, ws=P, n=need, gate=(None, 0, 0), table=P):
        return lib.gdn_attn_decode(r, P, c, table, 2, P, None, *gate, scale, P, None, ws, n, None)

    assert decode(n=need - 1) == decode(ws=None) == decode(ws=P + 8) == 1
    assert decode(scale=math.inf) == decode(scale=math.nan) == 1
    assert decode(gate=(P + 2, 256, 64)) == decode(gate=(P, 4, 64)) == 1
    need = attn.gdn_qk_norm_rope_backward_workspace_size(d)
    assert need > 0
    assert abi_calls(lib, attn, d, ws_bytes=need - 1, only=["bwd"])["bwd"] == 1


@pytest.mark.parametrize("T", [0, 9])
def test_decode_takes_one_to_eight_tokens(lib, attn, T):
    assert abi_calls(lib, attn, dims(T=T), only=["decode"])["decode"] == 2
    assert attn.gdn_attn_decode_workspace_size(dims(T=T)) == 0


def test_empty_batches_are_noops(lib, attn):
    got = abi_calls(lib, attn, dims(B=0), heads=(None, 0, 0), table=None, idx=None, ptr=None, wq=None, wk=None)
    assert set(got.values()) == {0}


def test_status_string_of_a_bad_page(lib):
    from gated_deltanet_linear_04_gb300 import gdn
    assert gdn.status_string(gdn.GDN_ERR_BAD_PAGE).startswith("GDN_ERR_BAD_PAGE")


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def meta(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def binding_call(attn, **kw):
    d = dims()
    a = dict(q=meta(2, 3, 4, 64), k=meta(2, 3, 2, 64), wq=meta(64, dtype=F32), wk=meta(64, dtype=F32),
             freqs=meta(16, dtype=torch.int64), pos=meta(2, 3, dtype=torch.int32), mask=None,
             q_out=meta(2, 3, 4, 64), k_out=meta(2, 3, 2, 64))
    a.update(kw)
    attn.gdn_qk_norm_rope(d, **a)


@pytest.mark.parametrize("kw,error,text", [
    ({}, ValueError, "q must be a CUDA tensor"),
    ({"q": meta(2, 3, 4, 32)}, ValueError, "q must have shape"),
    ({"q": meta(2, 3, 4, 64, dtype=F32)}, TypeError, "q must be torch.bfloat16"),
    ({"q": None}, TypeError, "q must be a torch.Tensor"),
])
def test_binding_refuses_bad_heads(attn, kw, error, text):
    with pytest.raises(error, match=text):
        binding_call(attn, **kw)


def test_head_views(attn):
    """Views of a packed projection get as far as the device check; views
    without one token stride, dense channels or 16-byte heads are refused."""
    def call(t):
        d = dims(B=t.shape[0], T=t.shape[1], Hq=t.shape[2], Hkv=1)
        bt = (d.B, d.T)
        attn.gdn_qk_norm_rope(d, t, meta(*bt, 1, 64), None, None, None, meta(*bt, dtype=torch.int32), None,
                              meta(*bt, d.Hq, 64), meta(*bt, 1, 64))

    x = meta(2, 3, 12 * 64)
    for good in (x[..., 64:5 * 64].view(2, 3, 4, 64), x[..., :512].view(2, 3, 4, 128)[..., 64:],
                 meta(5, 7, 4, 64)[:, 2:3], meta(1, 1, 1, 64), meta(1, 3, 4, 64).expand(1, 3, 4, 64),
                 meta(2, 3, 1, 68)[..., :64].contiguous(), meta(1, 1, 1, 68)[..., :64]):
        with pytest.raises(ValueError, match="q must be a CUDA tensor"):
            call(good)
    for bad in (meta(2, 4, 4, 64)[:, :3], meta(2, 3, 64, 4).transpose(2, 3), meta(2, 3, 4, 66)[..., :64],
                meta(2, 3, 4, 128)[..., ::2], meta(3, 2, 4, 64).transpose(0, 1)):
        with pytest.raises(ValueError, match="stride"):
            call(bad)


def test_cache_handle_refusals(attn):
    e4, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    k = meta(4, 2, 16, 64)
    with pytest.raises(ValueError, match="one type"):
        attn.KVCache(k, meta(4, 2, 16, 32))
    with pytest.raises(TypeError, match="bfloat16 or float8_e4m3fn"):
        attn.KVCache(k.float(), k.float())
    with pytest.raises(ValueError, match="has no scales"):
        attn.KVCache(k, k, k, k)
    with pytest.raises(ValueError, match="needs k_scale"):
        attn.KVCache(k.to(e4), k.to(e4))
    with pytest.raises(ValueError, match="must be a CUDA tensor"):
        attn.KVCache(k, k)
    s = torch.zeros(4, 2, 16, dtype=torch.uint8)
    with pytest.raises((ValueError, TypeError)):
        attn.KVCache(k.to(e4), k.to(e4), s, s.view(e8))


# ---------------------------------------------------------------------------
# the frequency table
# ---------------------------------------------------------------------------
def test_rope_freqs_are_exact_fractions_of_a_turn(attn):
    inv = attn.rope_inv_freq(64, 1e7)
    assert inv[0] == 1.0 and inv.numel() == 32
    got = attn.rope_freqs(inv)
    assert got.dtype == torch.int64
    for f, bits in zip(inv.tolist(), got.tolist()):
        turns = Fraction(f) / (2 * Fraction(math.pi))
        # f / (2 pi) in f64: two roundings of 2^-53 relative (the division, and pi's own)
        assert abs(Fraction(bits % 2 ** 64, 2 ** 64) - turns) <= turns * Fraction(3, 2 ** 53) + Fraction(1, 2 ** 65)
    # whole turns drop out, a negative frequency turns back
    two = attn.rope_freqs(torch.tensor([math.pi, -math.pi / 2], dtype=torch.float64))
    assert [b % 2 ** 64 for b in two.tolist()] == [2 ** 63, 3 * 2 ** 62]


@pytest.mark.parametrize("pos", [0, 1, 12345, 1 << 20, (1 << 31) - 1, -7, -(1 << 31)])
def test_angle_product_mod_2_64(attn, pos):
    """The kernel's angle: the upper 32 bits of pos * freq mod 2^64, signed."""
    for f, bits in zip(attn.rope_inv_freq(32).tolist(), attn.rope_freqs(attn.rope_inv_freq(32)).tolist()):
        hi = (pos * (bits % 2 ** 64)) % 2 ** 64 >> 32
        x = (hi - 2 ** 32 if hi >= 2 ** 31 else hi) / 2.0 ** 31 * math.pi
        want = math.fmod(pos * f, 2 * math.pi)
        # f64 rounds pos * f to 2^-53 of up to 2^31; the angle is cut to 2^-32 turns
        tol = abs(pos * f) * 2.0 ** -51 + 2 * math.pi * 2.0 ** -32
        assert abs(math.sin(x) - math.sin(want)) <= tol and abs(math.cos(x) - math.cos(want)) <= tol


# ---------------------------------------------------------------------------
# the reference itself
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weighted", [False, True])
def test_reference_gradients_match_differences(inter, weighted):
    g = torch.Generator().manual_seed(3)
    B, T, H, D, rot = 1, 2, 2, 8, 4
    x, dy = (torch.randn((B, T, H, D), generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.rand(D, generator=g, dtype=torch.float64) + 0.5 if weighted else None
    pos = torch.tensor([[5, 900001]])
    inv = 10.0 ** -torch.arange(rot // 2, dtype=torch.float64)
    mask = torch.tensor([[1, 1]], dtype=torch.uint8)
    f = lambda x_, w_: float((R.norm_rope(x_, w_, pos, inv, inter, 1e-3, mask) * dy).sum())  # noqa: E731
    dx, dw, _ = R.norm_rope_bwd(x, w, dy, pos, inv, inter, 1e-3, mask)
    h = 1e-6
    for i in range(x.numel()):
        e = torch.zeros(x.numel(), dtype=torch.float64)
        e[i] = h
        e = e.view_as(x)
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - float(dx.flatten()[i])) < 1e-7
    if weighted:
        for i in range(D):
            e = torch.zeros(D, dtype=torch.float64)
            e[i] = h
            assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - float(dw[i])) < 1e-7


def test_reference_masked_steps_have_no_gradient():
    x = torch.randn((1, 3, 1, 8), dtype=torch.float64)
    mask = torch.tensor([[1, 0, 1]], dtype=torch.uint8)
    inv = torch.tensor([1.0], dtype=torch.float64)
    dx, dw, _ = R.norm_rope_bwd(x, torch.ones(8), torch.ones_like(x), torch.zeros(1, 3), inv, False, 0.0, mask)
    assert torch.all(dx[:, 1] == 0) and torch.isfinite(dw).all()
    assert torch.all(R.norm_rope(x, torch.ones(8), torch.zeros(1, 3), inv, False, 0.0, mask)[:, 1] == 0)


def test_reference_e4m3_rows():
    x = torch.tensor([[448.0, 1.0], [449.0, 1.0], [1.75, -0.3], [0.0, 0.0], [2.0 ** -140, 0.0], [1e30, -1e-5]],
                     dtype=torch.float64)
    codes, e = R.e4m3(x)
    assert e.tolist() == [0, 1, -8, -127, -127, 91]   # 1e30 <= 448 * 2^91 = 1.109e30
    # the codes are those of torch's own conversion of the exact quotient
    want = torch.ldexp(x, -e[:, None]).to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64)
    assert torch.equal(codes, want)
    assert torch.all((codes.abs() <= 448))


def test_reference_page_lookup():
    table = torch.tensor([[3, -1, 9]])
    assert R.lookup(table, 4, 16, 0, 15) == (3, 15)
    for p in (16, 31, 32, 47, 48, 1 << 40, -1):
        assert R.lookup(table, 4, 16, 0, p) is None
    k = torch.arange(4 * 1 * 16 * 2, dtype=torch.float64).view(4, 1, 16, 2)
    got, valid = R.gather(k, table, 16, 0, 20)
    assert torch.equal(got[:16, 0], k[3, 0]) and valid.tolist() == [True] * 16 + [False] * 4


def test_reference_decode_small_cases():
    """One key: its value; two equal keys: their mean; no key: zeros."""
    k = torch.zeros((2, 1, 16, 64), dtype=torch.float64)
    v = torch.randn((2, 1, 16, 64), dtype=torch.float64)
    q = torch.randn((3, 1, 2, 64), dtype=torch.float64)
    table = torch.tensor([[0], [1], [0]])
    out, lse, _, _ = R.decode(q, k, v, table, 16, [0, 1, 5], torch.tensor([1, 1, 0]), 1.0)
    assert torch.allclose(out[0, 0, 0], v[0, 0, 0]) and lse[0, 0, 0] == 0
    assert torch.allclose(out[1, 0, 1], (v[1, 0, 0] + v[1, 0, 1]) / 2) and abs(lse[1, 0, 1] - math.log(2)) < 1e-15
    assert torch.all(out[2] == 0) and torch.all(lse[2] == -math.inf)
