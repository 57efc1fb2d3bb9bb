"""Prompt attention, rotary axes and the verification of drafted tokens without
a GPU: refusals of the C ABI and of the binding, workspace sizes, and the
64-bit reference of the GPU tests against differences and exact cases."""
import ctypes
import math

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _prompt_ref as R

BF16, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


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


@pytest.fixture(scope="module")
def spec(lib):
    from gated_deltanet_linear_04_gb300 import spec as s
    return s


def dims(**kw):
    base = dict(B=2, T=3, Hq=4, Hkv=2, D=64)
    base.update(kw)
    return wl.AttnDims(**base)


BUF = ctypes.create_string_buffer(1 << 16)
P = (ctypes.addressof(BUF) + 255) // 256 * 256


def calls(lib, attn, d, q_rows=6, k_rows=8, q=(P, 256, 64), k=(P, 128, 64), v=(P, 128, 64), cu_q=None, cu_k=None, n_q=None,
          n_k=None, gate=(None, 0, 0), scale=0.125, ptr=P, lse=P, dgate=None, ws=P, ws_bytes=1 << 40):
    """(forward, backward) status.  Every call made here has to be refused (or
    be empty), so that nothing is launched: the addresses are host memory."""
    r = ctypes.byref(attn.make_attn_dims(d))
    head = (r, q_rows, k_rows, *q, *k, *v, cu_q, cu_k, n_q, n_k, *gate, scale)
    return (lib.gdn_attn_prefill(*head, ptr, lse, ws, ws_bytes, None),
            lib.gdn_attn_prefill_backward(*head, ptr, lse, ptr, ptr, ptr, ptr, dgate, ws, ws_bytes, None))


@pytest.mark.parametrize("kw,status", [
    ({"B": -1}, 1), ({"T": -1}, 1), ({"Hq": 0}, 1), ({"Hq": 5}, 1), ({"D": 0}, 1), ({"D": 96}, 2), ({"D": 512}, 2),
    ({"Hq": 34}, 2), ({"B": 65536}, 2), ({"Hq": 2048, "Hkv": 2048}, 2),
])
def test_bad_dims(lib, attn, kw, status):
    assert calls(lib, attn, dims(**kw)) == (status, status)
    assert attn.gdn_attn_prefill_workspace_size(dims(**kw), 6, 8) == 0
    assert attn.gdn_attn_prefill_backward_workspace_size(dims(**kw), 6, 8, True) == 0


@pytest.mark.parametrize("kw,status", [
    ({"q_rows": -2}, 1), ({"k_rows": -2}, 1), ({"q_rows": 1 << 31}, 2), ({"k_rows": 1 << 31}, 2),
    ({"q_rows": 7}, 1), ({"k_rows": 7}, 1),                       # no whole slots without offsets
    ({"q": (None, 256, 64)}, 1), ({"k": (None, 128, 64)}, 1), ({"v": (P + 8, 128, 64)}, 1), ({"q": (P, 252, 64)}, 1),
    ({"k": (P, -128, 64)}, 1), ({"q": (P, 0, 64)}, 2), ({"k": (P, 128, 0)}, 2), ({"v": (P, 1 << 39, 64)}, 2),
    ({"gate": (P, 0, 64)}, 2), ({"gate": (P + 2, 256, 64)}, 1),
    ({"cu_q": P + 2}, 1), ({"cu_k": P + 1}, 1), ({"n_q": P + 2}, 1), ({"n_k": P + 3}, 1),
    ({"scale": math.inf}, 1), ({"scale": math.nan}, 1), ({"ptr": None}, 1), ({"ptr": P + 2}, 1), ({"lse": P + 2}, 1),
    ({"ws": None}, 1), ({"ws": P + 8}, 1), ({"ws_bytes": 4096}, 1),
])
def test_refused_calls(lib, attn, kw, status):
    if "gate" in kw:
        kw = dict(kw, dgate=P)
    assert calls(lib, attn, dims(), **kw) == (status, status)


def test_gates_and_their_gradients_come_together(lib, attn):
    assert calls(lib, attn, dims(), dgate=P, ws_bytes=0) == (1, 1)
    assert calls(lib, attn, dims(), gate=(P, 256, 64), ws_bytes=0) == (1, 1)
    assert calls(lib, attn, dims(), lse=None, ws_bytes=0)[1] == 1


def test_empty_calls_are_noops(lib, attn):
    none = dict(q=(None, 0, 0), k=(None, 0, 0), v=(None, 0, 0), ptr=None, lse=None, ws=None, ws_bytes=0)
    assert calls(lib, attn, dims(B=0), q_rows=0, k_rows=0, **none) == (0, 0)
    assert calls(lib, attn, dims(), q_rows=0, k_rows=0, **none) == (0, 0)


def test_workspaces_grow_with_the_rows(lib, attn):
    d = dims(D=128, Hq=32, Hkv=8, B=7)
    f, b = attn.gdn_attn_prefill_workspace_size, attn.gdn_attn_prefill_backward_workspace_size
    assert 0 < f(d, 100, 100) <= f(d, 100000, 100) and 0 < b(d, 100, 100, False) < b(d, 100, 100, True)
    # dO of a gated call, and delta
    assert b(d, 4096, 64, True) - b(d, 4096, 64, False) == 4096 * 32 * 128 * 2
    assert b(d, 8192, 64, False) - b(d, 4096, 64, False) >= 4096 * 32 * 4


def test_status_string_of_bad_offsets(lib):
    from gated_deltanet_linear_04_gb300 import gdn
    assert gdn.status_string(gdn.GDN_ERR_BAD_OFFSETS).startswith("GDN_ERR_BAD_OFFSETS")


# ---------------------------------------------------------------------------
# the binding
# ---------------------------------------------------------------------------
def meta(*shape, dtype=BF16):
    return torch.zeros(shape, dtype=dtype)


def prompt_call(attn, d=None, **kw):
    a = dict(q=meta(2, 3, 4, 64), k=meta(2, 4, 2, 64), v=meta(2, 4, 2, 64))
    a.update(kw)
    attn.attn_prefill(d or dims(), **a)


PACKED = dict(q=meta(5, 4, 64), k=meta(7, 2, 64), v=meta(7, 2, 64))


@pytest.mark.parametrize("kw,error,text", [
    ({}, ValueError, "q must be a CUDA tensor"),
    (dict(PACKED, cu_q=meta(3, dtype=I32)), ValueError, "q must be a CUDA tensor"),
    ({"q": meta(2, 5, 4, 64)}, ValueError, "of the dims"),
    ({"q": meta(2, 3, 3, 64)}, ValueError, "q must have shape"),
    ({"q": meta(2, 3, 64)}, ValueError, "q must have shape"),
    ({"q": meta(2, 3, 4, 64, dtype=F32)}, TypeError, "q must be torch.bfloat16"),
    ({"v": meta(2, 5, 2, 64)}, ValueError, "same shape"),
    (PACKED, ValueError, "packed q needs cu_q"),
    ({"cu_q": meta(3, dtype=I32)}, ValueError, "cu_q goes with packed q"),
    ({"cu_k": meta(3, dtype=I32)}, ValueError, "cu_k goes with packed k"),
    (dict(k=PACKED["k"], v=PACKED["v"]), ValueError, "packed k needs cu_k"),
    (dict(PACKED, cu_q=meta(2, dtype=I32)), ValueError, "cu_q must have shape"),
    (dict(PACKED, cu_q=meta(3, dtype=torch.int64)), TypeError, "cu_q must be torch.int32"),
    ({"n_q": meta(3, dtype=I32)}, ValueError, "n_q must have shape"),
    ({"gate": meta(2, 3, 2, 64)}, ValueError, "gate must have shape"),
    ({"gate": meta(2, 4, 4, 64)}, ValueError, "gate must have q's shape"),
    (dict(PACKED, cu_q=meta(3, dtype=I32), gate=meta(4, 4, 64)), ValueError, "gate must have q's shape"),
    ({"q": meta(2, 3, 4, 128)[..., ::2]}, ValueError, "dense channels"),
    ({"q": meta(2, 6, 4, 64)[:, ::2][:, :3]}, ValueError, "q must be a CUDA tensor"),
    ({"q": meta(2, 4, 4, 64)[:, :3]}, ValueError, "one token stride"),
    (dict(PACKED, cu_q=meta(3, dtype=I32), q=meta(5, 4, 68)[..., :64]), ValueError, "multiples of 8"),
])
def test_binding_refuses(attn, kw, error, text):
    # (meta's tensors are on the CPU: whatever passes the other checks stops at the device)
    with pytest.raises(error, match=text):
        prompt_call(attn, **kw)


@pytest.mark.parametrize("kw,error,text", [
    ({"out": meta(2, 3, 4, 32)}, ValueError, "must have shape"), ({"lse": meta(2, 3, 4)}, TypeError, "float32"),
    ({"dout": meta(2, 3, 2, 64)}, ValueError, "must have shape"),
])
def test_backward_binding_refuses(attn, kw, error, text):
    a = dict(q=meta(2, 3, 4, 64), k=meta(2, 4, 2, 64), v=meta(2, 4, 2, 64), out=meta(2, 3, 4, 64), lse=meta(2, 3, 4, dtype=F32),
             dout=meta(2, 3, 4, 64))
    a.update(kw)
    with pytest.raises((error, ValueError), match=text + "|CUDA tensor"):
        attn.attn_prefill_backward(dims(), **a)


def test_outputs_must_be_given_to_the_abi_names(attn, spec):
    q, k = meta(2, 3, 4, 64), meta(2, 4, 2, 64)
    with pytest.raises(TypeError, match="out must be"):
        attn.gdn_attn_prefill(dims(), q, k, k, None, None, None, None, None, 1.0, None, None, meta(16, dtype=U8))
    with pytest.raises(TypeError, match="keep must be"):
        spec.gdn_spec_verify(meta(1, 2, 8, dtype=F32), None, meta(1, 1, dtype=I32), meta(1, 2, dtype=F32), None,
                             meta(1, 2, dtype=I32), None)


# ---------------------------------------------------------------------------
# axes
# ---------------------------------------------------------------------------
def test_rope_axes(attn):
    assert attn.rope_axes([2, 1, 3]).tolist() == [0, 0, 1, 2, 2, 2]
    assert attn.rope_axes([2, 1, 3], cyclic=True).tolist() == [0, 1, 2, 0, 2, 2]
    assert attn.rope_axes([4]).dtype == U8 and attn.rope_axes([0, 2]).tolist() == [1, 1]
    for bad in ([], [1, -1], [1] * 9):
        with pytest.raises(ValueError, match="rope_axes"):
            attn.rope_axes(bad)


@pytest.mark.parametrize("kw,status", [({"n_axes": 0}, 1), ({"n_axes": 9}, 1), ({"axes": None}, 1), ({"pos": None}, 1),
                                       ({"pos": P + 2}, 1), ({"freqs": None}, 1)])
def test_axes_refusals(lib, attn, kw, status):
    a = dict(axes=P, n_axes=3, pos=P, freqs=P)
    a.update(kw)
    d = dims(Drot=32)
    r = ctypes.byref(attn.make_attn_dims(d))
    heads = (P, 256, 64)
    c = ctypes.byref(attn.GdnKvCache(k=P, v=P, k_scale=None, v_scale=None, n_pages=4, page_size=16, format=0))
    ax = (a["freqs"], a["axes"], a["n_axes"], a["pos"])
    assert lib.gdn_qk_norm_rope_axes(r, *heads, *heads, P, P, *ax, None, P, P, None) == status
    assert lib.gdn_qk_norm_rope_axes_backward(r, *heads, *heads, P, P, *ax, None, P, P, P, P, P, P, P, 1 << 30, None) == status
    assert lib.gdn_kv_append_axes(r, *heads, *heads, *heads, P, P, *ax, c, P, 2, P, None, P, None) == status


def test_axes_binding_refusals(attn):
    d = dims(Drot=32)
    q, k, w = meta(2, 3, 4, 64), meta(2, 3, 2, 64), meta(64, dtype=F32)
    fr = meta(16, dtype=torch.int64)
    for axes, pos, error, text in ((meta(16, dtype=U8), meta(2, 3, dtype=I32), ValueError, "1 to 8 axes"),
                                   (meta(16, dtype=U8), meta(9, 2, 3, dtype=I32), ValueError, "1 to 8 axes"),
                                   (meta(15, dtype=U8), meta(3, 2, 3, dtype=I32), ValueError, "axes must have shape"),
                                   (meta(16, dtype=I32), meta(3, 2, 3, dtype=I32), TypeError, "axes must be torch.uint8"),
                                   (meta(16, dtype=U8), meta(3, 2, 4, dtype=I32), ValueError, "pos must have shape"),
                                   (meta(16, dtype=U8), meta(3, 2, 3, dtype=I32), ValueError, "axes must be a CUDA tensor")):
        with pytest.raises(error, match=text):
            attn.qk_norm_rope_axes(d, q, k, w, w, fr, axes, pos)


# ---------------------------------------------------------------------------
# drafted tokens
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("args,status", [
    ((-1, 2, 8), 1), ((1, -1, 8), 1), ((1, 2, 0), 1), ((1, 1024, 8), 2), ((1, 2, (1 << 24) + 1), 2),
])
def test_verify_sizes(lib, args, status):
    assert lib.gdn_spec_verify(*args, P, P, P, P, None, P, P, None) == status


def test_verify_pointers(lib):
    f = lib.gdn_spec_verify
    base = [P, P, P, P, P, P, P]
    for i in (0, 2, 3, 5, 6):
        bad = list(base)
        bad[i] = None
        assert f(1, 2, 8, *bad, None) == 1
    for i in range(7):
        bad = list(base)
        bad[i] = P + 2
        assert f(1, 2, 8, *bad, None) == 1
    assert f(0, 2, 8, None, None, None, None, None, None, None, None) == 0


def test_verify_binding_refusals(spec):
    t, k, u = meta(2, 4, 8, dtype=F32), meta(2, 3, dtype=I32), meta(2, 4, dtype=F32)
    for kw, error, text in (({"target": meta(2, 8, dtype=F32)}, ValueError, "target must have shape"),
                            ({"target": t.to(BF16)}, TypeError, "float32"),
                            ({"tokens": meta(2, 4, dtype=I32)}, ValueError, "tokens must have shape"),
                            ({"tokens": k.long()}, TypeError, "int32"), ({"u": meta(2, 3, dtype=F32)}, ValueError, "u must"),
                            ({"draft": t}, ValueError, "draft must have shape"),
                            ({"n": meta(3, dtype=I32)}, ValueError, "n must have shape"),
                            ({}, ValueError, "target must be a CUDA tensor")):
        a = dict(target=t, tokens=k, u=u)
        a.update(kw)
        with pytest.raises(error, match=text):
            spec.verify(**a)


# ---------------------------------------------------------------------------
# the reference itself
# ---------------------------------------------------------------------------
def test_reference_gradients_match_differences():
    g = torch.Generator().manual_seed(3)
    q, dout, gate = (torch.randn((5, 4, 8), generator=g, dtype=torch.float64) for _ in range(3))
    k, v = (torch.randn((7, 2, 8), generator=g, dtype=torch.float64) for _ in range(2))
    qs = R.sequences(2, 5, torch.tensor([0, 3, 5]), torch.tensor([2, 2]))
    ks = R.sequences(2, 7, torch.tensor([1, 5, 7]), torch.tensor([4, 1]))     # the second: its first query sees nothing
    got = R.prefill_backward(q, k, v, dout, qs, ks, 0.3, gate)

    def f():
        o = R.prefill(q, k, v, qs, ks, 0.3, gate)[0]
        return float(torch.nansum(o * dout))

    h = 1e-6
    for name, x in (("dq", q), ("dk", k), ("dv", v), ("dgate", gate)):
        want = torch.zeros_like(x).view(-1)
        for i in range(x.numel()):
            y = x.view(-1)
            old = float(y[i])
            y[i] = old + h
            a = f()
            y[i] = old - h
            want[i] = (a - f()) / (2 * h)
            y[i] = old
        assert torch.allclose(torch.nan_to_num(got[name][0]).view(-1), want, atol=1e-7), name


def test_reference_sees_its_own_end():
    assert R.seen(2, 4, "cpu").tolist() == [[True, True, True, False], [True] * 4]
    assert R.seen(3, 1, "cpu").tolist() == [[False], [False], [True]]
    v = torch.randn(4, 1, 8, dtype=torch.float64)
    out, lse, _, _ = R.prefill(torch.zeros(3, 1, 8), torch.zeros(4, 1, 8), v, [(0, 3, 3)], [(0, 1, 1)], 1.0)
    assert torch.all(out[:2] == 0) and torch.all(lse[:2] == -math.inf)
    assert torch.allclose(out[2, 0], v[0, 0]) and lse[2, 0] == 0


def test_reference_verification():
    t = torch.tensor([[[0.5, 0.25, 0.25], [0.0, 1.0, 0.0], [0.25, 0.25, 0.5]]])
    d = torch.tensor([[[0.25, 0.5, 0.25], [0.0, 1.0, 0.0]]])
    tok = torch.tensor([[1, 1]])
    # 0.6 * 0.5 >= 0.25: falls; what the target has above the draft is token 0
    assert R.verify(t, tok, torch.tensor([[0.6, 0.0, 0.9]]), d)[0].tolist() == [[0, -1, -1]]
    out, keep = R.verify(t, tok, torch.tensor([[0.4, 0.9, 0.5]]), d)
    assert out.tolist() == [[1, 1, 2]] and keep.tolist() == [3]
    # certain drafts: without the fallen token
    assert R.verify(t, tok, torch.tensor([[0.3, 0.0, 0.7]]))[0].tolist() == [[2, -1, -1]]
    # none drafted
    assert R.verify(t, tok, torch.tensor([[0.3, 0.0, 0.6]]), d, torch.tensor([0]))[0].tolist() == [[1, -1, -1]]
