"""The attention layer's operators one after the other, as a training step uses
them (examples/hybrid_decode.py): its gradients against the 64-bit formulas, with
each operator's bound carried through the next."""
import importlib.util
import os

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _prompt_ref as R
from tests import _attn_ref as A
from tests.test_gpu_attn import attn, status  # noqa: F401
from tests.test_gpu_axes import turned

pytestmark = pytest.mark.gpu

BF16, F64, I32 = torch.bfloat16, torch.float64, torch.int32
DEV = "cuda:0"
HALF = 2.0 ** -8                                       # half a step of bf16
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example(attn):  # noqa: F811
    spec = importlib.util.spec_from_file_location("hybrid_decode", os.path.join(ROOT, "examples", "hybrid_decode.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def inside(got, want, tol, what):
    bad = ~((got.to(F64) - want).abs() <= tol)
    assert not bad.any(), "%s: %d off, worst %.3e of %.3e" % (
        what, int(bad.sum()), float((got.to(F64) - want).abs()[bad].max()), float(tol.expand_as(want)[bad].max()))


@pytest.mark.parametrize("B,T,Hq,Hkv,D,rot", [(1, 64, 16, 2, 256, 64), (2, 201, 9, 3, 128, 128), (3, 77, 4, 4, 64, 32)])
def test_a_training_step(attn, example, B, T, Hq, Hkv, D, rot):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(T)
    d = wl.AttnDims(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D, Drot=rot)
    normal = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    qkv, gate, dout = (normal(B, T, n).to(BF16) for n in ((Hq + 2 * Hkv) * D, Hq * D, Hq * D))
    gate, dout = gate.view(B, T, Hq, D), dout.view(B, T, Hq, D)
    wq, wk = (torch.rand(D, generator=g, device=DEV) + 0.5 for _ in range(2))
    inv = attn.rope_inv_freq(rot)
    axes = attn.rope_axes([rot // 2 - 2 * (rot // 8), rot // 8, rot // 8], True, DEV)
    pos = example.image_positions(d, 5, 7, DEV)
    out, got = example.training_step(d, qkv, gate, dout, wq, wk, attn.rope_freqs(inv, DEV), axes, pos)
    assert status() == 0

    # the attention's gradients at the turned q and k, whose own bounds R knows
    q, k, v = example.split(d, qkv)
    qr, kr = attn.qk_norm_rope_axes(d, q, k, wq, wk, attn.rope_freqs(inv, DEV), axes, pos)
    flat = lambda x: x.reshape(-1, *x.shape[-2:])  # noqa: E731
    qs = R.sequences(B, B * T, None, None)
    want = R.prefill_backward(flat(qr), flat(kr), flat(v), flat(dout), qs, qs, D ** -0.5, flat(gate))
    for n in ("dv", "dgate"):
        inside(flat(got[n]), *want[n], n)
    # through the rotation and the norm: z = turned back, dx = r (w z - xh mean(xh w z)), dw = sum of xh z
    inv = inv.to(DEV)
    for n, x, w in (("q", q, wq), ("k", k, wk)):
        x, w = x.to(F64), w.to(F64)
        dy, tol = (y.view(B, T, -1, D) for y in want["d" + n])
        z = turned(None, dy, None, pos, axes, inv, False, None, -1.0, normed=False)
        ztol = tol.clone()
        half = rot // 2
        ztol[..., :half] = ztol[..., half:rot] = tol[..., :half] + tol[..., half:rot]
        r = (x.square().mean(-1, keepdim=True) + d.eps).rsqrt()
        xh = x * r
        dx = r * (w * z - xh * (xh * w * z).mean(-1, keepdim=True))
        dtol = r * (w * ztol + xh.abs() * (xh.abs() * w * ztol).mean(-1, keepdim=True))
        # its own: a rounding to bf16, and f32 arithmetic as in tests/test_gpu_axes.py
        noise = 2.0 ** -19 * r * ((w * z).abs().amax(-1, keepdim=True) * (1 + xh.abs() * xh.abs().amax(-1, keepdim=True)))
        inside(got["d" + n], dx, dtol + HALF * (dx.abs() + dtol) + noise, "d" + n)
        inside(got["dw" + n], (xh * z).sum((0, 1, 2)), (xh.abs() * (ztol + 2.0 ** -19 * z.abs())).sum((0, 1, 2)) + 1e-12, "dw" + n)


def test_the_example_takes_other_sizes(example):
    # one bf16 rounding of the result (2^-8), and of the weights before the product with V
    assert example.main(rows=3, prompt=700, steps=2) <= 2.0 ** -7
