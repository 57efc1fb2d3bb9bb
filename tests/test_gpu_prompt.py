"""A prompt's attention and its gradients on the GPU against their 64-bit
definitions (tests/_prompt_ref.py)."""
import math

import pytest
import torch

from gated_deltanet_linear_04_gb300 import workloads as wl
from tests import _prompt_ref as R
from tests.test_gpu_attn import attn, status  # noqa: F401

pytestmark = pytest.mark.gpu

BF16, F32, F64, I32 = torch.bfloat16, torch.float32, torch.float64, torch.int32
DEV = "cuda:0"


class Case:
    """Sequences of nq[s] queries and nk[s] keys: packed with `gap` rows in no
    slot before, between (as padding of the slots) and behind, or rows of a
    padded batch; q, k, v, gate as views of wider tensors."""

    def __init__(self, Hq, Hkv, D, nq, nk, packed, gated, seed=0, scale=None, gap=0, std=1.0):
        g = torch.Generator(device=DEV).manual_seed(seed)
        B = len(nq)
        self.scale = D ** -0.5 if scale is None else scale
        self.kw = {}
        if packed:
            def offsets(n):
                at = [gap]
                for x in n:
                    at.append(at[-1] + x + gap)
                return torch.tensor(at, dtype=I32)
            cu = [offsets(nq), offsets(nk)]
            rows, krows = (int(cu[0][-1]) + gap,), (int(cu[1][-1]) + gap,)
            self.kw.update(cu_q=cu[0].to(DEV), cu_k=cu[1].to(DEV))
            if gap:
                self.kw.update(n_q=torch.tensor(nq, dtype=I32, device=DEV), n_k=torch.tensor(nk, dtype=I32, device=DEV))
            T = 0
        else:
            T, Tk = max(nq), max(max(nk), 1)
            cu = [None, None]
            rows, krows = (B, T), (B, Tk)
            self.kw.update(n_q=torch.tensor(nq, dtype=I32, device=DEV), n_k=torch.tensor(nk, dtype=I32, device=DEV))
        self.d = wl.AttnDims(B=B, T=T, Hq=Hq, Hkv=Hkv, D=D)
        self.rows, self.krows = math.prod(rows), math.prod(krows)

        def heads(shape, H, wide, s):
            x = torch.randn(*shape, H * wide * D + 8, generator=g, device=DEV).mul_(s).to(BF16)
            return x[..., : H * wide * D].view(*shape, H, wide * D)[..., (wide - 1) * D:]
        self.q, self.k, self.v = heads(rows, Hq, 2, 1.5 * std), heads(krows, Hkv, 1, std), heads(krows, Hkv, 1, 1.0)
        self.dout = torch.randn(*rows, Hq, D, generator=g, device=DEV).mul_(0.3).to(BF16)
        if gated:
            self.kw["gate"] = heads(rows, Hq, 2, 1.5)
        self.qs = R.sequences(B, self.rows, cu[0], nq)
        self.ks = R.sequences(B, self.krows, cu[1], nk)

    def flat(self, x):
        return x.reshape(-1, *x.shape[-2:])

    def fwd(self, a, **kw):
        return a.attn_prefill(self.d, self.q, self.k, self.v, scale=self.scale, return_lse=True, **self.kw, **kw)

    def bwd(self, a, out, lse, **kw):
        return a.attn_prefill_backward(self.d, self.q, self.k, self.v, out, lse, self.dout, scale=self.scale, **self.kw, **kw)

    def want_fwd(self):
        g = self.kw.get("gate")
        return R.prefill(self.flat(self.q), self.flat(self.k), self.flat(self.v), self.qs, self.ks, self.scale,
                         None if g is None else self.flat(g))

    def want_bwd(self):
        g = self.kw.get("gate")
        return R.prefill_backward(self.flat(self.q), self.flat(self.k), self.flat(self.v), self.flat(self.dout), self.qs,
                                  self.ks, self.scale, None if g is None else self.flat(g))


def near(got, want, tol, what):
    got = got.to(F64)
    mine = ~torch.isnan(want)
    same = got == want                                   # (infinities)
    bad = mine & ~same & ~((got - want).abs() <= tol)
    assert not bad.any(), "%s: %d of %d off, worst %.3e of a bound of %.3e" % (
        what, int(bad.sum()), int(mine.sum()), float((got - want).abs()[bad].max()), float(tol[bad].max()))


# Hq, Hkv, D, queries, keys (None: as many), packed, gated
CASES = [
    (1, 1, 64, [1], None, False, False),
    (1, 1, 256, [1], None, False, True),
    (2, 1, 128, [2], [300], False, False),
    (16, 2, 256, [300], None, False, True),
    (16, 2, 256, [130, 5, 0, 77], [230, 105, 50, 1077], False, True),
    (9, 3, 64, [77], None, False, False),
    (32, 8, 128, [100, 700, 3, 0, 513], None, True, False),
    (12, 1, 128, [100, 300, 3, 0, 513], [103, 300, 4, 2, 1213], True, True),
    (13, 1, 256, [40, 600], [43, 600], True, True),
    (16, 1, 64, [5] * 40, [5 + 7 * i for i in range(40)], True, True),
    (8, 8, 256, [900, 1], None, True, False),
    (8, 8, 64, [128, 129, 127], None, True, True),
    (11, 1, 128, [64, 65, 63, 1], None, False, False),
    (16, 2, 256, [3, 200, 64], [1, 0, 63], True, False),          # queries before the first key see nothing
    (4, 4, 128, [257], [1300], False, True),
    (24, 4, 128, [1000], None, False, False),
    (1024, 1024, 64, [2, 3], None, True, False),
]


def make(case, **kw):
    Hq, Hkv, D, nq, nk, packed, gated = case
    return Case(Hq, Hkv, D, nq, nq if nk is None else nk, packed, gated, seed=sum(nq) + Hq, **kw)


@pytest.mark.parametrize("case", CASES)
def test_prefill(attn, case):  # noqa: F811
    c = make(case)
    out, lse = c.fwd(attn)
    want, wlse, tol, ltol = c.want_fwd()
    near(c.flat(out), want, tol, "out")
    near(lse.reshape(wlse.shape), wlse, ltol, "lse")


@pytest.mark.parametrize("case", CASES)
def test_prefill_backward(attn, case):  # noqa: F811
    c = make(case)
    out, lse = c.fwd(attn)
    got = c.bwd(attn, out, lse)
    want = c.want_bwd()
    assert set(got) == set(want)
    for n, (w, tol) in want.items():
        near(c.flat(got[n]), w, tol, n)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_slots_with_padding_and_rows_in_no_slot(attn, D):  # noqa: F811
    """Padding gives zeros; rows in no slot stay as they were."""
    c = Case(6, 2, D, [40, 0, 133], [50, 20, 133], True, True, gap=9)
    poison = [torch.full_like(x, 7.0) for x in (torch.empty(c.rows, 6, D, device=DEV, dtype=BF16),) * 3]
    out, dq, dgate = poison
    lse = torch.full((c.rows, 6), 7.0, device=DEV)
    dk, dv = (torch.full((c.krows, 2, D), 7.0, device=DEV, dtype=BF16) for _ in range(2))
    ws = torch.empty(attn.gdn_attn_prefill_workspace_size(c.d, c.rows, c.krows), dtype=torch.uint8, device=DEV)
    seqs = [c.kw[n] for n in ("cu_q", "cu_k", "n_q", "n_k", "gate")]
    attn.gdn_attn_prefill(c.d, c.q, c.k, c.v, *seqs, c.scale, out, lse, ws)
    ws = torch.empty(attn.gdn_attn_prefill_backward_workspace_size(c.d, c.rows, c.krows, True), dtype=torch.uint8, device=DEV)
    attn.gdn_attn_prefill_backward(c.d, c.q, c.k, c.v, *seqs, c.scale, out, lse, c.dout, dq, dk, dv, dgate, ws)
    assert status() == 0
    want, wlse, tol, ltol = c.want_fwd()
    near(out, want, tol, "out")
    near(lse, wlse, ltol, "lse")
    for n, x in (("dq", dq), ("dk", dk), ("dv", dv), ("dgate", dgate)):
        near(x, *c.want_bwd()[n], n)
    for x, qs in ((out, c.qs), (lse, c.qs), (dq, c.qs), (dgate, c.qs), (dk, c.ks), (dv, c.ks)):
        mine = torch.zeros(x.shape[0], dtype=torch.bool)
        for a, slot, n in qs:
            mine[a:a + slot] = True
            assert slot == n or not (x[a + n:a + slot] != (-math.inf if x is lse else 0)).any()
        assert (x[~mine.to(DEV)] == 7.0).all() and not mine.all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_what_is_not_seen_does_not_matter(attn, D, bad):  # noqa: F811
    """Keys, values, queries, gates and gradients behind a sequence's end, in
    padding and in no slot; a last token that only its own query sees."""
    c = Case(6, 2, D, [40, 3, 150], [70, 3, 150], True, True, gap=5)
    gate = c.kw["gate"]
    for x, seqs in ((c.q, c.qs), (gate, c.qs), (c.dout, c.qs), (c.k, c.ks), (c.v, c.ks)):
        mine = torch.zeros(x.shape[0], dtype=torch.bool, device=DEV)
        for a, _, n in seqs:
            mine[a:a + n] = True
        x[~mine] = bad
    out2, lse2 = c.fwd(attn)
    grads2 = c.bwd(attn, out2, lse2)
    want, wlse, tol, ltol = c.want_fwd()
    near(out2, want, tol, "out")
    near(lse2, wlse, ltol, "lse")
    before = c.want_bwd()
    for n, (w, t) in before.items():
        near(grads2[n], w, t, n)
    # the last key and value of the last sequence: every query but the last is as before
    a, _, n = c.ks[2]
    last = c.qs[2][0] + c.qs[2][2] - 1
    c.k[a + n - 1] = bad
    c.v[a + n - 1] = bad
    out3, lse3 = c.fwd(attn)
    grads3 = c.bwd(attn, out3, lse3)
    for s, (q0, _, nq) in enumerate(c.qs):
        rows = slice(q0, q0 + nq - (s == 2))
        near(out3[rows], want[rows], tol[rows], "out")
        near(lse3[rows], wlse[rows], ltol[rows], "lse")
        near(grads3["dq"][rows], before["dq"][0][rows], before["dq"][1][rows], "dq")
    # that query itself: its score there is NaN, +inf or -inf
    if bad != bad:
        assert torch.isnan(out3[last]).all() and torch.isnan(lse3[last]).all()
    # keys that it alone makes not finite are those that it sees, but none of another sequence
    for n in ("dk", "dv"):
        for a, _, m in c.ks[:2]:
            near(grads3[n][a:a + m], before[n][0][a:a + m], before[n][1][a:a + m], n)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_values_that_are_seen_come_through(attn, D):  # noqa: F811
    """A NaN key makes the queries that see it NaN, a NaN value its channel; a
    query whose scores are all -inf gives NaN and lse -inf."""
    c = Case(2, 2, D, [200], [200], False, False)
    c.v[0, 150, 0, 3] = math.nan
    c.v[0, 100, 0, 5] = math.inf
    out, lse = c.fwd(attn)
    assert torch.isfinite(lse).all()
    o = out[0].float()
    assert torch.isnan(o[150:, 0, 3]).all() and torch.isfinite(o[:150, 0, 3]).all()
    assert (o[100:, 0, 5] == math.inf).all() and torch.isfinite(o[:100, 0, 5]).all()
    assert torch.isfinite(o[:, 1]).all() and torch.isfinite(o[:, 0, 6:]).all()
    c = Case(2, 2, D, [200], [200], False, False)
    c.k[0, 130, 1, 0] = math.nan
    out, lse = c.fwd(attn)
    assert torch.isnan(out[0, 130:, 1]).all() and torch.isnan(lse[0, 130:, 1]).all()
    assert torch.isfinite(out[0, :130]).all() and torch.isfinite(out[0, :, 0]).all() and torch.isfinite(lse[0, :130]).all()
    c = Case(2, 2, D, [90], [90], False, False)
    c.q[0, :, 0] = 0
    c.q[0, :, 0, 0] = 1
    c.k[0, :, 0, 0] = -math.inf
    out, lse = c.fwd(attn)
    assert torch.isnan(out[0, :, 0]).all() and (lse[0, :, 0] == -math.inf).all() and torch.isfinite(out[0, :, 1]).all()
    c.k[0, 40, 0, 0] = 0.5                             # from here on one key counts
    out, lse = c.fwd(attn)
    assert torch.isnan(out[0, :40, 0]).all() and torch.allclose(lse[0, 40:, 0], torch.tensor(0.5 * c.scale, device=DEV))
    assert torch.equal(out[0, 40:, 0], c.v[0, 40, 0].expand(50, D))


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("scale,std", [(-0.07, 1.0), (0.0, 1.0), (0.5, 4.0), (1e-3, 1.0)])
def test_scales(attn, D, scale, std):  # noqa: F811
    """Negative and zero scales, and scores of some hundred whose maximum moves
    from step to step (the accumulators are rescaled)."""
    c = Case(4, 2, D, [70, 300], [70, 900], True, False, scale=scale, std=std)
    ramp = torch.linspace(0.1, 2.0, c.krows, device=DEV)[:, None, None]
    c.k.copy_((c.k.float() * ramp).to(BF16))
    out, lse = c.fwd(attn)
    want, wlse, tol, ltol = c.want_fwd()
    near(out, want, tol, "out")
    near(lse, wlse, ltol, "lse")
    for n, (w, t) in c.want_bwd().items():
        near(c.bwd(attn, out, lse)[n], w, t, n)


@pytest.mark.parametrize("D", [64, 256])
@pytest.mark.parametrize("which", ["q", "k", "v", "dout"])
def test_inputs_that_are_all_nan(attn, D, which):  # noqa: F811
    """NaN where the formulas give NaN, and numbers elsewhere."""
    c = make((8, 2, D, [700, 3], [700, 40], True, False))
    out, lse = attn.attn_prefill(c.d, c.q, c.k, c.v, return_lse=True, **c.kw)
    x = {"q": c.q, "k": c.k, "v": c.v, "dout": c.dout}
    x[which].fill_(math.nan)
    if which != "dout":
        out, lse = attn.attn_prefill(c.d, c.q, c.k, c.v, return_lse=True, **c.kw)
        assert out.isnan().all() and (lse.isnan().all() if which != "v" else lse.isfinite().all())
    got = attn.attn_prefill_backward(c.d, c.q, c.k, c.v, out, lse, c.dout, **c.kw)
    # dV = P^T dO; dQ and dK take the values through dP and delta
    finite = {"q": (), "k": (), "v": ("dv",), "dout": ()}[which]
    for name, g in got.items():
        assert (g.isfinite() if name in finite else g.isnan()).all(), name


def test_gradients_match_differences(attn):  # noqa: F811
    """Of a sum of outputs, along random directions: the forward pass itself,
    in 64 bits of the definition, at points a step away."""
    c = Case(4, 2, 64, [60, 33], [80, 33], True, True)
    out, lse = c.fwd(attn)
    got = c.bwd(attn, out, lse)
    g = torch.Generator(device=DEV).manual_seed(5)
    want = c.want_bwd()
    for name, x in (("dq", c.q), ("dk", c.k), ("dv", c.v), ("dgate", c.kw["gate"])):
        step = torch.randn(x.shape, generator=g, device=DEV, dtype=F64)
        base, h = x.to(F64), 1e-4

        def f(t):
            args = {"dq": c.q, "dk": c.k, "dv": c.v, "dgate": c.kw["gate"], name: base + t * step}
            o = R.prefill(args["dq"], args["dk"], args["dv"], c.qs, c.ks, c.scale, args["dgate"])[0]
            return float(torch.nansum(o * c.dout.to(F64)))

        diff = (f(h) - f(-h)) / (2 * h)
        along = float((got[name].to(F64) * step).sum())
        # (the bounds of all elements, and the differences' own h^2)
        assert abs(along - diff) <= float((want[name][1] * step.abs()).sum()) + 1e-4 * abs(diff) + 1e-4


def test_equal_calls_give_equal_bits(attn):  # noqa: F811
    for D in (64, 128, 256):
        c = Case(8, 2, D, [700, 90, 1], [800, 90, 40], True, True)
        out, lse = c.fwd(attn)
        grads = c.bwd(attn, out, lse)
        for _ in range(3):
            o, l = c.fwd(attn)
            assert torch.equal(o, out) and torch.equal(l, lse)
            for n, x in c.bwd(attn, out, lse).items():
                assert torch.equal(x, grads[n]), n


@pytest.mark.parametrize("cu", [[0, 50, 40, 60], [-1, 20, 40, 60], [0, 20, 40, 61], [0, 0, 100, 60]])
def test_bad_offsets_are_reported_and_nothing_is_written(attn, cu):  # noqa: F811
    from gated_deltanet_linear_04_gb300 import gdn
    d = wl.AttnDims(B=3, T=0, Hq=4, Hkv=2, D=128)
    q, k = torch.randn(60, 4, 128, device=DEV).to(BF16), torch.randn(60, 2, 128, device=DEV).to(BF16)
    off = torch.tensor(cu, dtype=I32, device=DEV)
    out, lse = torch.full_like(q, 3.0), torch.full((60, 4), 3.0, device=DEV)
    ws = torch.empty(attn.gdn_attn_prefill_workspace_size(d, 60, 60), dtype=torch.uint8, device=DEV)
    attn.gdn_attn_prefill(d, q, k, k, off, off, None, None, None, 0.1, out, lse, ws)
    assert status() == gdn.GDN_ERR_BAD_OFFSETS
    assert (out == 3.0).all() and (lse == 3.0).all()
    good = torch.tensor([0, 20, 40, 60], dtype=I32, device=DEV)
    dq, dk, dv = torch.full_like(q, 3.0), torch.full_like(k, 3.0), torch.full_like(k, 3.0)
    ws = torch.empty(attn.gdn_attn_prefill_backward_workspace_size(d, 60, 60, False), dtype=torch.uint8, device=DEV)
    attn.gdn_attn_prefill_backward(d, q, k, k, good, off, None, None, None, 0.1, out, lse, q, dq, dk, dv, None, ws)
    assert status() == gdn.GDN_ERR_BAD_OFFSETS
    assert (dq == 3.0).all() and (dk == 3.0).all() and (dv == 3.0).all()


def test_lengths_are_clamped_to_their_slots(attn):  # noqa: F811
    c = Case(4, 2, 64, [30, 20], [30, 20], False, False)
    a = c.fwd(attn)
    c.kw["n_q"] = torch.tensor([1000, 20], dtype=I32, device=DEV)
    c.kw["n_k"] = torch.tensor([2 ** 31 - 1, 20], dtype=I32, device=DEV)
    b = c.fwd(attn)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    c.kw["n_q"] = torch.tensor([-5, -2 ** 31], dtype=I32, device=DEV)
    out, lse = c.fwd(attn)
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("heads", [(16, 2), (16, 16), (10, 2)])
def test_many_tiles_of_many_steps_each(attn, D, heads):  # noqa: F811
    """Every CTA goes through several tiles, of queries and of keys."""
    c = make((*heads, D, [700, 1300, 257, 600], [900, 1300, 300, 600], True, True))
    out, lse = c.fwd(attn)
    want, wlse, tol, ltol = c.want_fwd()
    near(out, want, tol, "out")
    near(lse, wlse, ltol, "lse")
    got = c.bwd(attn, out, lse)
    for n, (w, t) in c.want_bwd().items():
        near(got[n], w, t, n)
    assert status() == 0


def test_empty_sides(attn):  # noqa: F811
    d = wl.AttnDims(B=2, T=5, Hq=4, Hkv=2, D=128)
    q, none = torch.randn(2, 5, 4, 128, device=DEV).to(BF16), torch.empty(2, 0, 2, 128, device=DEV, dtype=BF16)
    out, lse = attn.attn_prefill(d, q, none, none, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    g = attn.attn_prefill_backward(d, q, none, none, out, lse, q)
    assert (g["dq"] == 0).all() and g["dk"].shape == (2, 0, 2, 128)
    e, k = q[:, :0], torch.randn(2, 7, 2, 128, device=DEV).to(BF16)
    out, lse = attn.attn_prefill(d.with_(T=0), e, k, k, return_lse=True)
    assert out.shape == (2, 0, 4, 128) and lse.shape == (2, 0, 4)
    g = attn.attn_prefill_backward(d.with_(T=0), e, k, k, out, lse, e)
    assert (g["dk"] == 0).all() and (g["dv"] == 0).all() and g["dq"].numel() == 0
    b0 = attn.attn_prefill(d.with_(B=0), q[:0], none[:0], none[:0])
    assert b0.shape == (0, 5, 4, 128)


def test_long_strides_pass_32_bits(attn):  # noqa: F811
    """Token offsets above 2^31 elements."""
    n, stride = 300, 1 << 23
    base = torch.empty(n * stride // 2, dtype=F32, device=DEV)          # 5 GB
    wide = base.view(BF16).view(n, stride)
    c = Case(2, 2, 128, [n], [n], True, False)
    v = wide[:, 1 << 20:(1 << 20) + 256].view(n, 2, 128)
    v.copy_(c.v)
    want = c.fwd(attn)
    grads = c.bwd(attn, *want)
    c.v = v
    got = c.fwd(attn)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for k, x in c.bwd(attn, *want).items():
        assert torch.equal(x, grads[k])


def test_many_short_sequences(attn):  # noqa: F811
    """More sequences and units than the list's cache holds."""
    n = [(7 * i) % 4 for i in range(5000)]
    c = Case(1, 1, 64, n, n, True, False)
    out, lse = c.fwd(attn)
    grads = c.bwd(attn, out, lse)
    # sequences of one token: its value; of two and three by the definition, all at once
    cu = c.kw["cu_q"].long()
    at = torch.nonzero(torch.tensor(n, device=DEV) == 1)[:, 0]
    assert torch.equal(out[cu[at]], c.v[cu[at]])
    for m in (2, 3):
        s = cu[torch.nonzero(torch.tensor(n, device=DEV) == m)[:, 0]][:, None] + torch.arange(m, device=DEV)
        q, k, v = (x[s][:, :, 0].to(F64) for x in (c.q, c.k, c.v))
        z = (q @ k.transpose(1, 2) * c.scale).masked_fill(~R.seen(m, m, DEV), -math.inf)
        p = torch.softmax(z, -1)
        assert (out[s][:, :, 0].to(F64) - p @ v).abs().max() <= 2.0 ** -7 * v.abs().max()
        assert (lse[s][:, :, 0].to(F64) - torch.logsumexp(z, -1)).abs().max() <= 1e-5
        do = c.dout[s][:, :, 0].to(F64)
        dv = p.transpose(1, 2) @ do
        assert (grads["dv"][s][:, :, 0].to(F64) - dv).abs().max() <= 2.0 ** -6 * do.abs().max()


def test_two_captured_calls_replay_on_new_inputs(attn):  # noqa: F811
    """Forward and backward in one graph each, sharing no scratch, replayed in
    turn on other inputs."""
    cs = [Case(8, 2, 256, [100, 300], [100, 300], True, True, seed=1), Case(8, 2, 64, [333], [400], False, False, seed=2)]
    graphs, outs = [], []
    for c in cs:
        c.bwd(attn, *c.fwd(attn))
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o, l = c.fwd(attn)
            r = c.bwd(attn, o, l)
        graphs.append(g)
        outs.append((o, l, r))
    for c in cs:
        c.q.mul_(-0.5)
        c.v.add_(1.0)
        if "n_q" in c.kw:
            c.kw["n_q"].fill_(200)
            c.kw["n_k"].fill_(390)
    for g in graphs * 2:
        g.replay()
    torch.cuda.synchronize()
    for c, (o, l, r) in zip(cs, outs):
        o2, l2 = c.fwd(attn)
        assert torch.equal(o, o2) and torch.equal(l, l2)
        for n, x in c.bwd(attn, o2, l2).items():
            assert torch.equal(x, r[n]), n


def test_calls_on_two_streams_at_once(attn):  # noqa: F811
    cs = [Case(8, 2, 256, [900], [900], False, True, seed=3), Case(32, 8, 128, [300, 500], [300, 500], True, False, seed=4)]
    want = []
    for c in cs:
        o, l = c.fwd(attn)
        want.append((o, l, c.bwd(attn, o, l)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cs]
    got = []
    for _ in range(4):
        got = []
        for c, s in zip(cs, streams):
            o, l = c.fwd(attn, stream=s)
            got.append((o, l, c.bwd(attn, o, l, stream=s.cuda_stream)))
    torch.cuda.synchronize()
    for (o, l, r), (o2, l2, r2) in zip(want, got):
        assert torch.equal(o, o2) and torch.equal(l, l2)
        for n in r:
            assert torch.equal(r[n], r2[n])


def test_a_prompt_into_the_cache_and_back(attn):  # noqa: F811
    """A chunk of a prompt over a prefix kept in the cache: what the cache gives
    back is attended to as decode attends to it."""
    B, T, P = 3, 8, 16
    d = wl.AttnDims(B=B, T=T, Hq=16, Hkv=2, D=256, Drot=64)
    g = torch.Generator(device=DEV).manual_seed(9)
    n0 = torch.tensor([0, 5, 200], dtype=I32, device=DEV)
    cache = attn.KVCache.empty(d, 64, P, BF16, DEV)
    table = torch.randperm(60, generator=torch.Generator().manual_seed(1)).view(3, 20).to(I32).to(DEV)
    w = [torch.rand(256, generator=g, device=DEV) + 0.5 for _ in range(2)]
    fr = attn.rope_freqs(attn.rope_inv_freq(64), DEV)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(BF16)  # noqa: E731
    dp = d.with_(T=200)
    attn.kv_append(dp, r(B, 200, 16, 256), r(B, 200, 2, 256), r(B, 200, 2, 256), *w, fr, cache, table,
                   torch.zeros(B, dtype=I32, device=DEV), n0)
    q = attn.kv_append(d, r(B, T, 16, 256), r(B, T, 2, 256), r(B, T, 2, 256), *w, fr, cache, table, n0)
    total = (n0 + T).to(I32)
    k, v = attn.kv_read(d.with_(T=208), cache, table, torch.zeros(B, dtype=I32, device=DEV), total)
    gate = r(B, T, 16, 256)
    out, lse = attn.attn_prefill(d, q, k, v, n_k=total, gate=gate, return_lse=True)
    out2, lse2 = attn.attn_decode(d, q, cache, table, n0, gate=gate, return_lse=True)
    # both round their weights and their result: twice two halves of a step of bf16
    assert (lse - lse2).abs().max() <= 1e-5
    assert ((out.float() - out2.float()).abs() <= 2.0 ** -7 * out2.float().abs() + 2.0 ** -7 * v.float().abs().max() * torch.sigmoid(gate.float())).all()
