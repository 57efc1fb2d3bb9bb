"""The verification of drafted tokens on the GPU against exact rational
numbers, and the distribution of what comes out."""
import math

import pytest
import torch

from tests import _prompt_ref as R
from tests.test_gpu_attn import attn, status  # noqa: F401

pytestmark = pytest.mark.gpu

F32, I32 = torch.float32, torch.int32
DEV = "cuda:0"


@pytest.fixture(scope="module")
def spec(attn):  # noqa: F811
    from gated_deltanet_linear_04_gb300 import spec as s
    return s


def make(B, T, V, near, seed, drafted=True):
    g = torch.Generator().manual_seed(seed)
    logits = torch.randn(B, T + 1, V, generator=g) * 2
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :T] + near * torch.randn(B, T, V, generator=g), -1)
    p = draft if drafted else target[:, :T].sqrt()
    tokens = torch.multinomial(p.reshape(-1, V), 1, generator=g).view(B, T).to(I32) if T else torch.zeros(B, 0, dtype=I32)
    u = torch.rand(B, T + 1, generator=g)
    return target, tokens, u, draft if drafted else None


def call(spec, target, tokens, u, draft=None, n=None, **kw):
    dev = [None if x is None else x.to(DEV) for x in (target, tokens, u, draft, n)]
    out, keep = spec.verify(dev[0], dev[1], dev[2], draft=dev[3], n=dev[4], **kw)
    return out.cpu(), keep.cpu()


CASES = [(1, 1, 1, 0.5, True), (1, 1, 2, 1.0, True), (3, 4, 33, 1.0, True), (5, 8, 1000, 0.3, True), (2, 3, 4097, 2.0, True),
         (4, 5, 777, 1.0, False), (7, 0, 130, 1.0, True), (2, 40, 50, 0.05, True), (300, 2, 65, 1.0, True), (1, 2, 20011, 1.0, False)]


@pytest.mark.parametrize("case", CASES)
def test_against_exact_numbers(spec, case):
    B, T, V, near, drafted = case
    target, tokens, u, draft = make(B, T, V, near, B + T + V, drafted)
    n = None if B < 3 else torch.tensor([(i * 5) % (T + 3) - 1 for i in range(B)], dtype=I32)
    out, keep = call(spec, target, tokens, u, draft, n)
    want, wkeep = R.verify(target, tokens, u, draft, n)
    assert torch.equal(out, want) and torch.equal(keep, wkeep)


@pytest.mark.parametrize("V", [5, 64, 1000, 9001])
def test_borders(spec, V):
    """u of 0 and next to 1, probabilities that are equal, zeros, single tokens,
    drafts outside the vocabulary, rows of zeros and of NaN."""
    top = float(torch.nextafter(torch.tensor(1.0), torch.tensor(0.0)))
    p = torch.full((1, 2, V), 1.0 / V)
    one = torch.zeros(1, 2, V)
    one[..., V - 2] = 1.0
    zero = torch.zeros(1, 2, V)
    nan = torch.full((1, 2, V), math.nan)
    last = torch.zeros(1, 2, V)
    last[..., V - 1] = 2.0 ** -70                       # (below the sums' unit: as a row of zeros)
    for target in (p, one, zero, nan, last):
        for draft in (None, p[:, :1], one[:, :1]):
            for tok in (0, V - 2, V - 1, -1, V, 2 ** 31 - 1):
                for u0 in (0.0, 0.5, top):
                    for u1 in (0.0, 2.0 ** -140, 0.25, top, 1.0):
                        u, t = torch.tensor([[u0, u1]]), torch.tensor([[tok]], dtype=I32)
                        out, keep = call(spec, target, t, u, draft)
                        if u1 < 1.0 and target is not last:
                            want, wkeep = R.verify(target, t, u, draft)
                            assert torch.equal(out, want) and torch.equal(keep, wkeep), (tok, u0, u1)
                        got = int(out[0, int(keep[0]) - 1])
                        assert 0 <= got < V


@pytest.mark.parametrize("V", [17, 64, 5000, 131072])
@pytest.mark.parametrize("drafted", [True, False])
def test_rows_that_are_no_probabilities_give_some_token(spec, V, drafted):
    """Sums of 16 and more pass 64 bits."""
    B, T = 6, 3
    g = torch.Generator().manual_seed(V)
    target = torch.rand(B, T + 1, V, generator=g) * torch.tensor([1.0, 1.0, 4.0, 1e30, 0.01, math.inf]).view(B, 1, 1)
    tokens = torch.randint(0, V, (B, T), generator=g).to(I32)
    draft = torch.rand(B, T, V, generator=g) * 0.5 if drafted else None
    out, keep = call(spec, target, tokens, torch.rand(B, T + 1, generator=g), draft)
    for b in range(B):
        a = int(keep[b]) - 1
        assert 0 <= a <= T and torch.equal(out[b, :a], tokens[b, :a])
        assert 0 <= int(out[b, a]) < V and (out[b, a + 1:] == -1).all()


def test_a_cumulative_sum_next_to_u(spec):
    """Sums that are exact in binary, u on the border between two tokens."""
    V = 256
    p = torch.zeros(V + 1, 1, V)
    p[:] = 2.0 ** -8
    u = (torch.arange(V + 1).float() / V).clamp(max=float(torch.nextafter(torch.tensor(1.0), torch.tensor(0.0))))[:, None]
    out, keep = call(spec, p, torch.zeros(V + 1, 0, dtype=I32), u)
    # the first sum above i / 256 is that of token i
    assert out[:V, 0].tolist() == list(range(V)) and int(out[V, 0]) == V - 1
    below = torch.nextafter(u[1:V], torch.zeros(1))
    out, _ = call(spec, p[1:V], torch.zeros(V - 1, 0, dtype=I32), below)
    assert out[:, 0].tolist() == list(range(V - 1))


def test_tokens_come_out_as_the_target_has_them(spec):
    """Drafts from q, what comes first from p: 200,000 rows, chi-squared of 7
    degrees of freedom below 40 (1e-6)."""
    B, V = 200000, 8
    g = torch.Generator(device=DEV).manual_seed(3)
    p = torch.tensor([0.3, 0.05, 0.2, 0.02, 0.13, 0.1, 0.15, 0.05], device=DEV)
    q = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.1, 0.05, 0.05, 0.1], device=DEV)
    target = p.expand(B, 2, V).contiguous()
    for draft in (q.expand(B, 1, V).contiguous(), None):
        tok = torch.multinomial(q, B, replacement=True, generator=g)[:, None].to(I32)
        if draft is None:
            tok.fill_(3)
        u = torch.rand(B, 2, generator=g, device=DEV)
        out, keep = spec.verify(target, tok, u, draft=draft)
        for at, rows in ((0, torch.ones(B, dtype=torch.bool, device=DEV)), (1, keep == 2)):
            got = torch.bincount(out[rows, at].long(), minlength=V).double()
            want = p.double() * rows.sum()
            assert float(((got - want) ** 2 / want).sum()) < 40, (draft is None, at)


def test_a_large_vocabulary_with_few_and_many_rows(spec):
    """However a row is split over CTAs, its token is the same."""
    target, tokens, u, draft = make(2, 2, 131072, 0.7, 5)
    one = [call(spec, *(x[i:i + 1] for x in (target, tokens, u)), draft[i:i + 1]) for i in range(2)]
    dev = [x.to(DEV).repeat(*([400] + [1] * (x.dim() - 1))) for x in (target, tokens, u, draft)]
    out, keep = spec.verify(dev[0], dev[1], dev[2], draft=dev[3])
    for i in range(800):
        assert torch.equal(out[i].cpu(), one[i % 2][0][0]) and int(keep[i]) == int(one[i % 2][1])
    want, wkeep = R.verify(target, tokens, u, draft)
    assert torch.equal(torch.cat([o for o, _ in one]), want)


def test_unaligned_rows_streams_and_graphs(spec):
    target, tokens, u, draft = (x.to(DEV) for x in make(3, 2, 1001, 1.0, 11))
    want = spec.verify(target, tokens, u, draft=draft)
    raw = torch.empty(target.numel() + 1, device=DEV)
    moved = raw[1:].view(target.shape)                  # (4-byte aligned)
    moved.copy_(target)
    got = spec.verify(moved, tokens, u, draft=draft)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = spec.verify(target, tokens, u, draft=draft, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = spec.verify(target, tokens, u, draft=draft)
    u.mul_(0.5)
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(spec.verify(target, tokens, u, draft=draft), out))
    b0 = spec.verify(target[:0], tokens[:0], u[:0])
    assert b0[0].shape == (0, 3) and b0[1].shape == (0,)


def test_keep_commits_a_window(spec):
    """What verify keeps of a window is what gdn.decode_window takes."""
    from gated_deltanet_linear_04_gb300 import gdn, workloads as wl
    B, T, V = 4, 3, 500
    target, tokens, u, draft = (x.to(DEV) for x in make(B, T, V, 1.0, 21))
    out, keep = spec.verify(target, tokens, u, draft=draft)
    d = wl.Dims(B=B, T=T + 1, Hk=2, Hv=4, Dk=128, Dv=128)
    x = {k: v.to(DEV) for k, v in wl.make_activations(d, 3).items()}
    p = {k: v.to(DEV) for k, v in wl.make_params(d, 1).items()}
    s = {k: v.to(DEV) for k, v in wl.make_states(d, 2, "normal", "normal").items()}
    one = {k: v.clone() for k, v in s.items()}
    gdn.decode_window(d, x["qkv"], p["conv_w"], s["conv_state"], x["a"], x["b"], p["A_log"], p["dt_bias"], s["state"], keep)
    for b in range(B):
        st = {k: v[b:b + 1].clone() for k, v in one.items()}
        for t in range(int(keep[b])):
            gdn.recurrent_decode(d.with_(B=1, T=1), x["qkv"][b:b + 1, t].clone(), p["conv_w"], st["conv_state"],
                                 x["a"][b:b + 1, t].clone(), x["b"][b:b + 1, t].clone(), p["A_log"], p["dt_bias"],
                                 st["state"])
        assert torch.equal(st["conv_state"], s["conv_state"][b:b + 1])
        assert (st["state"] - s["state"][b:b + 1]).abs().max() <= 1e-4
