"""A Gated DeltaNet layer's core and a full-attention layer's core side by
side, as the layers of a hybrid model use them: a training step of the
attention layer (positions on three axes, as of tokens of an image), ragged
prompts into the paged e4m3 cache and their attention, decode steps of both
layers replayed as one CUDA graph, and a step of drafted tokens that are
verified.

The projections around the cores are random matrices.  Run on a GB300 after
``python -c "import __graft_entry__ as g; g.build()"``:

    python examples/hybrid_decode.py [rows] [prompt] [steps]
"""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

from gated_deltanet_linear_04_gb300 import attn, gdn, spec, workloads as wl  # noqa: E402

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def visible_attention(q, k, v, first):
    """Plain attention in f32: token t of q sees the positions up to first + t of k, v."""
    G = q.shape[2] // k.shape[2]
    k, v = (x.float().repeat_interleave(G, 2) for x in (k, v))
    s = torch.einsum("bthd,blhd->bhtl", q.float(), k) * q.shape[-1] ** -0.5
    at = torch.arange(k.shape[1], device=q.device)
    last = first[:, None] + torch.arange(q.shape[1], device=q.device)
    s = s.masked_fill(at > last[:, None, :, None], float("-inf"))
    return torch.einsum("bhtl,blhd->bthd", torch.softmax(s, -1), v)


def training_step(d, qkv, gate, dout, wq, wk, freqs, axes, pos):
    """Forward and backward of the attention layer's core from its packed
    projection and its gate, for the output's gradient dout: the output and
    the gradients of q, k, v, the gate and the norm weights."""
    q, k, v = split(d, qkv)
    qr, kr = attn.qk_norm_rope_axes(d, q, k, wq, wk, freqs, axes, pos)
    out, lse = attn.attn_prefill(d, qr, kr, v, gate=gate, return_lse=True)
    g = attn.attn_prefill_backward(d, qr, kr, v, out, lse, dout, gate=gate)
    grads = attn.qk_norm_rope_axes_backward(d, q, k, wq, wk, freqs, axes, pos, g["dq"], g["dk"])
    return out, dict(grads, dv=g["dv"], dgate=g["dgate"])


def image_positions(d, start, width, dev):
    """[3, B, T]: tokens of an image of `width` columns (its time, row, column), from `start` on."""
    t = torch.arange(d.T, device=dev)
    at = torch.stack([torch.zeros_like(t), t // width, t % width]) + start
    return at.to(I32)[:, None].expand(-1, d.B, -1).contiguous()


def split(d, qkv):
    """q, k, v views [B, T, heads, D] of a packed projection."""
    n, m = d.Hq * d.D, d.Hkv * d.D
    return (qkv[..., :n].view(d.B, d.T, d.Hq, d.D), qkv[..., n:n + m].view(d.B, d.T, d.Hkv, d.D),
            qkv[..., n + m:].view(d.B, d.T, d.Hkv, d.D))


def main(rows=8, prompt=700, steps=16):
    torch.manual_seed(0)
    dev = torch.device("cuda")
    B, P = rows, 64
    d = wl.AttnDims(B=B, T=prompt, Hq=16, Hkv=2, D=256, Drot=64)
    wq, wk = (torch.rand(d.D, device=dev) + 0.5 for _ in range(2))
    freqs = attn.rope_freqs(attn.rope_inv_freq(d.Drot, 1e7), dev)
    width = (d.Hq + 2 * d.Hkv) * d.D

    # training: gradients through norm, rotation and attention
    dt = d.with_(B=1, T=64)
    axes = attn.rope_axes([12, 10, 10], cyclic=True, device=dev)
    x = torch.randn((1, 64, width), device=dev).to(BF16)
    gate, dout = (torch.randn((1, 64, d.Hq, d.D), device=dev).to(BF16) for _ in range(2))
    out, grads = training_step(dt, x, gate, dout, wq, wk, freqs, axes, image_positions(dt, 0, 8, dev))
    for name, g in grads.items():
        assert torch.isfinite(g.float()).all(), name

    # serving: prompts of different lengths into the cache, pages in any order
    pages = -(-(prompt + steps + 4) // P)
    cache = attn.KVCache.empty(d, B * pages, P, attn.E4M3, dev)
    table = torch.randperm(B * pages, device=dev).view(B, pages).to(I32)
    length = torch.linspace(1, prompt, B, device=dev).round().to(I32)
    start = torch.zeros(B, dtype=I32, device=dev)
    q = attn.kv_append(d, *split(d, torch.randn((B, prompt, width), device=dev).to(BF16)), wq, wk, freqs, cache, table,
                       start, length)
    # the prompts' attention over what the cache holds; rows are aligned at their ends
    k, v = attn.kv_read(d, cache, table, start, length)
    out = attn.attn_prefill(d, q, k, v, n_q=length, n_k=length)
    want = visible_attention(q, k, v, start.long())
    valid = (torch.arange(prompt, device=dev) < length[:, None])[..., None, None]
    worst = float(((out.float() - want) * valid).norm() / (want * valid).norm())

    # one step of both layers; inputs and outputs in fixed buffers, replayed as a graph
    da, dg = d.with_(T=1), wl.Dims(B=B, T=1, Hk=16, Hv=32, Dk=128, Dv=128)
    pos = length.clone()
    qkv = torch.empty((B, 1, width), dtype=BF16, device=dev)
    gate = torch.empty((B, 1, d.Hq, d.D), dtype=BF16, device=dev)
    gdn_in = {k: v.to(dev) for k, v in wl.make_params(dg, 1).items()}
    gdn_in.update({k: v.to(dev) for k, v in wl.make_states(dg, 2, "normal", "normal").items()})
    x = {k: v[:, 0].contiguous().to(dev) for k, v in wl.make_activations(dg, 3).items()}

    def step():
        y = gdn.recurrent_decode(dg, x["qkv"], gdn_in["conv_w"], gdn_in["conv_state"], x["a"], x["b"], gdn_in["A_log"],
                                 gdn_in["dt_bias"], gdn_in["state"])
        q = attn.kv_append(da, *split(da, qkv), wq, wk, freqs, cache, table, pos)
        out, lse = attn.attn_decode(da, q, cache, table, pos, gate=gate, return_lse=True)
        pos.add_(1)
        return y, q, out, lse

    qkv.normal_()
    gate.normal_()
    first = (gdn_in["conv_state"].clone(), gdn_in["state"].clone(), pos.clone())
    step()                                        # sets kernel attributes; then back to the start
    for t, saved in zip((gdn_in["conv_state"], gdn_in["state"], pos), first):
        t.copy_(saved)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, q, out, lse = step()
    for _ in range(steps):
        qkv.normal_()
        gate.normal_()
        graph.replay()
        # the step against plain attention over what the cache holds
        n = int(pos.max())
        k, v = attn.kv_read(d.with_(T=n), cache, table, start, pos)
        want = visible_attention(q, k, v, (pos - 1).long()) * torch.sigmoid(gate.float())
        worst = max(worst, float((out.float() - want).norm() / want.norm()))
        assert torch.isfinite(y.float()).all()

    # a step of drafted tokens: a window of the last token and T drafts through both layers, then which of them stand
    T, V = 3, 1000
    dw, dgw = d.with_(T=T + 1), dg.with_(T=T + 1)
    xw = {k: v.to(dev) for k, v in wl.make_activations(dgw, 4).items()}
    head = torch.randn((d.Hq * d.D, V), device=dev) * 0.3

    def window(keep):   # advances the state by keep tokens
        return gdn.decode_window(dgw, xw["qkv"], gdn_in["conv_w"], gdn_in["conv_state"], xw["a"], xw["b"],
                                 gdn_in["A_log"], gdn_in["dt_bias"], gdn_in["state"], keep)

    y = window(torch.zeros(B, dtype=I32, device=dev))
    q = attn.kv_append(dw, *split(dw, torch.randn((B, T + 1, width), device=dev).to(BF16)), wq, wk, freqs, cache, table, pos)
    gate = torch.randn((B, T + 1, d.Hq, d.D), device=dev).to(BF16)
    out = attn.attn_decode(dw, q, cache, table, pos, gate=gate)
    n = int(pos.max()) + T + 1
    k, v = attn.kv_read(d.with_(T=n), cache, table, start, pos + T + 1)
    want = visible_attention(q, k, v, pos.long()) * torch.sigmoid(gate.float())
    worst = max(worst, float((out.float() - want).norm() / want.norm()))
    logits = out.float().view(B, T + 1, -1) @ head
    target, draft = torch.softmax(logits, -1), torch.softmax(logits[:, :T] + torch.randn((B, T, V), device=dev), -1)
    drafted = torch.multinomial(draft.view(-1, V), 1).view(B, T).to(I32)
    tokens, keep = spec.verify(target, drafted, torch.rand((B, T + 1), device=dev), draft=draft)
    window(keep)
    pos.add_(keep)                                # (positions behind are written again by the next step)
    assert torch.isfinite(y.float()).all() and ((tokens >= 0).sum(1) == keep).all()

    status = gdn.gdn_device_status()
    assert status == gdn.GDN_OK, gdn.status_string(status)
    print("%d rows, prompts up to %d, %d steps, %d of %d drafts stood: attention within %.1e (relative) of the plain form" % (
        B, prompt, steps, int(keep.sum()) - B, B * T, worst))
    return worst


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:4]))
