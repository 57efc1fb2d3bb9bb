"""A Gated DeltaNet layer's core and a full-attention layer's core side by
side, as the layers of a hybrid model use them: a training step of the
attention layer's norm and rotation, a ragged prompt into the paged e4m3
cache, and decode steps of both layers replayed as one CUDA graph.

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

from gated_deltanet_linear_04_gb300 import attn, gdn, workloads as wl  # noqa: E402

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


def training_step(d, qkv, wq, wk, freqs):
    """Forward and backward of the attention layer from its packed projection;
    returns the gradients of q, k and the norm weights."""
    q, k, v = split(d, qkv)
    pos = torch.arange(d.T, dtype=I32, device=q.device).expand(d.B, -1).contiguous()
    qr, kr = attn.qk_norm_rope(d, q, k, wq, wk, freqs, pos)
    qa, ka = qr.clone().requires_grad_(), kr.clone().requires_grad_()
    out = visible_attention(qa, ka, v, torch.zeros(d.B, dtype=torch.long, device=q.device))
    dq, dk = torch.autograd.grad(out.square().mean() * 1e3, (qa, ka))
    return attn.qk_norm_rope_backward(d, q, k, wq, wk, freqs, pos, dq.contiguous(), dk.contiguous())


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

    # training: gradients through the norm and the rotation
    dt = d.with_(B=1, T=64)
    grads = training_step(dt, torch.randn((1, 64, width), device=dev).to(BF16), wq, wk, freqs)
    for name, g in grads.items():
        assert torch.isfinite(g.float()).all(), name

    # serving: prompts of different lengths into the cache, pages in any order
    pages = -(-(prompt + steps) // P)
    cache = attn.KVCache.empty(d, B * pages, P, attn.E4M3, dev)
    table = torch.randperm(B * pages, device=dev).view(B, pages).to(I32)
    length = torch.linspace(1, prompt, B, device=dev).round().to(I32)
    start = torch.zeros(B, dtype=I32, device=dev)
    attn.kv_append(d, *split(d, torch.randn((B, prompt, width), device=dev).to(BF16)), wq, wk, freqs, cache, table,
                   start, length)

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
    worst = 0.0
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
    status = gdn.gdn_device_status()
    assert status == gdn.GDN_OK, gdn.status_string(status)
    print("%d rows, prompts up to %d, %d steps: attention within %.1e (relative) of the plain form" % (
        B, prompt, steps, worst))
    return worst


if __name__ == "__main__":
    main(*(int(a) for a in sys.argv[1:4]))
