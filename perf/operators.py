"""The operators of the full-attention layers that stand between the Gated
DeltaNet layers of a hybrid model, as one table of cases: what each call gets,
what it returns, and the same results in plain torch operations.

  norm_rope      per-head RMS norm of q and k with the rotary position
                 embedding in the same pass (training, prefill)
  norm_rope_bwd  its gradients: dq, dk and the two norm weights' gradients
  append         norm + rotation of new tokens, keys and values written into a
                 paged cache (bf16, or e4m3 with one power-of-two scale per
                 token and head)
  read           a span of positions read back from the cache as bf16
  decode         attention of 1..8 new tokens per row over the paged cache,
                 optionally gated, with the log-sum-exp of the scores

``own`` selects the framework's kernels; otherwise ``run`` computes the plain
form.  Sizes: 16 query heads and 2 key heads of 256 channels, 64 of them
rotated, B = 128 rows and T = 8192 tokens go with the layer sizes of the
repository's workloads; the others are generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _nr(name, op, B, T, Hq, Hkv, D, R, base=10000.0, far=0, lo=None, inter=False):
    """lo: the shortest row (right-padded rows with lengths lo..T and a mask);
    None: all rows full, no mask.  far: largest first position."""
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "base": base, "far": far,
            "lo": -1 if lo is None else lo, "interleaved": inter}


def _ap(name, B, T, Hq, Hkv, D, R, P, fmt, lo, hi, ragged=False, base=10000.0, inter=False):
    """lo..hi: tokens already in the cache; ragged: rows take 0..T new tokens."""
    return {"name": name, "op": "append", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "P": P, "fmt": fmt,
            "lo": lo, "hi": hi, "ragged": ragged, "base": base, "interleaved": inter}


def _rd(name, B, T, Hkv, D, P, fmt, lo, hi):
    """T positions per row from a start in lo..hi; every other row a shorter span."""
    return {"name": name, "op": "read", "B": B, "T": T, "Hkv": Hkv, "D": D, "P": P, "fmt": fmt, "lo": lo, "hi": hi}


def _de(name, B, T, Hq, Hkv, D, P, fmt, lo, hi, gated=False):
    """lo..hi: tokens in the cache before the T new ones."""
    return {"name": name, "op": "decode", "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "P": P, "fmt": fmt,
            "lo": lo, "hi": hi, "gated": gated}


def listed():
    return [
        # one long prompt through the attention layer, positions far out
        _nr("norm_rope_t8192", "norm_rope", 1, 8192, 16, 2, 256, 64, 1e7, 200000),
        # a right-padded batch with narrower heads, whole-head rotation in pairs
        _nr("norm_rope_ragged", "norm_rope", 8, 1021, 32, 8, 128, 128, 10000.0, 0, 100, True),
        # the backward pass of the long prompt
        _nr("norm_rope_bwd_t8192", "norm_rope_bwd", 1, 8192, 16, 2, 256, 64, 1e7, 200000),
        # a small padded training batch of odd sizes
        _nr("norm_rope_bwd_small", "norm_rope_bwd", 3, 509, 9, 3, 64, 32, 10000.0, 0, 1),
        # a batched serving step, the cache quantised as it is written: one token of each row
        _ap("append_b128_e4m3", 128, 1, 16, 2, 256, 64, 64, "e4m3", 1, 1023, False, 1e7),
        # a long prompt into the quantised cache
        _ap("append_t8192_e4m3", 1, 8192, 16, 2, 256, 64, 64, "e4m3", 0, 0, False, 1e7),
        # prefixes read back from the quantised cache for a prefill
        _rd("read_ragged_e4m3", 8, 4093, 2, 256, 64, "e4m3", 0, 500),
        # a short span of an unquantised cache with small pages
        _rd("read_bf16", 3, 700, 8, 128, 16, "bf16", 17, 333),
        # one user, a short context: latency
        _de("decode_b1", 1, 1, 16, 2, 256, 16, "bf16", 1000, 1000, True),
        # the ordinary batch: ragged contexts, quantised cache, gated output
        _de("decode_b128_e4m3", 128, 1, 16, 2, 256, 64, "e4m3", 1, 4095, True),
        # a verify window of four tokens, narrower heads
        _de("decode_window_t4", 32, 4, 32, 8, 128, 32, "bf16", 500, 4091),
        # one row with a very long context: the length is split over the GPU
        _de("decode_long", 1, 1, 16, 2, 256, 64, "bf16", 262143, 262143),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    Hq, Hkv = rng.choice([(16, 2), (32, 8), (8, 8), (9, 3), (24, 4), (12, 1), (16, 1)])
    D = rng.choice([64, 128, 256])
    R = rng.choice([16, D // 4 // 16 * 16, D // 2, D])
    base = rng.choice([10000.0, 1e6, 1e7])
    inter = rng.random() < 0.3
    P = rng.choice([16, 32, 64, 128])
    fmt = rng.choice(["bf16", "e4m3"])
    op = rng.choice(["norm_rope", "norm_rope_bwd", "append", "read", "decode", "decode", "decode"])
    if op in ("norm_rope", "norm_rope_bwd"):
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 8192 * 18 * 256 // (B * (Hq + Hkv) * D)))
        c = _nr("", op, B, T, Hq, Hkv, D, R, base, rng.choice([0, 200000]), rng.choice([None, 0, max(1, T // 2)]), inter)
    elif op == "append":
        B = _log(rng, 1, 128)
        T = _log(rng, 1, max(1, 8192 * 18 * 256 // (B * (Hq + 2 * Hkv) * D)))
        hi = _log(rng, 1, 1024)
        c = _ap("", B, T, Hq, Hkv, D, R, P, fmt, rng.randint(0, hi), hi, rng.random() < 0.5, base, inter)
    elif op == "read":
        B = _log(rng, 1, 64)
        T = _log(rng, 1, max(1, 30_000_000 // (B * Hkv * D)))
        hi = _log(rng, 1, 1024)
        c = _rd("", B, T, Hkv, D, P, fmt, rng.randint(0, hi), hi)
    else:
        B = _log(rng, 1, 160)
        hi = _log(rng, 1, max(1, min(200000, 100_000_000 // (B * Hkv * D))))
        c = _de("", B, rng.choice([1, 1, 1, 2, 3, 4, 8]), Hq, Hkv, D, P, fmt, rng.randint(0, hi), hi, rng.random() < 0.5)
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n lengths spread evenly over lo..hi (their sum does not depend on a seed)."""
    return [lo + int((hi - lo) * (i + 0.5) / n + 0.5) for i in range(n)]


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _inputs(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    order = torch.Generator().manual_seed(int(seed) + 1)
    B, T, Hkv, D, op = c["B"], c["T"], c["Hkv"], c["D"], c["op"]
    bf = torch.bfloat16
    s = {"case": c}

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(bf)

    if "Hq" in c and op != "decode":
        # q, k, v as views of one packed projection
        Hq = c["Hq"]
        x = normal(B, T, (Hq + 2 * Hkv) * D, std=1.5)
        s["q"] = x[..., : Hq * D].view(B, T, Hq, D)
        s["k"] = x[..., Hq * D: (Hq + Hkv) * D].view(B, T, Hkv, D)
        s["v"] = x[..., (Hq + Hkv) * D:].view(B, T, Hkv, D)
        s["wq"] = torch.rand(D, generator=g, device=dev) + 0.5
        s["wk"] = torch.rand(D, generator=g, device=dev) + 0.5
        i = torch.arange(c["R"] // 2, dtype=torch.float64, device=dev)
        s["inv_freq"] = c["base"] ** (-2.0 * i / c["R"])
    if op in ("norm_rope", "norm_rope_bwd"):
        first = torch.randint(0, c["far"] + 1, (B, 1), generator=g, device=dev)
        s["pos"] = (first + torch.arange(T, device=dev)).to(torch.int32)
        s["mask"] = None
        if c["lo"] >= 0:
            n = torch.tensor(_spread(c["lo"], T, B))[torch.randperm(B, generator=order)].to(dev)
            s["mask"] = (torch.arange(T, device=dev)[None, :] < n[:, None]).to(torch.uint8)
        if op == "norm_rope_bwd":
            s["dq_out"] = normal(B, T, c["Hq"], D, std=0.1)
            s["dk_out"] = normal(B, T, Hkv, D, std=0.1)
        return s
    # paged cache: pages of all rows in random order
    P = c["P"]
    before = torch.tensor(_spread(c["lo"], c["hi"], B))[torch.randperm(B, generator=order)]
    pages = -(-(c["hi"] + T) // P)
    n_pages = B * pages + 3
    s["page_table"] = torch.randperm(n_pages, generator=g, device=dev)[: B * pages].view(B, pages).to(torch.int32)
    s["pos"] = _i32(before.tolist(), dev)
    shape = (n_pages, Hkv, P, D)
    for name in ("k", "v"):
        if op == "append":
            s[name + "_pages"] = torch.zeros(shape, dtype=bf, device=dev)
        else:
            s[name + "_pages"] = torch.randn(shape, generator=g, device=dev, dtype=bf)
        s[name + "_scale"] = None
        if c["fmt"] == "e4m3":
            s[name + "_pages"] = (s[name + "_pages"] * 100.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
            byte = torch.randint(119, 122, shape[:3], generator=g, device=dev, dtype=torch.uint8)
            s[name + "_scale"] = (byte * (op != "append")).view(torch.float8_e8m0fnu)
    s["n"] = None
    if op == "append" and c["ragged"]:
        s["n"] = _i32([_spread(0, T, B)[i] for i in torch.randperm(B, generator=order).tolist()], dev)
    if op == "read":
        s["n"] = _i32([T if i % 2 == 0 else T // 2 for i in range(B)], dev)
    if op == "decode":
        s["q"] = normal(B, T, c["Hq"], D, std=1.5)
        s["gate"] = None
        if c["gated"]:
            # the second half of every head of a query projection twice as wide
            s["gate"] = normal(B, T, c["Hq"], 2 * D)[..., D:]
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        from gated_deltanet_linear_04_gb300 import attn, workloads as wl
        c = case
        s["dims"] = wl.AttnDims(B=c["B"], T=c["T"], Hq=c.get("Hq", c["Hkv"]), Hkv=c["Hkv"], D=c["D"],
                                Drot=c.get("R", 0), interleaved=c.get("interleaved", False))
        if "inv_freq" in s:
            s["freqs"] = attn.rope_freqs(s["inv_freq"])
        if "page_table" in s:
            s["cache"] = attn.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
EPS = 1e-6


def _angles(pos, inv_freq):
    """cos and sin of pos * inv_freq, shaped pos.shape + [1, R/2]."""
    a = (pos.double()[..., None] * inv_freq)[..., None, :]
    return torch.cos(a).float(), torch.sin(a).float()


def _pairs(x, R, interleaved):
    r = x[..., :R]
    return (r[..., 0::2], r[..., 1::2]) if interleaved else (r[..., : R // 2], r[..., R // 2:])


def _unpair(a, b, rest, interleaved):
    r = torch.stack((a, b), -1).flatten(-2) if interleaved else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _norm_rope(x, w, cos, sin, R, interleaved):
    x = x.float()
    z = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w
    a, b = _pairs(z, R, interleaved)
    return _unpair(a * cos - b * sin, b * cos + a * sin, z[..., R:], interleaved)


def _norm_rope_bwd(x, w, dy, keep, cos, sin, R, interleaved):
    x, dy = x.float(), dy.float() * keep
    a, b = _pairs(dy, R, interleaved)
    dz = _unpair(a * cos + b * sin, b * cos - a * sin, dy[..., R:], interleaved)
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xhat = x * rstd
    dw = (dz * xhat).sum((0, 1, 2))
    dxhat = dz * w
    return (rstd * (dxhat - xhat * (dxhat * xhat).mean(-1, keepdim=True))).to(torch.bfloat16), dw


def _quantize(x):
    """(e4m3 codes, exponent byte): the smallest power of two that holds the row."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    codes = torch.ldexp(x, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, (e + 127).to(torch.uint8).view(torch.float8_e8m0fnu)


def _store(pages, scale, page, slot, valid, x):
    """x [B, T, Hkv, D] into pages[page, :, slot] where valid [B, T]."""
    page, slot, x = page[valid], slot[valid], x[valid]
    if scale is None:
        pages[page, :, slot] = x.to(torch.bfloat16)
        return
    codes, byte = _quantize(x)
    pages.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
    scale.view(torch.uint8)[page, :, slot] = byte.view(torch.uint8)


def _gather(pages, scale, page, slot):
    """f32 [B, T, Hkv, D] of the positions' pages and slots [B, T]."""
    if scale is None:
        return pages[page, :, slot].float()
    x = pages.view(torch.uint8)[page, :, slot].view(torch.float8_e4m3fn).float()
    return x * scale.view(torch.uint8)[page, :, slot].view(torch.float8_e8m0fnu).float()[..., None]


def _where(page_table, p, P):
    """(page, slot) of positions p [B, T], positions past the table clamped."""
    at = (p // P).clamp(max=page_table.shape[1] - 1)
    return page_table.long().gather(1, at), p % P


def _plain(s):
    c = s["case"]
    op, B, T = c["op"], c["B"], c["T"]
    if op in ("norm_rope", "norm_rope_bwd"):
        cos, sin = _angles(s["pos"], s["inv_freq"])
        keep = 1.0 if s["mask"] is None else s["mask"].float()[..., None, None]
        how = (cos, sin, c["R"], c["interleaved"])
        if op == "norm_rope":
            return {"q": (_norm_rope(s["q"], s["wq"], *how) * keep).to(torch.bfloat16),
                    "k": (_norm_rope(s["k"], s["wk"], *how) * keep).to(torch.bfloat16)}
        dq, dwq = _norm_rope_bwd(s["q"], s["wq"], s["dq_out"], keep, *how)
        dk, dwk = _norm_rope_bwd(s["k"], s["wk"], s["dk_out"], keep, *how)
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    t = torch.arange(T, device=s["pos"].device)
    p = s["pos"].long()[:, None] + t
    if op in ("append", "read"):
        page, slot = _where(s["page_table"], p, c["P"])
        valid = torch.ones_like(p, dtype=torch.bool) if s["n"] is None else t < s["n"][:, None]
        if op == "read":
            keep = valid[..., None, None]
            return {"k": (_gather(s["k_pages"], s["k_scale"], page, slot) * keep).to(torch.bfloat16),
                    "v": (_gather(s["v_pages"], s["v_scale"], page, slot) * keep).to(torch.bfloat16)}
        how = (*_angles(p, s["inv_freq"]), c["R"], c["interleaved"])
        q = _norm_rope(s["q"], s["wq"], *how) * valid[..., None, None]
        _store(s["k_pages"], s["k_scale"], page, slot, valid, _norm_rope(s["k"], s["wk"], *how))
        _store(s["v_pages"], s["v_scale"], page, slot, valid, s["v"].float())
        return _appended(s, q.to(torch.bfloat16))
    # decode
    Hkv, D = c["Hkv"], c["D"]
    G = c["Hq"] // Hkv
    L = c["hi"] + T
    at = torch.arange(L, device=t.device).expand(B, L)
    page, slot = _where(s["page_table"], at, c["P"])
    k = _gather(s["k_pages"], s["k_scale"], page, slot)
    v = _gather(s["v_pages"], s["v_scale"], page, slot)
    q = s["q"].float().view(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    scores = torch.matmul(q, k.permute(0, 2, 3, 1)) * D ** -0.5
    seen = (at[:, None, :] <= p[:, :, None]).repeat_interleave(G, 1)[:, None]
    scores = scores.masked_fill(~seen, -math.inf)
    m = scores.amax(-1, keepdim=True)
    e = torch.exp(scores - m)
    l = e.sum(-1, keepdim=True)
    out = torch.matmul(e / l, v.permute(0, 2, 1, 3))
    out = out.view(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, c["Hq"], D)
    lse = (m + torch.log(l)).view(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, c["Hq"])
    if s["gate"] is not None:
        out = out * torch.sigmoid(s["gate"].float())
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _appended(s, q):
    out = {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["k_scale"] is not None:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    from gated_deltanet_linear_04_gb300 import attn
    op, d = s["case"]["op"], s["dims"]
    if op == "norm_rope":
        q, k = attn.qk_norm_rope(d, s["q"], s["k"], s["wq"], s["wk"], s["freqs"], s["pos"], s["mask"])
        return {"q": q, "k": k}
    if op == "norm_rope_bwd":
        return attn.qk_norm_rope_backward(d, s["q"], s["k"], s["wq"], s["wk"], s["freqs"], s["pos"], s["dq_out"],
                                          s["dk_out"], s["mask"])
    if op == "append":
        q = attn.kv_append(d, s["q"], s["k"], s["v"], s["wq"], s["wk"], s["freqs"], s["cache"], s["page_table"],
                           s["pos"], s["n"])
        return _appended(s, q)
    if op == "read":
        k, v = attn.kv_read(d, s["cache"], s["page_table"], s["pos"], s["n"])
        return {"k": k, "v": v}
    out, lse = attn.attn_decode(d, s["q"], s["cache"], s["page_table"], s["pos"], gate=s["gate"], return_lse=True)
    return {"out": out, "lse": lse}


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the least each pass reads, writes and computes
# ---------------------------------------------------------------------------
def work(case):
    c = case
    op, B, T, Hkv, D = c["op"], c["B"], c["T"], c["Hkv"], c["D"]
    Hq = c.get("Hq", 0)
    per_row = (D + 1) if c.get("fmt") == "e4m3" else 2 * D     # one head's key or value of one token
    if op in ("norm_rope", "norm_rope_bwd"):
        kept = B * T if c["lo"] < 0 else sum(_spread(c["lo"], T, B))
        heads = Hq + Hkv
        if op == "norm_rope":
            return {"bytes": 2 * heads * D * (kept + B * T) + 4 * B * T + 8 * D, "flops": 9 * heads * D * kept}
        return {"bytes": 2 * heads * D * (2 * kept + B * T) + 4 * B * T + 16 * D, "flops": 18 * heads * D * kept}
    if op == "append":
        kept = sum(_spread(0, T, B)) if c["ragged"] else B * T
        return {"bytes": 2 * (Hq + 2 * Hkv) * D * kept + 2 * Hq * D * B * T + 2 * Hkv * per_row * kept + 8 * D,
                "flops": (9 * (Hq + Hkv) + 4 * Hkv) * D * kept}
    if op == "read":
        kept = sum(T if i % 2 == 0 else T // 2 for i in range(B))
        return {"bytes": 2 * Hkv * (per_row * kept + 2 * D * B * T), "flops": 2 * Hkv * D * kept}
    keys = sum(n + T for n in _spread(c["lo"], c["hi"], B))
    seen = sum(n + t + 1 for n in _spread(c["lo"], c["hi"], B) for t in range(T))
    return {"bytes": 2 * Hkv * per_row * keys + 2 * B * T * Hq * D * (3 if c["gated"] else 2) + 4 * B * T * Hq,
            "flops": 4 * Hq * D * seen}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the forms above
# ---------------------------------------------------------------------------
def _rotate64(z, pos, case, inv_freq, sign=1.0):
    """Each pair as a complex number, turned by sign * position * frequency."""
    R = case["R"]
    half = R // 2
    index = torch.arange(R, device=z.device)
    first = index[0::2] if case["interleaved"] else index[:half]
    second = index[1::2] if case["interleaved"] else index[half:]
    w = torch.complex(z[..., first], z[..., second])
    ang = pos.to(torch.float64).unsqueeze(-1).unsqueeze(-1) * inv_freq
    w = w * torch.polar(torch.ones_like(ang), sign * ang)
    out = z.clone()
    out[..., first] = w.real
    out[..., second] = w.imag
    return out


def _heads64(x, w, pos, case, inv_freq):
    rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS).sqrt()
    return _rotate64(x / rms * w, pos, case, inv_freq)


def _e4m3_64(x):
    """(codes, scale): the nearest e4m3 values of x / scale, ties to even."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((top / E4M3_MAX).clamp(min=2.0 ** -127))).clamp(-127, 127)
    smaller = (e > -127) & (top <= E4M3_MAX * torch.pow(torch.full_like(e, 2.0), e - 1))   # log2 a step too high
    e = torch.where(smaller, e - 1, e)
    y = x * torch.pow(torch.full_like(e, 2.0), -e)
    step = torch.pow(torch.full_like(y, 2.0), torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.pow(torch.full_like(e, 2.0), e).squeeze(-1)


def exact(case, seed):
    s = _inputs(case, seed)
    op, B, T, D = case["op"], case["B"], case["T"], case["D"]
    f64 = torch.float64
    if op in ("norm_rope", "norm_rope_bwd"):
        grad = op == "norm_rope_bwd"
        q, k = (s[n].to(f64).requires_grad_(grad) for n in ("q", "k"))
        wq, wk = (s[n].to(f64).requires_grad_(grad) for n in ("wq", "wk"))
        qo, ko = _heads64(q, wq, s["pos"], case, s["inv_freq"]), _heads64(k, wk, s["pos"], case, s["inv_freq"])
        if s["mask"] is not None:
            gone = (s["mask"] == 0)[..., None, None]
            qo, ko = qo.masked_fill(gone, 0.0), ko.masked_fill(gone, 0.0)
        if not grad:
            return {"q": qo, "k": ko}
        dq, dk, dwq, dwk = torch.autograd.grad((qo, ko), (q, k, wq, wk), (s["dq_out"].to(f64), s["dk_out"].to(f64)))
        return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}
    P, table = case["P"], s["page_table"].long()
    start = s["pos"].long()
    if op == "append":
        b, t = torch.meshgrid(torch.arange(B, device=table.device), torch.arange(T, device=table.device), indexing="ij")
        if s["n"] is not None:
            live = t < s["n"].long()[:, None]
            b, t = b[live], t[live]
        else:
            b, t = b.flatten(), t.flatten()
        p = start[b] + t
        page, slot = table[b, p // P], p % P
        q = torch.zeros((B, T, case["Hq"], D), dtype=f64, device=table.device)
        q[b, t] = _heads64(s["q"][b, t].to(f64), s["wq"].to(f64), p, case, s["inv_freq"])
        out = {"q": q}
        for name, x in (("k", _heads64(s["k"][b, t].to(f64), s["wk"].to(f64), p, case, s["inv_freq"])),
                        ("v", s["v"][b, t].to(f64))):
            pages = s[name + "_pages"].to(f64)
            if case["fmt"] == "e4m3":
                x, sc = _e4m3_64(x)
                scale = s[name + "_scale"].to(f64)
                scale[page, :, slot] = sc
                out[name + "_scale"] = scale
            pages[page, :, slot] = x
            out[name + "_pages"] = pages
        return out
    Hkv = case["Hkv"]
    span = T if op == "read" else case["hi"] + T
    pos = torch.arange(span, device=table.device)[None, :] + (start[:, None] if op == "read" else torch.zeros_like(start)[:, None])
    page = table[torch.arange(B, device=table.device)[:, None], torch.clamp(pos // P, max=table.shape[1] - 1)]
    flat = page * P + pos % P
    kv = {}
    for name in ("k", "v"):
        x = s[name + "_pages"].to(f64)
        if case["fmt"] == "e4m3":
            x = x * s[name + "_scale"].to(f64).unsqueeze(-1)
        kv[name] = x.permute(0, 2, 1, 3).reshape(-1, Hkv, D)[flat]              # [B, span, Hkv, D]
        del x
    if op == "read":
        gone = torch.arange(T, device=table.device)[None, :] >= s["n"].long()[:, None]
        return {n: kv[n].masked_fill(gone[..., None, None], 0.0) for n in ("k", "v")}
    G = case["Hq"] // Hkv
    qq = s["q"].to(f64).reshape(B, T, Hkv, G, D)
    z = torch.einsum("bthgd,blhd->bthgl", qq, kv["k"]) / math.sqrt(D)
    last = start[:, None] + torch.arange(T, device=table.device)
    hidden = pos[:, None, :] > last[:, :, None]
    z = z.masked_fill(hidden[:, :, None, None, :], -math.inf)
    lse = torch.logsumexp(z, -1)
    out = torch.einsum("bthgl,blhd->bthgd", torch.exp(z - lse[..., None]), kv["v"]).reshape(B, T, case["Hq"], D)
    if s["gate"] is not None:
        out = out / (1.0 + torch.exp(-s["gate"].to(f64)))
    return {"out": out, "lse": lse.reshape(B, T, case["Hq"])}
