"""The operators around a prompt of the hybrid model's full-attention layers and
around its drafted tokens, as one table of cases: what each call gets, what it
returns, and the same results in plain torch operations.

  prefill       causal attention of whole prompts, or of chunks over a kept
                prefix: grouped heads, sequences of different lengths (packed
                one after the other, or rows of a padded batch), the layer's
                sigmoid gate and the log-sum-exp
  prefill_bwd   its gradients: dq, dk, dv and the gate's
  axes          per-head RMS norm of q and k with a rotary embedding whose
                pairs turn with one of several positions of a token (time,
                height and width of an image or video)
  axes_bwd      its gradients: dq, dk and the two norm weights'
  axes_append   the same for new tokens that go into the paged cache
  verify        drafted tokens against the target's probabilities, from given
                random numbers: how many stand, and the token after them

``own`` selects the framework's kernels; otherwise ``run`` computes the plain
form.  16 query heads and 2 key heads of 256 channels, 64 of them rotated, B =
128 rows, windows of a few tokens and T = 8192 go with the sizes of the
repository's workloads; the others are generic.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _pf(name, op, B, T, Hq, Hkv, D, lo=None, packed=False, plo=0, phi=0, gated=False):
    """Sequences of lo..T new tokens (None: all T), each after plo..phi earlier
    ones whose keys and values are there; packed, or rows of a padded batch."""
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "lo": T if lo is None else lo,
            "packed": packed, "plo": plo, "phi": phi, "gated": gated}


def _ax(name, op, B, T, Hq, Hkv, D, R, base=1e7, lo=None, inter=False, cyclic=False, image=32, P=64, fmt="e4m3"):
    """Text and images of up to image x image patches in turn, three axes; the
    axes' pairs in blocks, or one after the other (cyclic).  lo: the shortest
    row.  P, fmt: the cache of axes_append."""
    return {"name": name, "op": op, "B": B, "T": T, "Hq": Hq, "Hkv": Hkv, "D": D, "R": R, "base": base,
            "lo": -1 if lo is None else lo, "interleaved": inter, "cyclic": cyclic, "image": image, "P": P, "fmt": fmt}


def _ve(name, B, T, V, near=1.0, drafted=True, lo=None):
    """Up to T drafted tokens (lo..T) per row over V tokens; near: how far the
    draft's logits are from the target's (standard deviation); not drafted:
    tokens from a lookup, without probabilities of their own."""
    return {"name": name, "op": "verify", "B": B, "T": T, "V": V, "near": near, "drafted": drafted,
            "lo": T if lo is None else lo}


def listed():
    return [
        # one long prompt, gated
        _pf("prefill_t8192", "prefill", 1, 8192, 16, 2, 256, gated=True),
        # prompts of a training or serving batch packed one after the other, narrower heads
        _pf("prefill_packed", "prefill", 8, 4093, 32, 8, 128, 100, True),
        # chunks of prompts over prefixes read back from the cache: few rows, many keys
        _pf("prefill_chunk", "prefill", 2, 509, 16, 2, 256, plo=3000, phi=16001, gated=True),
        # one short prompt: latency
        _pf("prefill_short", "prefill", 1, 77, 9, 3, 64),
        # the backward pass of the long prompt
        _pf("prefill_bwd_t8192", "prefill_bwd", 1, 8192, 16, 2, 256, gated=True),
        # that of a packed training batch
        _pf("prefill_bwd_packed", "prefill_bwd", 8, 2045, 32, 8, 128, 100, True),
        # a long document with images through norm and rotation
        _ax("axes_t8192", "axes", 1, 8192, 16, 2, 256, 64),
        # the backward pass of a padded batch, all channels rotated in pairs, the axes in turn
        _ax("axes_bwd_ragged", "axes_bwd", 8, 1021, 32, 8, 128, 128, 10000.0, 100, True, True),
        # a prompt with images into the quantised cache
        _ax("axes_append_e4m3", "axes_append", 4, 2039, 16, 2, 256, 64, lo=300),
        # a serving step's drafts: a batch, a large vocabulary
        _ve("verify_b128", 128, 4, 131072),
        # one user's drafts from a lookup, a small odd vocabulary: latency
        _ve("verify_b1_lookup", 1, 5, 32003, drafted=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["prefill", "prefill", "prefill", "prefill_bwd", "prefill_bwd", "axes", "axes_bwd", "axes_append",
                     "verify", "verify"])
    Hq, Hkv = rng.choice([(16, 2), (32, 8), (8, 8), (9, 3), (24, 4), (12, 1), (16, 1)])
    D = rng.choice([64, 128, 256])
    if op in ("prefill", "prefill_bwd"):
        most = 16 * 256 * 8192 * 4096 // (1 if op == "prefill" else 2)     # heads x channels x scores
        B = _log(rng, 1, 24)
        T = _log(rng, 1, min(8192, max(1, int((2 * most / (B * Hq * D)) ** 0.5))))
        phi = 0
        if op == "prefill" and rng.random() < 0.4:
            phi = _log(rng, 1, max(1, min(30000, most // (B * Hq * D * T))))
        c = _pf("", op, B, T, Hq, Hkv, D, rng.choice([None, 0, max(1, T // 3)]), rng.random() < 0.6,
                rng.randint(0, phi), phi, rng.random() < 0.5)
    elif op == "verify":
        V = _log(rng, 1000, 200000)
        T = rng.choice([1, 2, 3, 4, 5, 7, 8])
        B = _log(rng, 1, max(1, min(160, 128 * 4 * 131072 // (T * V))))
        c = _ve("", B, T, V, rng.choice([0.3, 1.0, 2.0]), rng.random() < 0.75, rng.choice([None, 0]))
    else:
        B = _log(rng, 1, 64)
        heads = Hq + Hkv * (2 if op == "axes_append" else 1)
        T = _log(rng, 1, max(1, 8192 * 18 * 256 // (B * heads * D)))
        c = _ax("", op, B, T, Hq, Hkv, D, rng.choice([16, D // 4 // 16 * 16, D // 2, D]), rng.choice([10000.0, 1e6, 1e7]),
                rng.choice([None, 0, max(1, T // 2)]), rng.random() < 0.3, rng.random() < 0.5, rng.choice([3, 17, 32]),
                rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "e4m3"]))
    del c["name"]
    return c


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _spread(lo, hi, n):
    """n lengths spread evenly over lo..hi (their sum does not depend on a seed)."""
    return [lo + int((hi - lo) * (i + 0.5) / n + 0.5) for i in range(n)]


def _shuffled(values, order):
    return [values[i] for i in torch.randperm(len(values), generator=order).tolist()]


def _i32(values, dev):
    return torch.tensor(values, dtype=torch.int32, device=dev)


def _starts(lengths):
    at = [0]
    for n in lengths:
        at.append(at[-1] + n)
    return at


def _document(T, image, order):
    """Positions [3][T] of text and images in turn: a text token moves all axes
    on by one; an image's patches have one time, their row and their column, and
    what follows starts after its larger side."""
    cols, at = ([], [], []), 0
    while len(cols[0]) < T:
        for _ in range(int(torch.randint(1, 200, (1,), generator=order))):
            for c in cols:
                c.append(at)
            at += 1
        h, w = (int(x) for x in torch.randint(1, image + 1, (2,), generator=order))
        for y in range(h):
            for x in range(w):
                cols[0].append(at)
                cols[1].append(at + y)
                cols[2].append(at + x)
        at += max(h, w)
    return [c[:T] for c in cols]


def _axis_of_pairs(case):
    n = case["R"] // 2
    return [i % 3 for i in range(n)] if case["cyclic"] else [min(2, 3 * i // n) for i in range(n)]


def _inputs(c, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed))
    order = torch.Generator().manual_seed(int(seed) + 1)
    bf, op, B, T = torch.bfloat16, c["op"], c["B"], c["T"]
    s = {"case": c}

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(bf)

    if op == "verify":
        V = c["V"]
        logits = torch.randn((B, T + 1, V), generator=g, device=dev).mul_(2.5)
        s["target"] = torch.softmax(logits, -1)
        s["draft"] = None
        if c["drafted"]:
            logits[:, :T].add_(torch.randn((B, T, V), generator=g, device=dev), alpha=c["near"])
            s["draft"] = torch.softmax(logits[:, :T], -1)
        del logits
        # a drafted token is a sample of the draft (of the target, flattened, for a lookup)
        p = s["draft"] if c["drafted"] else s["target"][:, :T].sqrt()
        keys = torch.rand(p.shape, generator=g, device=dev).clamp_(min=1e-30).log_().div_(p)
        s["tokens"] = keys.argmax(-1).to(torch.int32)
        s["u"] = torch.rand((B, T + 1), generator=g, device=dev)
        s["n"] = None if c["lo"] == T else _i32(_shuffled(_spread(c["lo"], T, B), order), dev)
        return s
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if op in ("prefill", "prefill_bwd"):
        nq = _shuffled(_spread(c["lo"], T, B), order)
        nk = [n + m for n, m in zip(nq, _shuffled(_spread(c["plo"], c["phi"], B), order))]
        Tk = T + c["phi"]
        if c["packed"]:
            qa, ka, rows, krows = _starts(nq), _starts(nk), (sum(nq),), (sum(nk),)
            s["cu_q"] = _i32(qa, dev)
            s["cu_k"] = s["cu_q"] if nk == nq else _i32(ka, dev)
            s["n_q"] = s["n_k"] = None
            s["seqs"] = list(zip(qa, nq, nq, ka, nk))
        else:
            rows, krows = (B, T), (B, Tk)
            s["cu_q"] = s["cu_k"] = None
            s["n_q"] = None if min(nq) == T else _i32(nq, dev)
            s["n_k"] = None if min(nk) == Tk else _i32(nk, dev)
            s["seqs"] = [(b * T, T, nq[b], b * Tk, nk[b]) for b in range(B)]
        # queries and keys as norm and rotation leave them; new values as a part of the projection
        s["q"], s["k"] = normal(*rows, Hq, D, std=1.5), normal(*krows, Hkv, D)
        if nk == nq and rows == krows:
            s["v"] = normal(*krows, (Hq + 2 * Hkv) * D)[..., (Hq + Hkv) * D:].view(*krows, Hkv, D)
        else:
            s["v"] = normal(*krows, Hkv, D)
        # the gate: the second half of every head of a query projection twice as wide
        s["gate"] = normal(*rows, Hq, 2 * D)[..., D:] if c["gated"] else None
        if op == "prefill_bwd":
            fwd = _plain_prefill(s)
            s["out"], s["lse"] = fwd["out"], fwd["lse"]
            s["dout"] = normal(*rows, Hq, D, std=0.1)
        return s
    # norm and rotation: q, k, v as views of one packed projection
    R = c["R"]
    x = normal(B, T, (Hq + 2 * Hkv) * D, std=1.5)
    s["q"] = x[..., : Hq * D].view(B, T, Hq, D)
    s["k"] = x[..., Hq * D: (Hq + Hkv) * D].view(B, T, Hkv, D)
    s["v"] = x[..., (Hq + Hkv) * D:].view(B, T, Hkv, D)
    s["wq"] = torch.rand(D, generator=g, device=dev) + 0.5
    s["wk"] = torch.rand(D, generator=g, device=dev) + 0.5
    s["inv_freq"] = c["base"] ** (-2.0 * torch.arange(R // 2, dtype=torch.float64, device=dev) / R)
    docs = [_document(T, c["image"], order) for _ in range(B)]
    s["pos"] = _i32(docs, dev).transpose(0, 1).contiguous()                 # [3, B, T]
    s["axes"] = torch.tensor(_axis_of_pairs(c), dtype=torch.uint8, device=dev)
    lengths = None if c["lo"] < 0 else _shuffled(_spread(c["lo"], T, B), order)
    if op == "axes_append":
        P = c["P"]
        s["n"] = None if lengths is None else _i32(lengths, dev)
        s["start"] = torch.zeros(B, dtype=torch.int32, device=dev)
        pages = -(-T // P)
        n_pages = B * pages + 3
        s["page_table"] = torch.randperm(n_pages, generator=g, device=dev)[: B * pages].view(B, pages).to(torch.int32)
        fp8 = c["fmt"] == "e4m3"
        for name in ("k", "v"):
            s[name + "_pages"] = torch.zeros((n_pages, Hkv, P, D), dtype=bf, device=dev)
            s[name + "_scale"] = None
            if fp8:
                s[name + "_pages"] = s[name + "_pages"].to(torch.float8_e4m3fn)
                s[name + "_scale"] = torch.zeros((n_pages, Hkv, P), dtype=torch.uint8,
                                                 device=dev).view(torch.float8_e8m0fnu)
        return s
    s["mask"] = None
    if lengths is not None:
        s["mask"] = (torch.arange(T, device=dev) < _i32(lengths, dev)[:, None]).to(torch.uint8)
    if op == "axes_bwd":
        s["dq_out"], s["dk_out"] = normal(B, T, Hq, D, std=0.1), normal(B, T, Hkv, D, std=0.1)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own and case["op"] != "verify":
        from gated_deltanet_linear_04_gb300 import attn, workloads as wl
        c = case
        s["dims"] = wl.AttnDims(B=c["B"], T=c["T"], Hq=c["Hq"], Hkv=c["Hkv"], D=c["D"], Drot=c.get("R", 0),
                                interleaved=c.get("interleaved", False))
        if "inv_freq" in s:
            s["freqs"] = attn.rope_freqs(s["inv_freq"])
        if "page_table" in s:
            s["cache"] = attn.KVCache(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"])
    return s


# ---------------------------------------------------------------------------
# the plain forms
# ---------------------------------------------------------------------------
EPS = 1e-6


def _flat(x):
    """[rows, heads, D] of packed or padded heads."""
    return x.reshape(-1, *x.shape[-2:])


def _scores(s, seq):
    """(queries [Hkv, nq*G, D], keys [Hkv, nk, D], scores with -inf where a
    query does not see) of one sequence: its last query sees its last key."""
    c = s["case"]
    q0, _, nq, k0, nk = seq
    Hkv, D, G = c["Hkv"], c["D"], c["Hq"] // c["Hkv"]
    q = _flat(s["q"])[q0:q0 + nq].float().view(nq, Hkv, G, D).permute(1, 0, 2, 3).reshape(Hkv, nq * G, D)
    k = _flat(s["k"])[k0:k0 + nk].float().permute(1, 0, 2)
    z = torch.matmul(q, k.transpose(1, 2)) * D ** -0.5
    last = nk - nq + torch.arange(nq, device=z.device).repeat_interleave(G)
    z.masked_fill_(torch.arange(nk, device=z.device) > last[:, None], -math.inf)
    return q, k, z


def _per_head(x, Hkv, nq):
    """[Hkv, nq*G, D] as [nq, Hq, D]."""
    return x.view(Hkv, nq, -1, x.shape[-1]).permute(1, 0, 2, 3).reshape(nq, -1, x.shape[-1])


def _grouped(x, Hkv):
    """[nq, Hq, D] as [Hkv, nq*G, D]."""
    nq, Hq, D = x.shape
    return x.reshape(nq, Hkv, Hq // Hkv, D).permute(1, 0, 2, 3).reshape(Hkv, -1, D)


def _plain_prefill(s):
    c = s["case"]
    Hkv = c["Hkv"]
    out = torch.zeros(s["q"].shape, device=s["q"].device)
    lse = torch.full(s["q"].shape[:-1], -math.inf, device=out.device)
    for seq in s["seqs"]:
        q0, _, nq, k0, nk = seq
        if nq == 0 or nk == 0:
            continue
        _, _, z = _scores(s, seq)
        m = z.amax(-1, keepdim=True)
        z.sub_(m).exp_()
        l = z.sum(-1, keepdim=True)
        v = _flat(s["v"])[k0:k0 + nk].float().permute(1, 0, 2)
        _flat(out)[q0:q0 + nq] = _per_head(torch.matmul(z, v) / l, Hkv, nq)
        lse.view(-1, c["Hq"])[q0:q0 + nq] = _per_head(m + torch.log(l), Hkv, nq)[..., 0]
        del z
    if s["gate"] is not None:
        out.mul_(torch.sigmoid(s["gate"].float()))
    return {"out": out.to(torch.bfloat16), "lse": lse}


def _plain_prefill_bwd(s):
    c = s["case"]
    Hkv, Hq, D = c["Hkv"], c["Hq"], c["D"]
    scale, dev = D ** -0.5, s["q"].device
    dout, out = s["dout"].float(), s["out"].float()
    r = {"dq": torch.zeros(s["q"].shape, device=dev), "dk": torch.zeros(s["k"].shape, device=dev),
         "dv": torch.zeros(s["k"].shape, device=dev)}
    do = dout
    if s["gate"] is not None:
        sg = torch.sigmoid(s["gate"].float())
        do = dout * sg
        r["dgate"] = torch.zeros(s["q"].shape, device=dev)
        for q0, _, nq, k0, nk in s["seqs"]:
            _flat(r["dgate"])[q0:q0 + nq] = _flat(dout)[q0:q0 + nq] * _flat(out)[q0:q0 + nq] * (1 - _flat(sg)[q0:q0 + nq])
    for seq in s["seqs"]:
        q0, _, nq, k0, nk = seq
        if nq == 0 or nk == 0:
            continue
        q, k, p = _scores(s, seq)
        p.sub_(_grouped(s["lse"].view(-1, Hq, 1)[q0:q0 + nq], Hkv)).exp_()
        d = _grouped(_flat(do)[q0:q0 + nq], Hkv)
        v = _flat(s["v"])[k0:k0 + nk].float().permute(1, 0, 2)
        _flat(r["dv"])[k0:k0 + nk] = torch.matmul(p.transpose(1, 2), d).permute(1, 0, 2)
        # a row's sum p (dp - sum p dp) is 0: the inner sum from these p and dp, not from the rounded output, which is too
        # far off where a row has few keys
        ds = torch.matmul(d, v.transpose(1, 2))
        ds.sub_((ds * p).sum(-1, keepdim=True)).mul_(p).mul_(scale)
        del p
        _flat(r["dq"])[q0:q0 + nq] = _per_head(torch.matmul(ds, k), Hkv, nq)
        _flat(r["dk"])[k0:k0 + nk] = torch.matmul(ds.transpose(1, 2), q).permute(1, 0, 2)
        del ds
    return {n: x.to(torch.bfloat16) for n, x in r.items()}


def _angles(pos, axes, inv_freq):
    """cos and sin [B, T, 1, R/2] of the pairs' own positions, pos [3, B, T]."""
    a = (pos.double()[axes.long()].permute(1, 2, 0) * inv_freq)[:, :, None]
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


def _store(pages, scale, page, slot, valid, x):
    """x [B, T, Hkv, D] into pages[page, :, slot] where valid [B, T]; e4m3 with
    the smallest power of two that holds the row."""
    page, slot, x = page[valid], slot[valid], x[valid]
    if scale is None:
        pages[page, :, slot] = x.to(torch.bfloat16)
        return
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    e = torch.where(m == 0, torch.full_like(e, -127), e.clamp(-127, 127))
    codes = torch.ldexp(x, -e[..., None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    pages.view(torch.uint8)[page, :, slot] = codes.view(torch.uint8)
    scale.view(torch.uint8)[page, :, slot] = (e + 127).to(torch.uint8)


def _cached(s, q):
    """The append's results: the cache as the values that it stands for."""
    out = {"q": q, "k_pages": s["k_pages"], "v_pages": s["v_pages"]}
    if s["k_scale"] is not None:
        out.update(k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out


def _plain_axes(s):
    c = s["case"]
    how = (*_angles(s["pos"], s["axes"], s["inv_freq"]), c["R"], c["interleaved"])
    if c["op"] == "axes_append":
        t = torch.arange(c["T"], device=s["pos"].device)
        p = s["start"].long()[:, None] + t
        page, slot = s["page_table"].long().gather(1, p // c["P"]), p % c["P"]
        valid = torch.ones_like(p, dtype=torch.bool) if s["n"] is None else t < s["n"][:, None]
        _store(s["k_pages"], s["k_scale"], page, slot, valid, _norm_rope(s["k"], s["wk"], *how))
        _store(s["v_pages"], s["v_scale"], page, slot, valid, s["v"].float())
        return _cached(s, (_norm_rope(s["q"], s["wq"], *how) * valid[..., None, None]).to(torch.bfloat16))
    keep = 1.0 if s["mask"] is None else s["mask"].float()[..., None, None]
    if c["op"] == "axes":
        return {"q": (_norm_rope(s["q"], s["wq"], *how) * keep).to(torch.bfloat16),
                "k": (_norm_rope(s["k"], s["wk"], *how) * keep).to(torch.bfloat16)}
    dq, dwq = _norm_rope_bwd(s["q"], s["wq"], s["dq_out"], keep, *how)
    dk, dwk = _norm_rope_bwd(s["k"], s["wk"], s["dk_out"], keep, *how)
    return {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def _plain_verify(s):
    """A drafted token x stands while u q(x) < p(x); the token after the last
    one that stands is drawn from what the target has above the draft,
    max(p - q, 0), or from the target's next row if all stand: the first whose
    cumulative sum is above u times the whole.  Products and sums in 64 bits."""
    p, q, tok, u = s["target"], s["draft"], s["tokens"].long(), s["u"].double()
    B, T = tok.shape
    t = torch.arange(T, device=tok.device)
    n = torch.full((B,), T, device=tok.device) if s["n"] is None else s["n"].long()
    px = p[:, :T].gather(2, tok[..., None])[..., 0].double()
    qx = torch.ones_like(px) if q is None else q.gather(2, tok[..., None])[..., 0].double()
    stands = (u[:, :T] * qx < px) & (t < n[:, None])
    a = stands.long().cumprod(1).sum(1)
    rows = torch.arange(B, device=tok.device)
    at = a.clamp(max=T - 1)
    pr = p[rows, a].double()
    if q is None:
        rest = pr.scatter(1, tok[rows, at][:, None], 0.0)
    else:
        rest = (pr - q[rows, at].double()).clamp_(min=0.0)
    rest = torch.where((a < n)[:, None], rest, pr)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, pr)
    sums = rest.cumsum(1)
    x = u[:, T] * sums[:, -1]
    last = p.shape[2] - 1 - (rest.flip(1) > 0).to(torch.uint8).argmax(1)
    token = torch.minimum((sums <= x[:, None]).sum(1), last)
    out = torch.where(t < a[:, None], tok, torch.full_like(tok, -1))
    out = torch.cat((out, torch.full_like(out[:, :1], -1)), 1)
    out[rows, a] = token
    return {"tokens": out.to(torch.int32), "keep": (a + 1).to(torch.int32)}


def _plain(s):
    op = s["case"]["op"]
    if op == "prefill":
        return _plain_prefill(s)
    if op == "prefill_bwd":
        return _plain_prefill_bwd(s)
    return _plain_verify(s) if op == "verify" else _plain_axes(s)


# ---------------------------------------------------------------------------
# the framework's calls
# ---------------------------------------------------------------------------
def _own(s):
    op = s["case"]["op"]
    if op == "verify":
        from gated_deltanet_linear_04_gb300 import spec
        tokens, keep = spec.verify(s["target"], s["tokens"], s["u"], draft=s["draft"], n=s["n"])
        return {"tokens": tokens, "keep": keep}
    from gated_deltanet_linear_04_gb300 import attn
    d = s["dims"]
    if op in ("prefill", "prefill_bwd"):
        seqs = {n: s[n] for n in ("cu_q", "cu_k", "n_q", "n_k", "gate")}
        if op == "prefill":
            out, lse = attn.attn_prefill(d, s["q"], s["k"], s["v"], return_lse=True, **seqs)
            return {"out": out, "lse": lse}
        return attn.attn_prefill_backward(d, s["q"], s["k"], s["v"], s["out"], s["lse"], s["dout"], **seqs)
    if op == "axes_append":
        return _cached(s, attn.kv_append_axes(d, s["q"], s["k"], s["v"], s["wq"], s["wk"], s["freqs"], s["axes"],
                                              s["pos"], s["cache"], s["page_table"], s["start"], s["n"]))
    if op == "axes":
        q, k = attn.qk_norm_rope_axes(d, s["q"], s["k"], s["wq"], s["wk"], s["freqs"], s["axes"], s["pos"], s["mask"])
        return {"q": q, "k": k}
    return attn.qk_norm_rope_axes_backward(d, s["q"], s["k"], s["wq"], s["wk"], s["freqs"], s["axes"], s["pos"],
                                           s["dq_out"], s["dk_out"], s["mask"])


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# the least each pass reads, writes and computes
# ---------------------------------------------------------------------------
def work(case):
    c = case
    op, B, T = c["op"], c["B"], c["T"]
    if op == "verify":
        # the rows that the tokens after the drafts are drawn from: the target's, and the draft's where one fell.  (How
        # many rows keep all their drafts depends on the numbers; one in six of each token falls at near = 1.)
        fell = 0.0 if not c["drafted"] else B * (1.0 - 0.6 ** (c["near"] * c["lo"]))
        return {"bytes": 4 * c["V"] * (B + fell) + 16 * B * T, "flops": 2 * c["V"] * (B + fell)}
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if op in ("prefill", "prefill_bwd"):
        nq, past = _spread(c["lo"], T, B), sum(_spread(c["plo"], c["phi"], B))
        tokens, keys, mean = sum(nq), sum(nq) + past, past / B
        seen = sum(n * (n + 1) / 2 + n * mean for n in nq)
        q, kv, lse = 2 * Hq * D * tokens, 2 * Hkv * D * keys, 4 * Hq * tokens
        if op == "prefill":
            return {"bytes": q * (3 if c["gated"] else 2) + 2 * kv + lse, "flops": 4 * Hq * D * seen}
        return {"bytes": q * (6 if c["gated"] else 4) + 4 * kv + lse, "flops": 10 * Hq * D * seen}
    kept = B * T if c["lo"] < 0 else sum(_spread(c["lo"], T, B))
    if op == "axes_append":
        per_row = (D + 1) if c["fmt"] == "e4m3" else 2 * D
        return {"bytes": 2 * (Hq + 2 * Hkv) * D * kept + 2 * Hq * D * B * T + 2 * Hkv * per_row * kept + 12 * kept,
                "flops": (9 * (Hq + Hkv) + 4 * Hkv) * D * kept}
    heads = Hq + Hkv
    if op == "axes":
        return {"bytes": 2 * heads * D * (kept + B * T) + 12 * B * T, "flops": 9 * heads * D * kept}
    return {"bytes": 2 * heads * D * (2 * kept + B * T) + 12 * B * T, "flops": 18 * heads * D * kept}


# ---------------------------------------------------------------------------
# the definitions in 64 bits, written apart from the forms above
# ---------------------------------------------------------------------------
def _exact_prefill(s, case):
    """Head by head: softmax over the seen keys, and its derivative."""
    f64, dev = torch.float64, s["q"].device
    Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
    grad = case["op"] == "prefill_bwd"
    flat = {n: s[n].reshape(-1, *s[n].shape[-2:]) for n in ("q", "k", "v", "gate", "dout") if s.get(n) is not None}
    res = {n: torch.zeros(flat["q"].shape, dtype=f64, device=dev) for n in (("dq", "dgate") if grad else ("out",))}
    if grad:
        res.update({n: torch.zeros(flat["k"].shape, dtype=f64, device=dev) for n in ("dk", "dv")})
    else:
        res["lse"] = torch.full(flat["q"].shape[:2], -math.inf, dtype=f64, device=dev)
    for q0, _, nq, k0, nk in s["seqs"]:
        if nq == 0:
            continue
        i = torch.arange(nq, device=dev)[:, None] + (nk - nq)
        unseen = torch.arange(nk, device=dev)[None, :] > i
        none = (i < 0).view(-1)
        for h in range(Hq):
            kh = h // (Hq // Hkv)
            q, k, v = flat["q"][q0:q0 + nq, h].to(f64), flat["k"][k0:k0 + nk, kh].to(f64), flat["v"][k0:k0 + nk, kh].to(f64)
            z = (q @ k.T / math.sqrt(D)).masked_fill_(unseen, -math.inf)
            lse = torch.logsumexp(z, 1)
            w = z.sub_(lse.masked_fill(none, 0.0)[:, None]).exp_()
            o = w @ v
            sg = 1.0 / (1.0 + torch.exp(-flat["gate"][q0:q0 + nq, h].to(f64))) if "gate" in flat else None
            if not grad:
                res["out"][q0:q0 + nq, h] = o if sg is None else o * sg
                res["lse"][q0:q0 + nq, h] = lse
                continue
            d = flat["dout"][q0:q0 + nq, h].to(f64)
            if sg is not None:
                res["dgate"][q0:q0 + nq, h] = d * o * sg * (1.0 - sg)
                d = d * sg
            res["dv"][k0:k0 + nk, kh] += w.T @ d
            dz = w * (d @ v.T - (d * o).sum(1, keepdim=True)) / math.sqrt(D)
            res["dq"][q0:q0 + nq, h] = dz @ k
            res["dk"][k0:k0 + nk, kh] += dz.T @ q
    if grad and "gate" not in flat:
        del res["dgate"]
    shapes = {"lse": s["q"].shape[:-1], "dk": s["k"].shape, "dv": s["k"].shape}
    return {n: x.reshape(shapes.get(n, s["q"].shape)) for n, x in res.items()}


def _turn64(z, s, case, sign=1.0):
    """Each pair as a complex number, turned by the position on its axis."""
    R = case["R"]
    index = torch.arange(R, device=z.device)
    first, second = (index[0::2], index[1::2]) if case["interleaved"] else (index[: R // 2], index[R // 2:])
    w = torch.complex(z[..., first], z[..., second])
    for i, axis in enumerate(s["axes"].tolist()):
        ang = sign * s["pos"][axis].to(torch.float64) * s["inv_freq"][i]
        w[..., i] *= torch.polar(torch.ones_like(ang), ang)[..., None]
    out = z.clone()
    out[..., first] = w.real
    out[..., second] = w.imag
    return out


def _heads64(x, w, s, case):
    rms = (torch.linalg.vector_norm(x, dim=-1, keepdim=True) ** 2 / x.shape[-1] + EPS).sqrt()
    return _turn64(x / rms * w, s, case)


def _e4m3_64(x):
    """(codes, scale): the nearest e4m3 values of x / scale, ties to even."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.ceil(torch.log2((top / E4M3_MAX).clamp(min=2.0 ** -127))).clamp(-127, 127)
    smaller = (e > -127) & (top <= E4M3_MAX * torch.pow(torch.full_like(e, 2.0), e - 1))   # log2 a step too high
    e = torch.where(smaller, e - 1, e)
    y = x * torch.pow(torch.full_like(e, 2.0), -e)
    step = torch.pow(torch.full_like(y, 2.0), torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(y / step) * step, torch.pow(torch.full_like(e, 2.0), e).squeeze(-1)


def _exact_axes(s, case):
    f64, op, B, T = torch.float64, case["op"], case["B"], case["T"]
    if op != "axes_append":
        # the derivative in closed form, from z's own gradient
        q, k = s["q"].to(f64), s["k"].to(f64)
        kept = torch.ones((B, T), dtype=torch.bool, device=q.device) if s["mask"] is None else s["mask"] != 0
        res = {}
        for n, x, w in (("q", q, s["wq"].to(f64)), ("k", k, s["wk"].to(f64))):
            if op == "axes":
                res[n] = _heads64(x, w, s, case).masked_fill(~kept[..., None, None], 0.0)
                continue
            dz = _turn64(s["d%s_out" % n].to(f64).masked_fill(~kept[..., None, None], 0.0), s, case, -1.0)
            ms = x.pow(2).mean(-1, keepdim=True) + EPS
            res["dw" + n] = torch.einsum("bthd,bthd->d", dz, x / ms.sqrt())
            res["d" + n] = (dz * w - x * (dz * w * x).mean(-1, keepdim=True) / ms) / ms.sqrt()
        return res
    P, table = case["P"], s["page_table"].long()
    live = torch.arange(T, device=table.device)[None, :].expand(B, T)
    live = live < T if s["n"] is None else live < s["n"].long()[:, None]
    b, t = torch.nonzero(live, as_tuple=True)
    p = s["start"].long()[b] + t
    page, slot = table[b, p // P], p % P
    out = {"q": _heads64(s["q"].to(f64), s["wq"].to(f64), s, case).masked_fill(~live[..., None, None], 0.0)}
    for name, x in (("k", _heads64(s["k"].to(f64), s["wk"].to(f64), s, case)[b, t]), ("v", s["v"][b, t].to(f64))):
        pages = s[name + "_pages"].to(f64)
        if case["fmt"] == "e4m3":
            x, sc = _e4m3_64(x)
            scale = s[name + "_scale"].to(f64)
            scale[page, :, slot] = sc
            out[name + "_scale"] = scale
        pages[page, :, slot] = x
        out[name + "_pages"] = pages
    return out


def _exact_verify(s):
    """Row by row, token by token."""
    tok, u = s["tokens"].tolist(), s["u"].to(torch.float64).tolist()
    B, T = len(tok), len(tok[0])
    n = [T] * B if s["n"] is None else s["n"].tolist()
    tokens, keep = torch.full((B, T + 1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        target = s["target"][b].to(torch.float64)
        draft = None if s["draft"] is None else s["draft"][b].to(torch.float64)
        t = 0
        while t < n[b]:
            x = tok[b][t]
            if not u[b][t] * (1.0 if draft is None else float(draft[t, x])) < float(target[t, x]):
                break
            tokens[b, t] = x
            t += 1
        mass = target[t].clone()
        if t < n[b]:
            if draft is None:
                mass[tok[b][t]] = 0.0
            else:
                mass = torch.relu(mass - draft[t])
            if float(mass.sum()) == 0.0:
                mass = target[t].clone()
        total = torch.cumsum(mass, 0)
        at = int(torch.searchsorted(total, (u[b][T] * total[-1]).reshape(1), right=True))
        tokens[b, t] = min(at, int(torch.nonzero(mass)[-1])) if float(total[-1]) > 0 else 0
        keep[b] = t + 1
    dev = s["tokens"].device
    return {"tokens": tokens.to(dev), "keep": keep.to(dev)}


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s)
    return _exact_prefill(s, case) if case["op"] in ("prefill", "prefill_bwd") else _exact_axes(s, case)
