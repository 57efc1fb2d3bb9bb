"""Plain definitions of the full-attention operators in 64 bits (CPU, torch),
and the error bounds of their 16- and 8-bit results.

A bound counts roundings: half a step of the result's type relative to the
value (bf16 2^-8, e4m3 2^-4), plus the f32 arithmetic behind it."""
import math

import torch

F64 = torch.float64
E4M3_MAX = 448.0


def rotate(z, pos, inv_freq, interleaved, sign=1.0):
    """z [B, T, H, D] turned by pos [B, T] * inv_freq [R/2]."""
    half = inv_freq.numel()
    R = 2 * half
    ang = sign * pos.to(F64)[..., None, None] * inv_freq
    c, s = torch.cos(ang), torch.sin(ang)
    out = z.clone()
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, half), slice(half, R))
    out[..., a] = z[..., a] * c - z[..., b] * s
    out[..., b] = z[..., b] * c + z[..., a] * s
    return out


def norm(x, w, eps):
    if w is None:
        return x
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w


def norm_rope(x, w, pos, inv_freq, interleaved, eps, mask=None):
    y = rotate(norm(x.to(F64), None if w is None else w.to(F64), eps), pos, inv_freq, interleaved)
    return y if mask is None else torch.where((mask != 0)[..., None, None], y, torch.zeros_like(y))


def norm_rope_bwd(x, w, dy, pos, inv_freq, interleaved, eps, mask=None):
    """(dx, dw or None, sum |dz xhat|) by the formula."""
    x, dy = x.to(F64), dy.to(F64)
    if mask is not None:
        dy = torch.where((mask != 0)[..., None, None], dy, torch.zeros_like(dy))
    dz = rotate(dy, pos, inv_freq, interleaved, -1.0)
    if w is None:
        return dz, None, None
    rstd = 1.0 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    xhat = x * rstd
    g = dz * w.to(F64)
    dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
    return dx, (dz * xhat).sum((0, 1, 2)), (dz * xhat).abs().sum((0, 1, 2))


def scale_exponent(x):
    """[...] of rows x [..., D]: least e >= -127 with max|x| <= 448 * 2^e."""
    m, e = torch.frexp(x.abs().amax(-1))
    e = torch.where(m > 0.875, e - 8, e - 9)
    return torch.where(m == 0, torch.full_like(e, -127), e.clamp(min=-127))


def e4m3(x):
    """(values of the codes, exponent) of f64 rows, round to nearest even."""
    e = scale_exponent(x)
    y = torch.ldexp(x, -e[..., None])
    _, k = torch.frexp(y)
    step = torch.ldexp(torch.ones_like(y), (k - 1).clamp(min=-6) - 3)
    return torch.round(y / step) * step, e


def lookup(page_table, n_pages, page_size, b, p):
    """(page, slot) of position p of row b, or None without a valid page."""
    if p < 0 or p // page_size >= page_table.shape[1]:
        return None
    page = int(page_table[b, p // page_size])
    return (page, p % page_size) if 0 <= page < n_pages else None


def gather(cache64, page_table, page_size, b, n):
    """([n, Hkv, D] f64, valid [n]) of positions 0 .. n-1 of row b; cache64
    [n_pages, Hkv, page_size, D]."""
    out = torch.zeros((n, cache64.shape[1], cache64.shape[3]), dtype=F64)
    valid = torch.zeros(n, dtype=torch.bool)
    for p0 in range(0, n, page_size):
        at = lookup(page_table, cache64.shape[0], page_size, b, p0)
        m = min(page_size, n - p0)
        if at is not None:
            out[p0:p0 + m] = cache64[at[0], :, :m].permute(1, 0, 2)
            valid[p0:p0 + m] = True
    return out, valid


def decode(q, k64, v64, page_table, page_size, pos, n_new, scale, gate=None):
    """out, lse and the bounds of their errors, all f64.  Non-finite keys or
    values at unseen positions do not enter."""
    B, T, Hq, D = q.shape
    Hkv = k64.shape[1]
    G = Hq // Hkv
    out = torch.zeros((B, T, Hq, D), dtype=F64)
    lse = torch.full((B, T, Hq), -math.inf, dtype=F64)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    g64 = None if gate is None else torch.sigmoid(gate.to(F64))
    for b in range(B):
        n = T if n_new is None else max(0, min(T, int(n_new[b])))
        total = max(0, int(pos[b]) + n) if n else 0
        total = min(total, page_table.shape[1] * page_size)
        k, valid = gather(k64, page_table, page_size, b, total)
        v, _ = gather(v64, page_table, page_size, b, total)
        for t in range(n):
            see = torch.nonzero(valid & (torch.arange(total) <= int(pos[b]) + t))[:, 0]
            if not len(see):
                continue
            for h in range(Hkv):
                ks, vs = k[see, h], v[see, h]
                qs = q[b, t, h * G:(h + 1) * G].to(F64)
                s = scale * qs @ ks.T
                m = s.amax(-1, keepdim=True)
                l = torch.exp(s - m).sum(-1, keepdim=True)
                p = torch.exp(s - m) / l
                hs = slice(h * G, (h + 1) * G)
                out[b, t, hs] = p @ vs
                lse[b, t, hs] = (m + torch.log(l))[:, 0]
                # a score's f32 error: D products summed, the factor, the exponent's argument and function
                ds = 2.0 ** -24 * ((D + 4) * abs(scale) * (qs.abs() @ ks.abs().T) + 4 * s.abs()) + 2.0 ** -21
                # weights: e^ds, their own 16-bit rounding, a sum of len(see) terms in f32
                rel = 2 * ds + 2.0 ** -8 + 2.0 ** -24 * (len(see) ** 0.5 * 8 + 32)
                out_tol[b, t, hs] = (p * rel) @ vs.abs()
                lse_tol[b, t, hs] = ds.amax(-1) + 2.0 ** -20 + 2.0 ** -22 * lse[b, t, hs].abs()
    if g64 is not None:
        out, out_tol = out * g64, out_tol * g64 + 2.0 ** -20 * out.abs()
    return out, lse, out_tol + 2.0 ** -8 * out.abs(), lse_tol
