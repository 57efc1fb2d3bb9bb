"""Plain definitions of a prompt's attention and its gradients, and of the
verification of drafted tokens, in 64 bits, with bounds of the kernels' errors.

A bound counts roundings (half a step relative to the value: bf16 2^-8) of the
softmax weights, of dS, of dO where there is a gate, and of the results, plus
the f32 arithmetic behind them."""
import math
from fractions import Fraction

import torch

F64 = torch.float64
BF = 2.0 ** -8
F32 = 2.0 ** -24
# The kernels' exponential gives 0 below 2^-126, the smallest normal f32 (and bf16) number, and a product's operand or
# result below it may count as 0: each weight and each dS is off by up to that, whatever its size.
TINY = 2.0 ** -126


def sequences(B, rows, cu, n):
    """(start, slot, valid) of every sequence."""
    at = [rows // B * s for s in range(B + 1)] if cu is None else cu.tolist()
    out = []
    for s in range(B):
        slot = at[s + 1] - at[s]
        out.append((at[s], slot, slot if n is None else max(0, min(slot, int(n[s])))))
    return out


def seen(nq, nk, device):
    """[nq, nk]: the last query sees the last key."""
    i = torch.arange(nq, device=device)[:, None] + nk - nq
    return torch.arange(nk, device=device)[None, :] <= i


def score_error(q, k, s, scale):
    """f32 error of the scores: D products summed, the factor, and the
    exponent's argument and function."""
    D = q.shape[-1]
    return F32 * ((D + 4) * abs(scale) * (q.abs() @ k.abs().T) + 4 * s.abs()) + 2.0 ** -21


def prefill(q, k, v, qs, ks, scale, gate=None):
    """q [N, Hq, D], k, v [M, Hkv, D]; qs, ks from sequences().  out, lse and
    their bounds [N, Hq, ...], NaN in rows of no slot."""
    N, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.full(q.shape, math.nan, dtype=F64, device=q.device)
    lse = torch.full((N, Hq), math.nan, dtype=F64, device=q.device)
    out_tol, lse_tol = torch.zeros_like(out), torch.zeros_like(lse)
    for (q0, slot, nq), (k0, _, nk) in zip(qs, ks):
        out[q0:q0 + slot] = 0.0
        lse[q0:q0 + slot] = -math.inf
        if nq == 0 or nk == 0:
            continue
        vis = seen(nq, nk, q.device)
        rows = vis.any(1)
        for h in range(Hq):
            qq, kk, vv = (x[a:a + n, i].to(F64) for x, a, n, i in ((q, q0, nq, h), (k, k0, nk, h // G), (v, k0, nk, h // G)))
            s = scale * qq @ kk.T
            z = s.masked_fill(~vis, -math.inf)
            m = z.amax(-1, keepdim=True).masked_fill(~rows[:, None], 0.0)
            l = torch.exp(z - m).sum(-1, keepdim=True)
            p = torch.exp(z - m) / l.masked_fill(~rows[:, None], 1.0)
            o = p @ vv
            ds = score_error(qq, kk, s, scale) * vis
            rel = 2 * ds + 2 * ds.amax(-1, keepdim=True) + BF + F32 * (8 * nk ** 0.5 + 64)
            tol = (p * rel + TINY) @ vv.abs() + TINY
            if gate is not None:
                sg = torch.sigmoid(gate[q0:q0 + nq, h].to(F64))
                o, tol = o * sg, tol * sg + 2.0 ** -20 * (o * sg).abs()
            out[q0:q0 + nq, h] = o
            out_tol[q0:q0 + nq, h] = tol + BF * o.abs()
            lse[q0:q0 + nq, h] = torch.where(rows, (m + torch.log(l))[:, 0], torch.full_like(m[:, 0], -math.inf))
            lse_tol[q0:q0 + nq, h] = ds.amax(-1) + 2.0 ** -20 + 2.0 ** -22 * torch.where(rows, lse[q0:q0 + nq, h], 0 * m[:, 0]).abs()
    return out, lse, out_tol, lse_tol


def prefill_backward(q, k, v, dout, qs, ks, scale, gate=None):
    """Gradients by the formula and their bounds: {name: (value, bound)}, NaN in
    rows of no slot."""
    Hq = q.shape[1]
    G = Hq // k.shape[1]
    r = {n: torch.full(x.shape, math.nan, dtype=F64, device=q.device) for n, x in (("dq", q), ("dk", k), ("dv", k), ("dgate", q))}
    t = {n: torch.zeros_like(x) for n, x in r.items()}
    for (q0, slot, nq), (k0, kslot, nk) in zip(qs, ks):
        for n, a, w in (("dq", q0, slot), ("dgate", q0, slot), ("dk", k0, kslot), ("dv", k0, kslot)):
            r[n][a:a + w] = 0.0
        if nq == 0 or nk == 0:
            continue
        vis = seen(nq, nk, q.device)
        rows = vis.any(1)
        for h in range(Hq):
            qi, ki = slice(q0, q0 + nq), slice(k0, k0 + nk)
            kh = h // G
            qq, kk, vv, d = q[qi, h].to(F64), k[ki, kh].to(F64), v[ki, kh].to(F64), dout[qi, h].to(F64)
            s = scale * qq @ kk.T
            z = s.masked_fill(~vis, -math.inf)
            lse = torch.logsumexp(z, -1, keepdim=True).masked_fill(~rows[:, None], 0.0)
            p = torch.exp(z - lse)
            o = p @ vv
            do, do_err = d, 0.0
            if gate is not None:
                sg = torch.sigmoid(gate[qi, h].to(F64))
                r["dgate"][qi, h] = d * o * sg * (1 - sg)
                # out as given: rounded, with the forward's own error; the product rounded
                t["dgate"][qi, h] = ((d * (1 - sg)).abs() * (2 * BF * (o * sg).abs() + BF * (p @ vv.abs()) * sg)
                                     + BF * r["dgate"][qi, h].abs() + 2.0 ** -20 * (d * o).abs())
                do, do_err = d * sg, BF
            dp = do @ vv.T
            delta = (p * dp).sum(-1, keepdim=True)
            ds = p * (dp - delta)
            e_s = 2 * score_error(qq, kk, s, scale) * vis + 2.0 ** -20 + 2.0 ** -20 * lse.abs()
            mag = do.abs() @ vv.abs().T
            e_dp = mag * (do_err + F32 * (q.shape[-1] + 8))
            # delta from the rounded output, itself off by the weights' rounding
            e_delta = (do.abs() * (BF * o.abs() + 2 * BF * (p @ vv.abs()))).sum(-1, keepdim=True) + (p * e_dp).sum(-1, keepdim=True)
            e_ds = (p * (e_dp + e_delta) + ds.abs() * (BF + e_s) + TINY * (dp.abs() + delta.abs() + 2)) * vis
            n32 = F32 * (8 * (nk + nq * G) ** 0.5 + 64)
            r["dq"][qi, h] = scale * ds @ kk
            t["dq"][qi, h] = abs(scale) * (e_ds + n32 * ds.abs()) @ kk.abs() + BF * r["dq"][qi, h].abs() + TINY
            r["dk"][ki, kh] += scale * ds.T @ qq
            t["dk"][ki, kh] += abs(scale) * (e_ds + n32 * ds.abs()).T @ qq.abs()
            r["dv"][ki, kh] += p.T @ do
            t["dv"][ki, kh] += (p * (BF + do_err + e_s + n32) + TINY * vis).T @ do.abs()
        for n in ("dk", "dv"):
            t[n][k0:k0 + nk] += BF * r[n][k0:k0 + nk].abs() + TINY
    if gate is None:
        del r["dgate"], t["dgate"]
    return {n: (r[n], t[n]) for n in r}


def verify(target, tokens, u, draft=None, n=None):
    """tokens_out, keep with exact rational numbers; target, draft, u f32 CPU."""
    B, T1, V = target.shape
    out, keep = torch.full((B, T1), -1, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)

    def value(x):
        x = float(x)
        return Fraction(0) if x != x or x <= 0 else Fraction(min(x, 1.0))

    for b in range(B):
        m = T1 - 1 if n is None else max(0, min(T1 - 1, int(n[b])))
        a = 0
        while a < m:
            x = int(tokens[b, a])
            if not 0 <= x < V:
                break
            q = 1.0 if draft is None else float(draft[b, a, x])
            if not float(u[b, a]) * q < float(target[b, a, x]):   # (both sides exact in 64 bits)
                break
            out[b, a] = x
            a += 1
        p = [value(x) for x in target[b, a]]
        rest = list(p)
        if a < m:
            if draft is None:
                if 0 <= int(tokens[b, a]) < V:
                    rest[int(tokens[b, a])] = Fraction(0)
            else:
                rest = [max(x - value(y), Fraction(0)) for x, y in zip(p, draft[b, a])]
            if sum(rest) == 0:
                rest = p
        total, c, token = sum(rest), Fraction(0), 0
        x = Fraction(float(u[b, T1 - 1])) * total
        for i, y in enumerate(rest):
            c += y
            if c > x:
                token = i
                break
        out[b, a] = token
        keep[b] = a + 1
    return out, keep
