"""Relative errors (root mean square) of a prompt's results against their 64-bit
definition: of whole tensors, of each head, and of blocks of 64 rows of a head,
so that a result that lacks a token, a step or a part of its sum, or is off by a
small factor, shows, which bounds of every single element cannot see.

One rounding to bf16 is off by at most 2^-8 of a value, and by 2^-8 / sqrt 3 =
0.00226 root mean square where every value is the worst one; independent ones
add in squares.  What enters a result: out: P, and its own rounding (2); dv: P,
dO (with a gate) and its own (3); dgate: P and the rounding in out, and its own
(3); dq and dk: dO in dP, out in delta, dS, and their own (4).  A third more is
allowed for rows in which delta takes away more of dP than of its error, and
half as much again for single blocks."""
import math

import torch

F64, BF16 = torch.float64, torch.bfloat16
ONE = 2.0 ** -8 / math.sqrt(3.0)
ROUNDINGS = {"out": 2, "dv": 3, "dgate": 3, "dq": 4, "dk": 4}


def bound(name):
    return 4.0 / 3.0 * math.sqrt(ROUNDINGS[name]) * ONE


def errors(got, want, rows=64):
    """(of the tensor, the worst head's, the worst block's); [N, H, D], rows of no slot (NaN) left out."""
    mine = ~torch.isnan(want).any(-1).any(-1)
    got, want = got[mine].to(F64), want[mine]
    e, w = (got - want).square().sum(-1), want.square().sum(-1)          # [n, H]

    def rel(e, w):
        return float(torch.where(w > 0, (e / w.clamp(min=1e-300)).sqrt(), (e > 0) * math.inf).max())

    n = max(1, e.shape[0] // rows)
    at = [rows * i for i in range(n)] + [e.shape[0]]                        # (the rest with the last block)
    blocks = [torch.stack([x[a:b].sum(0) for a, b in zip(at, at[1:])]) for x in (e, w)]
    return rel(e.sum(), w.sum()), rel(e.sum(0), w.sum(0)), rel(*blocks)


def check(got, want, name):
    b = bound(name)
    tensor, head, block = errors(got, want)
    assert tensor <= b and head <= b and block <= 1.5 * b, "%s: %.5f of the tensor, %.5f of a head (bound %.5f), %.5f of a block" % (
        name, tensor, head, b, block)


def seen_by(nq, nk, dev):
    return torch.arange(nk, device=dev)[None, :] <= torch.arange(nq, device=dev)[:, None] + nk - nq


def restated(q, k, v, dout, qs, ks, scale, gate=None, delta_of_few=True, drop_token=None, drop_step=None):
    """The kernels' arithmetic with its roundings, in 64 bits elsewhere.
    delta_of_few False: every row's delta from the rounded output.  drop_token,
    drop_step: (sequence, head, first query or key), a query (64 keys) left out of
    dk and dv (of dq)."""
    def r(x):
        return x.to(torch.float32).to(BF16).to(F64)

    G = q.shape[1] // k.shape[1]
    res = {n: torch.zeros(x.shape, dtype=F64) for n, x in (("out", q), ("dq", q), ("dk", k), ("dv", k), ("dgate", q))}
    for s, ((q0, _, nq), (k0, _, nk)) in enumerate(zip(qs, ks)):
        if nq == 0 or nk == 0:
            continue
        vis = seen_by(nq, nk, q.device)
        some = vis.any(1)
        few = vis.sum(1) <= (64 if delta_of_few else 0)
        qi, ki = slice(q0, q0 + nq), slice(k0, k0 + nk)
        for h in range(q.shape[1]):
            qq, kk, vv, d = (x.to(F64) for x in (q[qi, h], k[ki, h // G], v[ki, h // G], dout[qi, h]))
            z = (scale * qq @ kk.T).masked_fill(~vis, -math.inf)
            m = z.amax(1, keepdim=True).masked_fill(~some[:, None], 0.0)
            w = torch.exp(z - m)
            l = w.sum(1, keepdim=True).masked_fill(~some[:, None], 1.0)
            sg = torch.ones_like(d) if gate is None else torch.sigmoid(gate[qi, h].to(F64))
            o = r(r(w) @ vv / l * sg)
            res["out"][qi, h] = o
            p = w / l
            do = d if gate is None else r(d * sg)
            dp = do @ vv.T
            delta = torch.where(few, (p * dp).sum(1), (d * o).sum(1))[:, None]
            ds, pb = r(p * (dp - delta)) * vis, r(p)
            res["dgate"][qi, h] = r(d * o * (1 - sg))
            dsq = ds.clone()
            if drop_step is not None and drop_step[:2] == (s, h):
                dsq[:, drop_step[2]:drop_step[2] + 64] = 0
            res["dq"][qi, h] = r(scale * dsq @ kk)
            if drop_token is not None and drop_token[:2] == (s, h):
                ds[drop_token[2]] = 0
                pb[drop_token[2]] = 0
            res["dk"][ki, h // G] += scale * ds.T @ qq
            res["dv"][ki, h // G] += pb.T @ do
    res["dk"], res["dv"] = r(res["dk"]), r(res["dv"])
    if gate is None:
        del res["dgate"]
    return res
