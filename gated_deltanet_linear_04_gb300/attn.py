"""Binding of the full-attention operators of include/gdn.h (ctypes).

The layers that stand between the Gated DeltaNet layers of a hybrid model:
per-head norm and rotation of queries and keys (and its gradients), a paged
key-value cache written and read back in bf16 or e4m3, and the attention of
new tokens over it.  As in ``gdn``: argument checks and marshalling only, the
functions named like the ABI take caller-allocated outputs, the short names
allocate them, a non-zero status raises ``GdnError``, and work runs on
``stream`` (default: torch's current stream).

q, k, v and gate may be views [B, T, heads, D] of a packed projection: the
channels of a head dense, one stride from token to token over all rows and one
from head to head, both multiples of 8 elements.
"""
from __future__ import annotations

import ctypes
import math
from typing import Optional

import torch

from .gdn import BF16, F32, U8, GdnAttnDims, GdnKvCache, _check, _numel, _ptr, _stream, lib

I32, I64 = torch.int32, torch.int64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def make_attn_dims(d) -> GdnAttnDims:
    return GdnAttnDims(int(d.B), int(d.T), int(d.Hq), int(d.Hkv), int(d.D), int(d.Drot), int(bool(d.interleaved)),
                       float(d.eps))


def _heads(t: torch.Tensor, shape, name: str):
    """(address, token stride, head stride) of a bf16 [B, T, heads, D] view."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != BF16:
        raise TypeError("%s must be %s, got %s" % (name, BF16, t.dtype))
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    n = t.numel()
    if n == 0:
        return None, 0, 0
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    sb, st, sh, sd = t.stride()
    B, T, H, _ = shape
    if T == 1:
        st = sb if B > 1 else 0
    elif B > 1 and sb != T * st:
        raise ValueError("%s: its rows must follow each other at one token stride, got strides %s" % (name, t.stride()))
    if H == 1:
        sh = 0
    if sd != 1 or st % 8 or sh % 8:
        raise ValueError("%s must have dense channels and token and head strides that are multiples of 8, got "
                         "strides %s" % (name, t.stride()))
    return t.data_ptr(), st, sh


def _shaped(t: Optional[torch.Tensor], dtype, shape, name: str):
    """A dense tensor's address after its type and shape were compared."""
    if t is not None and isinstance(t, torch.Tensor) and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    return _ptr(t, dtype, name)


def _new(shape, dtype, device, stream):
    """A tensor for work on `stream`: made on the current stream, and not
    handed out again before `stream` is done with it."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device=device)
        t.record_stream(s)
    return t


# ---------------------------------------------------------------------------
# rotation frequencies and the cache
# ---------------------------------------------------------------------------
def rope_inv_freq(Drot: int, base: float = 10000.0) -> torch.Tensor:
    """The usual frequencies base^(-2i/Drot), i < Drot/2, in radians per position (f64, CPU)."""
    return float(base) ** (-2.0 * torch.arange(Drot // 2, dtype=torch.float64) / max(Drot, 1))


def rope_freqs(inv_freq: torch.Tensor, device=None) -> torch.Tensor:
    """The frequency table of the rotation: each of inv_freq (radians per
    position) in turns per position as a 64-bit binary fraction, as an int64
    tensor of the same bits on `device` (default: inv_freq's).  Made once;
    reads inv_freq on the host."""
    dev = inv_freq.device if device is None else device
    bits = [int(round(math.fmod(f, 2.0 * math.pi) / (2.0 * math.pi) * 2.0 ** 64)) % 2 ** 64
            for f in inv_freq.detach().double().cpu().tolist()]
    return torch.tensor([b - 2 ** 64 if b >= 2 ** 63 else b for b in bits], dtype=I64, device=dev)


class KVCache:
    """A paged cache: k, v [n_pages, Hkv, page_size, D] bf16, or float8_e4m3fn
    with k_scale, v_scale [n_pages, Hkv, page_size] float8_e8m0fnu.  Checked
    once here; the tensors must not be resized afterwards."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: Optional[torch.Tensor] = None,
                 v_scale: Optional[torch.Tensor] = None):
        if k.dim() != 4 or v.shape != k.shape or v.dtype != k.dtype:
            raise ValueError("KVCache: k and v must be [n_pages, Hkv, page_size, D] of one type, got %s %s and %s %s" % (
                tuple(k.shape), k.dtype, tuple(v.shape), v.dtype))
        if k.dtype not in (BF16, E4M3):
            raise TypeError("KVCache: k and v must be bfloat16 or float8_e4m3fn, got %s" % k.dtype)
        fp8 = k.dtype == E4M3
        if fp8 and (k_scale is None or v_scale is None):
            raise ValueError("KVCache: an e4m3 cache needs k_scale and v_scale")
        if not fp8 and (k_scale is not None or v_scale is not None):
            raise ValueError("KVCache: a bf16 cache has no scales")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.Hkv, self.page_size, self.D = k.shape
        self._c = GdnKvCache(_ptr(k, k.dtype, "k"), _ptr(v, v.dtype, "v"),
                             _shaped(k_scale, E8M0, k.shape[:3], "k_scale"),
                             _shaped(v_scale, E8M0, k.shape[:3], "v_scale"), self.n_pages, self.page_size, int(fp8))
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, dims, n_pages: int, page_size: int, dtype=BF16, device="cuda") -> "KVCache":
        """A zeroed cache of n_pages pages for these dims' heads."""
        shape = (int(n_pages), dims.Hkv, int(page_size), dims.D)
        k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != E4M3:
            return cls(k, v)
        return cls(k, v, *(torch.zeros(shape[:3], dtype=U8, device=device).view(E8M0) for _ in range(2)))


def _cache_args(dims, cache: KVCache, page_table, where: str):
    if cache.Hkv != dims.Hkv or cache.D != dims.D:
        raise ValueError("%s: the cache holds %d heads of %d channels, the dims say %d of %d" % (
            where, cache.Hkv, cache.D, dims.Hkv, dims.D))
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2 or page_table.shape[0] != dims.B:
        raise ValueError("%s: page_table must be a tensor [%d, width]" % (where, dims.B))
    return cache._ref, _ptr(page_table, I32, "page_table"), page_table.shape[1]


def _norm_args(dims, wq, wk, freqs):
    return (_shaped(wq, F32, (dims.D,), "wq"), _shaped(wk, F32, (dims.D,), "wk"),
            _shaped(freqs, I64, (dims.Drot // 2,), "freqs"))


# ---------------------------------------------------------------------------
# ABI-named calls (caller-allocated outputs)
# ---------------------------------------------------------------------------
def gdn_qk_norm_rope(dims, q, k, wq, wk, freqs, pos, mask, q_out, k_out, stream=None):
    B, T = dims.B, dims.T
    qs, ks = (B, T, dims.Hq, dims.D), (B, T, dims.Hkv, dims.D)
    _check(lib().gdn_qk_norm_rope(
        ctypes.byref(make_attn_dims(dims)), *_heads(q, qs, "q"), *_heads(k, ks, "k"), *_norm_args(dims, wq, wk, freqs),
        _shaped(pos, I32, (B, T), "pos"), _shaped(mask, U8, (B, T), "mask"), _shaped(q_out, BF16, qs, "q_out"),
        _shaped(k_out, BF16, ks, "k_out"), _stream(stream)), "gdn_qk_norm_rope")


def gdn_qk_norm_rope_backward_workspace_size(dims) -> int:
    return int(lib().gdn_qk_norm_rope_backward_workspace_size(ctypes.byref(make_attn_dims(dims))))


def gdn_qk_norm_rope_backward(dims, q, k, wq, wk, freqs, pos, mask, dq_out, dk_out, dq, dk, dwq, dwk, workspace,
                              stream=None):
    B, T = dims.B, dims.T
    qs, ks = (B, T, dims.Hq, dims.D), (B, T, dims.Hkv, dims.D)
    _check(lib().gdn_qk_norm_rope_backward(
        ctypes.byref(make_attn_dims(dims)), *_heads(q, qs, "q"), *_heads(k, ks, "k"), *_norm_args(dims, wq, wk, freqs),
        _shaped(pos, I32, (B, T), "pos"), _shaped(mask, U8, (B, T), "mask"), _shaped(dq_out, BF16, qs, "dq_out"),
        _shaped(dk_out, BF16, ks, "dk_out"), _shaped(dq, BF16, qs, "dq"), _shaped(dk, BF16, ks, "dk"),
        _shaped(dwq, F32, (dims.D,), "dwq"), _shaped(dwk, F32, (dims.D,), "dwk"), _ptr(workspace, U8, "workspace"),
        0 if workspace is None else workspace.numel(), _stream(stream)), "gdn_qk_norm_rope_backward")


def gdn_kv_append(dims, q, k, v, wq, wk, freqs, cache, page_table, pos, n_new, q_out, stream=None):
    B, T = dims.B, dims.T
    qs, ks = (B, T, dims.Hq, dims.D), (B, T, dims.Hkv, dims.D)
    _check(lib().gdn_kv_append(
        ctypes.byref(make_attn_dims(dims)), *_heads(q, qs, "q"), *_heads(k, ks, "k"), *_heads(v, ks, "v"),
        *_norm_args(dims, wq, wk, freqs), *_cache_args(dims, cache, page_table, "gdn_kv_append"),
        _shaped(pos, I32, (B,), "pos"), _shaped(n_new, I32, (B,), "n_new"), _shaped(q_out, BF16, qs, "q_out"),
        _stream(stream)), "gdn_kv_append")


def gdn_kv_read(dims, cache, page_table, start, n, k_out, v_out, stream=None):
    B, ks = dims.B, (dims.B, dims.T, dims.Hkv, dims.D)
    _check(lib().gdn_kv_read(
        ctypes.byref(make_attn_dims(dims)), *_cache_args(dims, cache, page_table, "gdn_kv_read"),
        _shaped(start, I32, (B,), "start"), _shaped(n, I32, (B,), "n"), _shaped(k_out, BF16, ks, "k_out"),
        _shaped(v_out, BF16, ks, "v_out"), _stream(stream)), "gdn_kv_read")


def gdn_attn_decode_workspace_size(dims) -> int:
    return int(lib().gdn_attn_decode_workspace_size(ctypes.byref(make_attn_dims(dims))))


def gdn_attn_decode(dims, q, cache, page_table, pos, n_new, gate, scale, out, lse, workspace, stream=None):
    B, T = dims.B, dims.T
    qs = (B, T, dims.Hq, dims.D)
    _check(lib().gdn_attn_decode(
        ctypes.byref(make_attn_dims(dims)), _shaped(q, BF16, qs, "q"),
        *_cache_args(dims, cache, page_table, "gdn_attn_decode"), _shaped(pos, I32, (B,), "pos"),
        _shaped(n_new, I32, (B,), "n_new"), *((None, 0, 0) if gate is None else _heads(gate, qs, "gate")),
        float(scale), _shaped(out, BF16, qs, "out"), _shaped(lse, F32, qs[:3], "lse"), _ptr(workspace, U8, "workspace"),
        0 if workspace is None else workspace.numel(), _stream(stream)), "gdn_attn_decode")


# ---------------------------------------------------------------------------
# allocating conveniences
# ---------------------------------------------------------------------------
def qk_norm_rope(dims, q, k, wq, wk, freqs, pos, mask=None, stream=None):
    """Returns (q_out, k_out): per-head norm and rotation of q and k."""
    q_out = _new((dims.B, dims.T, dims.Hq, dims.D), BF16, q.device, stream)
    k_out = _new((dims.B, dims.T, dims.Hkv, dims.D), BF16, q.device, stream)
    gdn_qk_norm_rope(dims, q, k, wq, wk, freqs, pos, mask, q_out, k_out, stream)
    return q_out, k_out


def qk_norm_rope_backward(dims, q, k, wq, wk, freqs, pos, dq_out, dk_out, mask=None, stream=None):
    """Gradients of qk_norm_rope; returns a dict dq, dk (bf16) and, with
    weights, dwq, dwk (f32)."""
    dev, norm = q.device, wq is not None
    out = {"dq": _new((dims.B, dims.T, dims.Hq, dims.D), BF16, dev, stream),
           "dk": _new((dims.B, dims.T, dims.Hkv, dims.D), BF16, dev, stream)}
    ws = None
    if norm:
        out["dwq"], out["dwk"] = (_new((dims.D,), F32, dev, stream) for _ in range(2))
        ws = _new((gdn_qk_norm_rope_backward_workspace_size(dims),), U8, dev, stream)
    gdn_qk_norm_rope_backward(dims, q, k, wq, wk, freqs, pos, mask, dq_out, dk_out, out["dq"], out["dk"],
                              out.get("dwq"), out.get("dwk"), ws, stream)
    return out


def kv_append(dims, q, k, v, wq, wk, freqs, cache, page_table, pos, n_new=None, stream=None):
    """New tokens into the cache (updated in place); returns the normed and
    rotated q [B, T, Hq, D]."""
    q_out = _new((dims.B, dims.T, dims.Hq, dims.D), BF16, q.device, stream)
    gdn_kv_append(dims, q, k, v, wq, wk, freqs, cache, page_table, pos, n_new, q_out, stream)
    return q_out


def kv_read(dims, cache, page_table, start, n=None, stream=None):
    """Positions start[b] .. start[b] + T - 1 as (k, v) bf16 [B, T, Hkv, D]."""
    k_out, v_out = (_new((dims.B, dims.T, dims.Hkv, dims.D), BF16, cache.k.device, stream) for _ in range(2))
    gdn_kv_read(dims, cache, page_table, start, n, k_out, v_out, stream)
    return k_out, v_out


def attn_decode(dims, q, cache, page_table, pos, n_new=None, gate=None, scale=None, return_lse=False, workspace=None,
                stream=None):
    """Attention of the T newest tokens per row over the cache; scale defaults
    to 1/sqrt(D).  Returns out [B, T, Hq, D], or (out, lse [B, T, Hq])."""
    dev = q.device
    out = _new((dims.B, dims.T, dims.Hq, dims.D), BF16, dev, stream)
    lse = _new((dims.B, dims.T, dims.Hq), F32, dev, stream) if return_lse else None
    if workspace is None:
        workspace = _new((gdn_attn_decode_workspace_size(dims),), U8, dev, stream)
    gdn_attn_decode(dims, q, cache, page_table, pos, n_new, gate, dims.D ** -0.5 if scale is None else scale, out, lse,
                    workspace, stream)
    return (out, lse) if return_lse else out
