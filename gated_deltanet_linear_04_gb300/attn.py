"""Binding of the full-attention operators of include/gdn.h.

The layers that stand between the Gated DeltaNet layers of a hybrid model:
per-head norm and rotation of queries and keys (and its gradients), a paged
key-value cache written and read back in bf16 or e4m3, and the attention of
new tokens over it.  As in ``gdn``: argument checks and marshalling only (here
in a small extension module, csrc/attn_bind.cpp), the functions named like the
ABI take caller-allocated outputs, the short names allocate them, a non-zero
status raises ``GdnError``, and work runs on ``stream`` (default: torch's
current stream).

q, k, v and gate may be views [B, T, heads, D] of a packed projection: the
channels of a head dense, one stride from token to token over all rows and one
from head to head, both multiples of 8 elements.  All other tensors are dense.
"""
from __future__ import annotations

import ctypes
import importlib.util
import math
import os
from typing import Optional

import torch

from .gdn import BF16, U8, GdnAttnDims, GdnError, GdnKvCache, _ptr, _stream, lib
from .workloads import AttnDims

I64 = torch.int64
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu

BIND_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_lib", "_attn_bind.so")
_bind_module = None


def _bind():
    """The extension module.  Raises if it has not been built."""
    global _bind_module
    if _bind_module is None:
        lib()
        if not os.path.exists(BIND_PATH):
            raise RuntimeError("_attn_bind.so is not built (%s); run __graft_entry__.build() first" % BIND_PATH)
        spec = importlib.util.spec_from_file_location("_attn_bind", BIND_PATH)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        m.set_error(GdnError)
        _bind_module = m
    return _bind_module


def make_attn_dims(d) -> GdnAttnDims:
    return GdnAttnDims(int(d.B), int(d.T), int(d.Hq), int(d.Hkv), int(d.D), int(d.Drot), int(bool(d.interleaved)),
                       float(d.eps))


def _dims(d) -> GdnAttnDims:
    """The ABI's struct of the dims; made once for each (immutable) AttnDims."""
    if type(d) is not AttnDims:
        return make_attn_dims(d)
    c = d.__dict__.get("_abi")
    if c is None:
        c = d.__dict__["_abi"] = make_attn_dims(d)
    return c


def _handle(stream) -> Optional[int]:
    return None if stream is None else (_stream(stream) or 0)


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


def rope_axes(sections, cyclic: bool = False, device=None) -> torch.Tensor:
    """The axis of each rotated pair (u8 [sum of sections]): sections[i] pairs
    turn with axis i, one axis after the other, or in turn (0, 1, 2, 0, 1, ...;
    an axis whose pairs are used up is passed over)."""
    left = [int(n) for n in sections]
    if not 1 <= len(left) <= 8 or min(left) < 0:
        raise ValueError("rope_axes: 1 to 8 sections of 0 or more pairs, got %s" % (left,))
    if not cyclic:
        pairs = [i for i, n in enumerate(left) for _ in range(n)]
    else:
        pairs = [i for k in range(max(left)) for i, n in enumerate(left) if k < n]
    return torch.tensor(pairs, dtype=U8, device=device)


class _CacheRecord(ctypes.Structure):
    _fields_ = [("c", GdnKvCache), ("Hkv", ctypes.c_int32), ("D", ctypes.c_int32), ("device", ctypes.c_int32)]


class KVCache:
    """A paged cache: k, v [n_pages, Hkv, page_size, D] bf16, or float8_e4m3fn
    with k_scale, v_scale [n_pages, Hkv, page_size] float8_e8m0fnu, all on one
    device.  Checked once here; the tensors must not be resized afterwards."""

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
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and t.shape != k.shape[:3]:
                raise ValueError("KVCache: %s must have shape %s, got %s" % (name, tuple(k.shape[:3]), tuple(t.shape)))
        for name, t in (("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t is not None and t.device != k.device:
                raise ValueError("KVCache: %s is on %s, k on %s" % (name, t.device, k.device))
        self._c = _CacheRecord(GdnKvCache(_ptr(k, k.dtype, "k"), _ptr(v, v.dtype, "v"), _ptr(k_scale, E8M0, "k_scale"),
                                          _ptr(v_scale, E8M0, "v_scale"), self.n_pages, self.page_size, int(fp8)),
                               self.Hkv, self.D, k.device.index if k.is_cuda and k.numel() else -1)

    @classmethod
    def empty(cls, dims, n_pages: int, page_size: int, dtype=BF16, device="cuda") -> "KVCache":
        """A zeroed cache of n_pages pages for these dims' heads."""
        shape = (int(n_pages), dims.Hkv, int(page_size), dims.D)
        k, v = (torch.zeros(shape, dtype=dtype, device=device) for _ in range(2))
        if dtype != E4M3:
            return cls(k, v)
        return cls(k, v, *(torch.zeros(shape[:3], dtype=U8, device=device).view(E8M0) for _ in range(2)))


_at = ctypes.addressof


# ---------------------------------------------------------------------------
# ABI-named calls (caller-allocated outputs)
# ---------------------------------------------------------------------------
def _given(where: str, **outputs):
    for name, t in outputs.items():
        if t is None:
            raise TypeError("%s: %s must be a torch.Tensor" % (where, name))


def gdn_qk_norm_rope(dims, q, k, wq, wk, freqs, pos, mask, q_out, k_out, stream=None):
    _given("gdn_qk_norm_rope", q_out=q_out, k_out=k_out)
    c = _dims(dims)
    _bind().qk_norm_rope(_at(c), q, k, wq, wk, freqs, pos, mask, q_out, k_out, _handle(stream))


def gdn_qk_norm_rope_backward_workspace_size(dims) -> int:
    return int(lib().gdn_qk_norm_rope_backward_workspace_size(ctypes.byref(_dims(dims))))


def gdn_qk_norm_rope_backward(dims, q, k, wq, wk, freqs, pos, mask, dq_out, dk_out, dq, dk, dwq, dwk, workspace,
                              stream=None):
    _given("gdn_qk_norm_rope_backward", dq=dq, dk=dk)
    if wq is not None:
        _given("gdn_qk_norm_rope_backward", dwq=dwq, dwk=dwk, workspace=workspace)
    c = _dims(dims)
    _bind().qk_norm_rope_backward(_at(c), q, k, wq, wk, freqs, pos, mask, dq_out, dk_out, dq, dk, dwq, dwk, workspace,
                                  _handle(stream))


def gdn_kv_append(dims, q, k, v, wq, wk, freqs, cache, page_table, pos, n_new, q_out, stream=None):
    _given("gdn_kv_append", q_out=q_out)
    c = _dims(dims)
    _bind().kv_append(_at(c), q, k, v, wq, wk, freqs, _at(cache._c), page_table, pos, n_new, q_out, _handle(stream))


def gdn_kv_read(dims, cache, page_table, start, n, k_out, v_out, stream=None):
    _given("gdn_kv_read", k_out=k_out, v_out=v_out)
    c = _dims(dims)
    _bind().kv_read(_at(c), _at(cache._c), page_table, start, n, k_out, v_out, _handle(stream))


def gdn_attn_decode_workspace_size(dims) -> int:
    return int(lib().gdn_attn_decode_workspace_size(ctypes.byref(_dims(dims))))


def gdn_attn_decode(dims, q, cache, page_table, pos, n_new, gate, scale, out, lse, workspace, stream=None):
    _given("gdn_attn_decode", out=out, workspace=workspace)
    c = _dims(dims)
    _bind().attn_decode(_at(c), q, _at(cache._c), page_table, pos, n_new, gate, scale, out, lse, False, workspace,
                        _handle(stream))


def gdn_qk_norm_rope_axes(dims, q, k, wq, wk, freqs, axes, pos, mask, q_out, k_out, stream=None):
    _given("gdn_qk_norm_rope_axes", q_out=q_out, k_out=k_out)
    c = _dims(dims)
    _bind().qk_norm_rope_axes(_at(c), q, k, wq, wk, freqs, axes, pos, mask, q_out, k_out, _handle(stream))


def gdn_qk_norm_rope_axes_backward(dims, q, k, wq, wk, freqs, axes, pos, mask, dq_out, dk_out, dq, dk, dwq, dwk, workspace,
                                   stream=None):
    _given("gdn_qk_norm_rope_axes_backward", dq=dq, dk=dk)
    if wq is not None:
        _given("gdn_qk_norm_rope_axes_backward", dwq=dwq, dwk=dwk, workspace=workspace)
    c = _dims(dims)
    _bind().qk_norm_rope_axes_backward(_at(c), q, k, wq, wk, freqs, axes, pos, mask, dq_out, dk_out, dq, dk, dwq, dwk,
                                       workspace, _handle(stream))


def gdn_kv_append_axes(dims, q, k, v, wq, wk, freqs, axes, rope_pos, cache, page_table, pos, n_new, q_out, stream=None):
    _given("gdn_kv_append_axes", q_out=q_out)
    c = _dims(dims)
    _bind().kv_append_axes(_at(c), q, k, v, wq, wk, freqs, axes, rope_pos, _at(cache._c), page_table, pos, n_new, q_out,
                           _handle(stream))


def gdn_attn_prefill_workspace_size(dims, q_rows, k_rows) -> int:
    return int(lib().gdn_attn_prefill_workspace_size(ctypes.byref(_dims(dims)), int(q_rows), int(k_rows)))


def gdn_attn_prefill(dims, q, k, v, cu_q, cu_k, n_q, n_k, gate, scale, out, lse, workspace, stream=None):
    _given("gdn_attn_prefill", out=out, workspace=workspace)
    c = _dims(dims)
    _bind().attn_prefill(_at(c), q, k, v, cu_q, cu_k, n_q, n_k, gate, scale, out, lse, False, workspace, _handle(stream))


def gdn_attn_prefill_backward_workspace_size(dims, q_rows, k_rows, gated) -> int:
    return int(lib().gdn_attn_prefill_backward_workspace_size(ctypes.byref(_dims(dims)), int(q_rows), int(k_rows),
                                                              int(bool(gated))))


def gdn_attn_prefill_backward(dims, q, k, v, cu_q, cu_k, n_q, n_k, gate, scale, out, lse, dout, dq, dk, dv, dgate,
                              workspace, stream=None):
    _given("gdn_attn_prefill_backward", dq=dq, dk=dk, dv=dv, workspace=workspace)
    if gate is not None:
        _given("gdn_attn_prefill_backward", dgate=dgate)
    c = _dims(dims)
    _bind().attn_prefill_backward(_at(c), q, k, v, cu_q, cu_k, n_q, n_k, gate, scale, out, lse, dout, dq, dk, dv, dgate,
                                  workspace, _handle(stream))


# ---------------------------------------------------------------------------
# allocating conveniences
# ---------------------------------------------------------------------------
def qk_norm_rope(dims, q, k, wq, wk, freqs, pos, mask=None, stream=None):
    """Returns (q_out, k_out): per-head norm and rotation of q and k."""
    c = _dims(dims)
    return _bind().qk_norm_rope(_at(c), q, k, wq, wk, freqs, pos, mask, None, None, _handle(stream))


def qk_norm_rope_backward(dims, q, k, wq, wk, freqs, pos, dq_out, dk_out, mask=None, stream=None):
    """Gradients of qk_norm_rope; returns a dict dq, dk (bf16) and, with
    weights, dwq, dwk (f32)."""
    c = _dims(dims)
    dq, dk, dwq, dwk = _bind().qk_norm_rope_backward(_at(c), q, k, wq, wk, freqs, pos, mask, dq_out, dk_out, None, None,
                                                     None, None, None, _handle(stream))
    return {"dq": dq, "dk": dk} if dwq is None else {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def kv_append(dims, q, k, v, wq, wk, freqs, cache, page_table, pos, n_new=None, stream=None):
    """New tokens into the cache (updated in place); returns the normed and
    rotated q [B, T, Hq, D]."""
    c = _dims(dims)
    return _bind().kv_append(_at(c), q, k, v, wq, wk, freqs, _at(cache._c), page_table, pos, n_new, None,
                             _handle(stream))


def kv_read(dims, cache, page_table, start, n=None, stream=None):
    """Positions start[b] .. start[b] + T - 1 as (k, v) bf16 [B, T, Hkv, D]."""
    c = _dims(dims)
    return _bind().kv_read(_at(c), _at(cache._c), page_table, start, n, None, None, _handle(stream))


def attn_decode(dims, q, cache, page_table, pos, n_new=None, gate=None, scale=None, return_lse=False, workspace=None,
                stream=None):
    """Attention of the T newest tokens per row over the cache; scale defaults
    to 1/sqrt(D).  Returns out [B, T, Hq, D], or (out, lse [B, T, Hq])."""
    c = _dims(dims)
    return _bind().attn_decode(_at(c), q, _at(cache._c), page_table, pos, n_new, gate,
                               dims.D ** -0.5 if scale is None else scale, None, None, bool(return_lse), workspace,
                               _handle(stream))


def qk_norm_rope_axes(dims, q, k, wq, wk, freqs, axes, pos, mask=None, stream=None):
    """qk_norm_rope with pos [axes, B, T], each pair turning with its own axis
    (axes: rope_axes); returns (q_out, k_out)."""
    c = _dims(dims)
    return _bind().qk_norm_rope_axes(_at(c), q, k, wq, wk, freqs, axes, pos, mask, None, None, _handle(stream))


def qk_norm_rope_axes_backward(dims, q, k, wq, wk, freqs, axes, pos, dq_out, dk_out, mask=None, stream=None):
    """Gradients of qk_norm_rope_axes, as qk_norm_rope_backward's."""
    c = _dims(dims)
    dq, dk, dwq, dwk = _bind().qk_norm_rope_axes_backward(_at(c), q, k, wq, wk, freqs, axes, pos, mask, dq_out, dk_out, None,
                                                          None, None, None, None, _handle(stream))
    return {"dq": dq, "dk": dk} if dwq is None else {"dq": dq, "dk": dk, "dwq": dwq, "dwk": dwk}


def kv_append_axes(dims, q, k, v, wq, wk, freqs, axes, rope_pos, cache, page_table, pos, n_new=None, stream=None):
    """kv_append with rotary positions rope_pos [axes, B, T]; pos [B] says where
    in the cache the new tokens go."""
    c = _dims(dims)
    return _bind().kv_append_axes(_at(c), q, k, v, wq, wk, freqs, axes, rope_pos, _at(cache._c), page_table, pos, n_new, None,
                                  _handle(stream))


def attn_prefill(dims, q, k, v, cu_q=None, cu_k=None, n_q=None, n_k=None, gate=None, scale=None, return_lse=False,
                 workspace=None, stream=None):
    """Causal attention of dims.B whole prompts, or of new tokens after a kept
    prefix; the last query of a sequence sees its last key.  q [B, T, Hq, D] and
    k, v [B, Tk, Hkv, D] with lengths n_q, n_k (None: all), or packed: q [N, Hq,
    D] with offsets cu_q [B + 1], k, v [M, Hkv, D] with cu_k (None: cu_q).  Returns
    out shaped as q, or (out, lse).  Rows in no slot (before cu_q[0], from cu_q[B]
    on; all rows, if the offsets are not in order: GDN_ERR_BAD_OFFSETS) are not
    written: in these new tensors they hold whatever their memory did.  Where such
    rows are read, hand tensors of your own to gdn_attn_prefill."""
    c = _dims(dims)
    return _bind().attn_prefill(_at(c), q, k, v, cu_q, cu_k, n_q, n_k, gate, dims.D ** -0.5 if scale is None else scale,
                                None, None, bool(return_lse), workspace, _handle(stream))


def attn_prefill_backward(dims, q, k, v, out, lse, dout, cu_q=None, cu_k=None, n_q=None, n_k=None, gate=None, scale=None,
                          workspace=None, stream=None):
    """Gradients of attn_prefill, from its inputs, its results out and lse, and
    the gradient of out; returns a dict dq, dk, dv and, with a gate, dgate (bf16).
    Rows in no slot are not written, as in attn_prefill: mask them, or hand zeroed
    tensors to gdn_attn_prefill_backward, before their sum goes into another
    gradient (a norm's weights)."""
    c = _dims(dims)
    dq, dk, dv, dgate = _bind().attn_prefill_backward(
        _at(c), q, k, v, cu_q, cu_k, n_q, n_k, gate, dims.D ** -0.5 if scale is None else scale, out, lse, dout, None, None,
        None, None, workspace, _handle(stream))
    return {"dq": dq, "dk": dk, "dv": dv} if dgate is None else {"dq": dq, "dk": dk, "dv": dv, "dgate": dgate}
