"""Binding of the drafted tokens' verification in include/gdn.h.

A step of speculative decoding runs a window of the last token and the drafted
ones through the layers (gdn.decode_window, attn.attn_decode); verify() then
says how many of them stand and draws the next token, and its `keep` is what
gdn.decode_window commits.  As in ``attn``: argument checks and marshalling only.
"""
from __future__ import annotations

from .attn import _bind, _given, _handle


def gdn_spec_verify(target, draft, tokens, u, n, tokens_out, keep, stream=None):
    _given("gdn_spec_verify", tokens_out=tokens_out, keep=keep)
    _bind().spec_verify(target, draft, tokens, u, n, tokens_out, keep, _handle(stream))


def verify(target, tokens, u, draft=None, n=None, stream=None):
    """target f32 [B, T + 1, V], tokens i32 [B, T], u f32 [B, T + 1] in [0, 1),
    draft f32 [B, T, V] (None: tokens from a lookup), n i32 [B] drafted tokens of
    a row (None: T).  Returns (tokens_out i32 [B, T + 1]: the standing tokens, the
    next one, then -1; keep i32 [B]: how many of them are there)."""
    return _bind().spec_verify(target, draft, tokens, u, n, None, None, _handle(stream))
