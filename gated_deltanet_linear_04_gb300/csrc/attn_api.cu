// The C ABI of the full-attention layers (second half of include/gdn.h):
// argument validation and dispatch to the kernels.
#include <math.h>

#include "internal.h"

namespace gdn {
namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// A required pointer of `elems` elements: aligned and, when it has elements, not null.
bool ok(const void *p, size_t elems, uintptr_t align = 16) { return aligned(p, align) && (elems == 0 || p != nullptr); }

bool ok_heads(const HeadsIn &h, size_t elems) {
    return ok(h.p, elems) && h.ts >= 0 && h.hs >= 0 && h.ts % 8 == 0 && h.hs % 8 == 0;
}

gdn_status check(const gdn_attn_dims *d, AttnSizes *s) {
    if (d == nullptr) return GDN_ERR_INVALID_ARG;
    if (d->B < 0 || d->T < 0 || d->Hq <= 0 || d->Hkv <= 0 || d->D <= 0 || d->Drot < 0 || d->Drot > d->D)
        return GDN_ERR_INVALID_ARG;
    if (d->Hq % d->Hkv != 0 || (d->interleaved != 0 && d->interleaved != 1)) return GDN_ERR_INVALID_ARG;
    if (!(d->eps >= 0.0f) || !isfinite(d->eps)) return GDN_ERR_INVALID_ARG;
    if ((d->D != 64 && d->D != 128 && d->D != 256) || d->Drot % 16 != 0) return GDN_ERR_UNSUPPORTED;
    if (d->Hq / d->Hkv > 16 || d->Hq > 1024 || d->B > 65535) return GDN_ERR_UNSUPPORTED;
    *s = AttnSizes{d->B, d->T, d->Hq, d->Hkv, d->D, d->Drot, d->interleaved != 0, d->eps};
    return GDN_OK;
}

gdn_status check_cache(const AttnSizes &s, const gdn_kv_cache *c, const int32_t *table, int32_t width,
                       PagedCache *out) {
    if (c == nullptr || c->n_pages < 0 || width < 0) return GDN_ERR_INVALID_ARG;
    if (c->format != 0 && c->format != 1) return GDN_ERR_UNSUPPORTED;
    int shift = -1;
    for (int i = 4; i <= 8; ++i)
        if (c->page_size == 1 << i) shift = i;
    if (shift < 0) return GDN_ERR_UNSUPPORTED;
    if (c->n_pages > 0x7fffffffLL / ((long long)s.Hkv << shift)) return GDN_ERR_UNSUPPORTED;
    const size_t n = (size_t)c->n_pages;
    if (!ok(c->k, n) || !ok(c->v, n)) return GDN_ERR_INVALID_ARG;
    const bool fp8 = c->format == 1;
    if (fp8 ? (!ok(c->k_scale, n) || !ok(c->v_scale, n)) : (c->k_scale != nullptr || c->v_scale != nullptr))
        return GDN_ERR_INVALID_ARG;
    if (!ok(table, (size_t)s.B * width, 4)) return GDN_ERR_INVALID_ARG;
    *out = PagedCache{c->k, c->v, c->k_scale, c->v_scale, table, c->n_pages, width, c->page_size, shift, fp8};
    return GDN_OK;
}

// The norm weights come together or not at all; frequencies when something turns.
bool ok_norm(const AttnSizes &s, const float *wq, const float *wk, const uint64_t *freqs) {
    if ((wq == nullptr) != (wk == nullptr) || !aligned(wq, 16) || !aligned(wk, 16)) return false;
    return ok(freqs, (size_t)s.Drot);
}

// [rows, H, D] views of a prompt: tensor maps take no stride of 0.
gdn_status check_rows(const HeadsIn &h, long long rows, int H) {
    if (!ok_heads(h, (size_t)rows)) return GDN_ERR_INVALID_ARG;
    if (rows == 0) return GDN_OK;
    const long long most = 1LL << 39;   // (elements: a tensor map's strides are below 2^40 bytes)
    if ((rows > 1 && (h.ts == 0 || h.ts >= most)) || (H > 1 && (h.hs == 0 || h.hs >= most))) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_prompt(const gdn_attn_dims *d, int64_t q_rows, int64_t k_rows, PromptSizes *out) {
    AttnSizes s;
    const gdn_status st = check(d, &s);
    if (st != GDN_OK) return st;
    if (q_rows < 0 || k_rows < 0) return GDN_ERR_INVALID_ARG;
    if (q_rows > 0x7fff0000LL || k_rows > 0x7fff0000LL) return GDN_ERR_UNSUPPORTED;
    *out = PromptSizes{s.B, s.Hq, s.Hkv, s.D, q_rows, k_rows};
    return GDN_OK;
}

gdn_status check_prompt_heads(const PromptSizes &s, const HeadsIn &q, const HeadsIn &k, const HeadsIn &v, const HeadsIn &gate) {
    gdn_status st = check_rows(q, s.Nq, s.Hq);
    if (st == GDN_OK) st = check_rows(k, s.Nk, s.Hkv);
    if (st == GDN_OK) st = check_rows(v, s.Nk, s.Hkv);
    if (st == GDN_OK && gate.p != nullptr) st = check_rows(gate, s.Nq, s.Hq);
    return st;
}

bool ok_sequences(const PromptSizes &s, const PromptSeqs &q) {
    if (!ok(q.cu_q, 0, 4) || !ok(q.cu_k, 0, 4) || !ok(q.n_q, 0, 4) || !ok(q.n_k, 0, 4)) return false;
    return s.B == 0 || ((q.cu_q != nullptr || s.Nq % s.B == 0) && (q.cu_k != nullptr || s.Nk % s.B == 0));
}

gdn_status from(cudaError_t e) {
    if (e == cudaSuccess) return GDN_OK;
    return e == cudaErrorNotSupported ? GDN_ERR_UNSUPPORTED : GDN_ERR_CUDA;
}

}  // namespace
}  // namespace gdn

using gdn::AttnSizes;
using gdn::HeadsIn;
using gdn::PagedCache;

namespace {

// one axis: axes null, pos [B, T] or of the cache
bool ok_axes(const AttnSizes &s, const gdn::AxesIn &x, bool several, size_t n) {
    return !several || ((x.axis != nullptr || s.Drot == 0) && x.n >= 1 && x.n <= 8 && gdn::ok(x.pos, n, 4));
}

gdn_status norm_rope(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride, int64_t q_head_stride,
                     const uint16_t *k, int64_t k_token_stride, int64_t k_head_stride, const float *wq,
                     const float *wk, const uint64_t *freqs, const int32_t *pos, const uint8_t *mask, uint16_t *q_out,
                     uint16_t *k_out, gdn_stream stream, bool several, const gdn::AxesIn &axes) {
    AttnSizes s;
    gdn_status st = gdn::check(dims, &s);
    if (st != GDN_OK) return st;
    const size_t n = (size_t)s.B * s.T;
    const HeadsIn hq{q, q_token_stride, q_head_stride}, hk{k, k_token_stride, k_head_stride};
    if (!gdn::ok_heads(hq, n) || !gdn::ok_heads(hk, n) || !gdn::ok_norm(s, wq, wk, freqs) ||
        !gdn::ok(pos, several ? 0 : n, 4) || !ok_axes(s, axes, several, n) || !gdn::ok(q_out, n) || !gdn::ok(k_out, n))
        return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    return gdn::from(
        gdn::launch_qk_norm_rope(s, hq, hk, wq, wk, freqs, pos, mask, q_out, k_out, (cudaStream_t)stream,
                                 axes));
}

gdn_status norm_rope_backward(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                              int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride, int64_t k_head_stride,
                              const float *wq, const float *wk, const uint64_t *freqs, const int32_t *pos,
                              const uint8_t *mask, const uint16_t *dq_out, const uint16_t *dk_out, uint16_t *dq,
                              uint16_t *dk, float *dwq, float *dwk, void *workspace, size_t ws_bytes,
                              gdn_stream stream, bool several, const gdn::AxesIn &axes) {
    AttnSizes s;
    gdn_status st = gdn::check(dims, &s);
    if (st != GDN_OK) return st;
    const size_t n = (size_t)s.B * s.T;
    const HeadsIn hq{q, q_token_stride, q_head_stride}, hk{k, k_token_stride, k_head_stride};
    if (!gdn::ok_heads(hq, n) || !gdn::ok_heads(hk, n) || !gdn::ok_norm(s, wq, wk, freqs) ||
        !gdn::ok(pos, several ? 0 : n, 4) || !ok_axes(s, axes, several, n) || !gdn::ok(dq_out, n) ||
        !gdn::ok(dk_out, n) || !gdn::ok(dq, n) || !gdn::ok(dk, n))
        return GDN_ERR_INVALID_ARG;
    const bool norm = wq != nullptr;
    if (!gdn::ok(dwq, norm) || !gdn::ok(dwk, norm) || (!norm && (dwq != nullptr || dwk != nullptr)))
        return GDN_ERR_INVALID_ARG;
    cudaStream_t cs = (cudaStream_t)stream;
    if (n == 0) {
        // no tokens: the weights' gradients are empty sums
        if (!norm) return GDN_OK;
        cudaError_t e = cudaMemsetAsync(dwq, 0, (size_t)s.D * sizeof(float), cs);
        if (e == cudaSuccess) e = cudaMemsetAsync(dwk, 0, (size_t)s.D * sizeof(float), cs);
        return gdn::from(e);
    }
    if (norm && (!gdn::ok(workspace, 1) || ws_bytes < gdn::qk_norm_rope_backward_workspace(s)))
        return GDN_ERR_INVALID_ARG;
    return gdn::from(gdn::launch_qk_norm_rope_backward(s, hq, hk, wq, wk, freqs, pos, mask, dq_out, dk_out, dq, dk,
                                                       dwq, dwk, workspace, cs, axes));
}

gdn_status kv_append(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride, int64_t q_head_stride,
                     const uint16_t *k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t *v,
                     int64_t v_token_stride, int64_t v_head_stride, const float *wq, const float *wk,
                     const uint64_t *freqs, const gdn_kv_cache *cache, const int32_t *page_table, int32_t table_width,
                     const int32_t *pos, const int32_t *n_new, uint16_t *q_out, gdn_stream stream, bool several,
                     const gdn::AxesIn &axes) {
    AttnSizes s;
    PagedCache c;
    gdn_status st = gdn::check(dims, &s);
    if (st == GDN_OK) st = gdn::check_cache(s, cache, page_table, table_width, &c);
    if (st != GDN_OK) return st;
    const size_t n = (size_t)s.B * s.T;
    const HeadsIn hq{q, q_token_stride, q_head_stride}, hk{k, k_token_stride, k_head_stride},
        hv{v, v_token_stride, v_head_stride};
    if (!gdn::ok_heads(hq, n) || !gdn::ok_heads(hk, n) || !gdn::ok_heads(hv, n) ||
        !gdn::ok_norm(s, wq, wk, freqs) || !gdn::ok(pos, n, 4) || !gdn::ok(n_new, 0, 4) || !gdn::ok(q_out, n) ||
        !ok_axes(s, axes, several, n))
        return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    unsigned *err = gdn::device_error_word();
    if (err == nullptr) return GDN_ERR_CUDA;
    return gdn::from(
        gdn::launch_kv_append(s, hq, hk, hv, wq, wk, freqs, c, pos, n_new, q_out, err, (cudaStream_t)stream, axes));
}

}  // namespace

extern "C" {

gdn_status gdn_qk_norm_rope(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                            int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride, int64_t k_head_stride,
                            const float *wq, const float *wk, const uint64_t *freqs, const int32_t *pos,
                            const uint8_t *mask, uint16_t *q_out, uint16_t *k_out, gdn_stream stream) {
    return norm_rope(dims, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, wq, wk, freqs, pos,
                     mask, q_out, k_out, stream, false, gdn::AxesIn());
}

gdn_status gdn_qk_norm_rope_axes(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                 int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                 int64_t k_head_stride, const float *wq, const float *wk, const uint64_t *freqs,
                                 const uint8_t *axes, int32_t n_axes, const int32_t *pos, const uint8_t *mask,
                                 uint16_t *q_out, uint16_t *k_out, gdn_stream stream) {
    return norm_rope(dims, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, wq, wk, freqs, nullptr,
                     mask, q_out, k_out, stream, true, gdn::AxesIn{axes, n_axes, pos});
}

size_t gdn_qk_norm_rope_backward_workspace_size(const gdn_attn_dims *dims) {
    AttnSizes s;
    if (gdn::check(dims, &s) != GDN_OK) return 0;
    return gdn::qk_norm_rope_backward_workspace(s);
}

gdn_status gdn_qk_norm_rope_backward(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                     int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                     int64_t k_head_stride, const float *wq, const float *wk, const uint64_t *freqs,
                                     const int32_t *pos, const uint8_t *mask, const uint16_t *dq_out,
                                     const uint16_t *dk_out, uint16_t *dq, uint16_t *dk, float *dwq, float *dwk,
                                     void *workspace, size_t ws_bytes, gdn_stream stream) {
    return norm_rope_backward(dims, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, wq, wk, freqs,
                              pos, mask, dq_out, dk_out, dq, dk, dwq, dwk, workspace, ws_bytes, stream, false,
                              gdn::AxesIn());
}

gdn_status gdn_qk_norm_rope_axes_backward(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                          int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                          int64_t k_head_stride, const float *wq, const float *wk,
                                          const uint64_t *freqs, const uint8_t *axes, int32_t n_axes,
                                          const int32_t *pos, const uint8_t *mask, const uint16_t *dq_out,
                                          const uint16_t *dk_out, uint16_t *dq, uint16_t *dk, float *dwq, float *dwk,
                                          void *workspace, size_t ws_bytes, gdn_stream stream) {
    return norm_rope_backward(dims, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, wq, wk, freqs,
                              nullptr, mask, dq_out, dk_out, dq, dk, dwq, dwk, workspace, ws_bytes, stream, true,
                              gdn::AxesIn{axes, n_axes, pos});
}

gdn_status gdn_kv_append(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride, int64_t q_head_stride,
                         const uint16_t *k, int64_t k_token_stride, int64_t k_head_stride, const uint16_t *v,
                         int64_t v_token_stride, int64_t v_head_stride, const float *wq, const float *wk,
                         const uint64_t *freqs, const gdn_kv_cache *cache, const int32_t *page_table,
                         int32_t table_width, const int32_t *pos, const int32_t *n_new, uint16_t *q_out,
                         gdn_stream stream) {
    return kv_append(dims, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, v, v_token_stride,
                     v_head_stride, wq, wk, freqs, cache, page_table, table_width, pos, n_new, q_out, stream, false,
                     gdn::AxesIn());
}

gdn_status gdn_kv_append_axes(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                              int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride, int64_t k_head_stride,
                              const uint16_t *v, int64_t v_token_stride, int64_t v_head_stride, const float *wq,
                              const float *wk, const uint64_t *freqs, const uint8_t *axes, int32_t n_axes,
                              const int32_t *rope_pos, const gdn_kv_cache *cache, const int32_t *page_table,
                              int32_t table_width, const int32_t *pos, const int32_t *n_new, uint16_t *q_out,
                              gdn_stream stream) {
    return kv_append(dims, q, q_token_stride, q_head_stride, k, k_token_stride, k_head_stride, v, v_token_stride,
                     v_head_stride, wq, wk, freqs, cache, page_table, table_width, pos, n_new, q_out, stream, true,
                     gdn::AxesIn{axes, n_axes, rope_pos});
}

gdn_status gdn_kv_read(const gdn_attn_dims *dims, const gdn_kv_cache *cache, const int32_t *page_table,
                       int32_t table_width, const int32_t *start, const int32_t *n_valid, uint16_t *k_out,
                       uint16_t *v_out, gdn_stream stream) {
    AttnSizes s;
    PagedCache c;
    gdn_status st = gdn::check(dims, &s);
    if (st == GDN_OK) st = gdn::check_cache(s, cache, page_table, table_width, &c);
    if (st != GDN_OK) return st;
    const size_t n = (size_t)s.B * s.T;
    if (!gdn::ok(start, n, 4) || !gdn::ok(n_valid, 0, 4) || !gdn::ok(k_out, n) || !gdn::ok(v_out, n))
        return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    unsigned *err = gdn::device_error_word();
    if (err == nullptr) return GDN_ERR_CUDA;
    return gdn::from(gdn::launch_kv_read(s, c, start, n_valid, k_out, v_out, err, (cudaStream_t)stream));
}

size_t gdn_attn_decode_workspace_size(const gdn_attn_dims *dims) {
    AttnSizes s;
    if (gdn::check(dims, &s) != GDN_OK || s.T < 1 || s.T > 8) return 0;
    return gdn::attn_decode_workspace(s);
}

gdn_status gdn_attn_decode(const gdn_attn_dims *dims, const uint16_t *q, const gdn_kv_cache *cache,
                           const int32_t *page_table, int32_t table_width, const int32_t *pos, const int32_t *n_new,
                           const uint16_t *gate, int64_t gate_token_stride, int64_t gate_head_stride, float scale,
                           uint16_t *out, float *lse, void *workspace, size_t ws_bytes, gdn_stream stream) {
    AttnSizes s;
    PagedCache c;
    gdn_status st = gdn::check(dims, &s);
    if (st == GDN_OK) st = gdn::check_cache(s, cache, page_table, table_width, &c);
    if (st != GDN_OK) return st;
    if (s.T < 1 || s.T > 8) return GDN_ERR_UNSUPPORTED;
    const size_t n = (size_t)s.B;
    const HeadsIn hg{gate, gate_token_stride, gate_head_stride};
    if (!gdn::ok(q, n) || !gdn::ok(pos, n, 4) || !gdn::ok(n_new, 0, 4) || !gdn::ok_heads(hg, 0) ||
        !gdn::ok(out, n) || !gdn::ok(lse, 0, 4) || !isfinite(scale))
        return GDN_ERR_INVALID_ARG;
    if (n == 0) return GDN_OK;
    if (!gdn::ok(workspace, 1) || ws_bytes < gdn::attn_decode_workspace(s)) return GDN_ERR_INVALID_ARG;
    unsigned *err = gdn::device_error_word();
    if (err == nullptr) return GDN_ERR_CUDA;
    return gdn::from(gdn::launch_attn_decode(s, q, c, pos, n_new, hg, scale, out, lse, workspace, err,
                                             (cudaStream_t)stream));
}

size_t gdn_attn_prefill_workspace_size(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows) {
    gdn::PromptSizes s;
    if (gdn::check_prompt(dims, q_rows, k_rows, &s) != GDN_OK) return 0;
    return gdn::attn_prefill_workspace(s);
}

gdn_status gdn_attn_prefill(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows, const uint16_t *q,
                            int64_t q_token_stride, int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                            int64_t k_head_stride, const uint16_t *v, int64_t v_token_stride, int64_t v_head_stride,
                            const int32_t *cu_q, const int32_t *cu_k, const int32_t *n_q, const int32_t *n_k,
                            const uint16_t *gate, int64_t gate_token_stride, int64_t gate_head_stride, float scale,
                            uint16_t *out, float *lse, void *workspace, size_t ws_bytes, gdn_stream stream) {
    gdn::PromptSizes s;
    gdn_status st = gdn::check_prompt(dims, q_rows, k_rows, &s);
    if (st != GDN_OK) return st;
    const HeadsIn hq{q, q_token_stride, q_head_stride}, hk{k, k_token_stride, k_head_stride},
        hv{v, v_token_stride, v_head_stride}, hg{gate, gate_token_stride, gate_head_stride};
    const gdn::PromptSeqs seqs{cu_q, cu_k, n_q, n_k};
    st = gdn::check_prompt_heads(s, hq, hk, hv, hg);
    if (st != GDN_OK) return st;
    if (!gdn::ok_sequences(s, seqs) || !gdn::ok(out, (size_t)s.Nq) || !gdn::ok(lse, 0, 4) || !isfinite(scale))
        return GDN_ERR_INVALID_ARG;
    if (s.Nq == 0 || s.B == 0) return GDN_OK;
    if (!gdn::ok(workspace, 1) || ws_bytes < gdn::attn_prefill_workspace(s)) return GDN_ERR_INVALID_ARG;
    unsigned *err = gdn::device_error_word();
    if (err == nullptr) return GDN_ERR_CUDA;
    return gdn::from(gdn::launch_attn_prefill(s, hq, hk, hv, seqs, hg, scale, out, lse, workspace, err,
                                              (cudaStream_t)stream));
}

size_t gdn_attn_prefill_backward_workspace_size(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows, int32_t gated) {
    gdn::PromptSizes s;
    if (gdn::check_prompt(dims, q_rows, k_rows, &s) != GDN_OK) return 0;
    return gdn::attn_prefill_backward_workspace(s, gated != 0);
}

gdn_status gdn_attn_prefill_backward(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows, const uint16_t *q,
                                     int64_t q_token_stride, int64_t q_head_stride, const uint16_t *k,
                                     int64_t k_token_stride, int64_t k_head_stride, const uint16_t *v,
                                     int64_t v_token_stride, int64_t v_head_stride, const int32_t *cu_q,
                                     const int32_t *cu_k, const int32_t *n_q, const int32_t *n_k, const uint16_t *gate,
                                     int64_t gate_token_stride, int64_t gate_head_stride, float scale,
                                     const uint16_t *out, const float *lse, const uint16_t *dout, uint16_t *dq,
                                     uint16_t *dk, uint16_t *dv, uint16_t *dgate, void *workspace, size_t ws_bytes,
                                     gdn_stream stream) {
    gdn::PromptSizes s;
    gdn_status st = gdn::check_prompt(dims, q_rows, k_rows, &s);
    if (st != GDN_OK) return st;
    const HeadsIn hq{q, q_token_stride, q_head_stride}, hk{k, k_token_stride, k_head_stride},
        hv{v, v_token_stride, v_head_stride}, hg{gate, gate_token_stride, gate_head_stride};
    const gdn::PromptSeqs seqs{cu_q, cu_k, n_q, n_k};
    st = gdn::check_prompt_heads(s, hq, hk, hv, hg);
    if (st != GDN_OK) return st;
    const size_t nq = (size_t)s.Nq, nk = (size_t)s.Nk;
    if (!gdn::ok_sequences(s, seqs) || !gdn::ok(out, nq) || !gdn::ok(lse, nq, 4) || !gdn::ok(dout, nq) ||
        !gdn::ok(dq, nq) || !gdn::ok(dk, nk) || !gdn::ok(dv, nk) || !isfinite(scale))
        return GDN_ERR_INVALID_ARG;
    if (gate != nullptr ? !gdn::ok(dgate, nq) : dgate != nullptr) return GDN_ERR_INVALID_ARG;
    if ((nq == 0 && nk == 0) || s.B == 0) return GDN_OK;
    if (!gdn::ok(workspace, 1) || ws_bytes < gdn::attn_prefill_backward_workspace(s, gate != nullptr))
        return GDN_ERR_INVALID_ARG;
    unsigned *err = gdn::device_error_word();
    if (err == nullptr) return GDN_ERR_CUDA;
    return gdn::from(gdn::launch_attn_prefill_backward(s, hq, hk, hv, seqs, hg, scale, out, lse, dout, dq, dk, dv, dgate,
                                                       workspace, err, (cudaStream_t)stream));
}

}  // extern "C"
