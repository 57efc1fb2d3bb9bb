/*
 * gdn.h -- C ABI of the GB300 (sm_103a) Gated DeltaNet layer core.
 *
 * The core is the linear-attention block of Qwen3-Next / Qwen3.5-style models
 * as defined by "mlex 0.1.2, src/models/gated_delta.rs" (GatedDeltaNet::load and
 * GatedDeltaNet::forward) and by "mlx-bun 0.4.0 -> 1.0.0,
 * package/src/model/qwen3-delta.ts" (the numerics table at its head, the
 * gated_delta_step kernel and its masked specialization, computeG,
 * gatedDeltaUpdate):
 *
 *   conv window   X = [conv_state || qkv] along time, conv_state' = last K-1 rows
 *   conv + SiLU   u[t,c] = sum_j w[c,j] X[t+j,c] (tap K-1 = current token); x = u*sigmoid(u)
 *   q/k norm      q = rms(x_q)/Dk, k = rms(x_k)/sqrt(Dk), v = x_v; rms(x) = x/sqrt(mean(x^2)+eps)
 *   gates         g = exp(-exp(A_log) * softplus(a + dt_bias)), beta = sigmoid(b)
 *   recurrence    per (b, hv), hk = hv / (Hv/Hk):  S <- g S;  delta = beta (v - S k);
 *                 S <- S + delta k^T;  y = S q          (S is [Dv, Dk], f32)
 *   mask          a step with mask 0 writes zero y (and zero q/k/v), does not enter
 *                 the conv window and leaves both states untouched.
 *
 * Conventions shared by every entry point
 *   - Memory: every pointer is a DEVICE pointer owned by the caller.  The library
 *     allocates nothing and keeps no state between calls except one device error
 *     word per device (see gdn_device_status).
 *   - Types: "bf16" buffers hold bfloat16 bit patterns (uint16_t); "f32" is IEEE
 *     single.  Every tensor is dense and row-major with the shape given.
 *   - Alignment: every tensor pointer must be 16-byte aligned, else
 *     GDN_ERR_INVALID_ARG.
 *   - Streams: work is enqueued on `stream` (a cudaStream_t; NULL = legacy
 *     default stream) and the call returns without waiting.  Argument errors are
 *     reported before anything is enqueued; GDN_ERR_CUDA reports a launch error.
 *   - Supported sizes: Dk, Dv in {32, 64, 128}; Hv % Hk == 0; 2 <= K <= 4;
 *     B, T >= 0 (a zero size is a no-op).  Others give GDN_ERR_UNSUPPORTED.
 *   - Channel order of qkv / conv_state / conv_w: C = 2*Hk*Dk + Hv*Dv channels,
 *     q heads [0, Hk*Dk), k heads [Hk*Dk, 2*Hk*Dk), v heads [2*Hk*Dk, C), each
 *     head's channels contiguous.
 *
 * The second half of this header (gdn_attn_dims on) holds the core of the
 * full-attention layers that stand between the Gated DeltaNet layers of those
 * models: per-head q/k norm with the rotary embedding, a paged key-value
 * cache and the attention of new tokens over it.  Its conventions are the ones
 * above except where it says otherwise.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Exported symbols keep default visibility even when the library is built
 * with hidden visibility. */
#if defined(__GNUC__)
#define GDN_API __attribute__((visibility("default")))
#else
#define GDN_API
#endif

/* A cudaStream_t, spelled without the CUDA headers. */
typedef struct CUstream_st *gdn_stream;

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID_ARG = 1,   /* null / misaligned pointer, negative size, Hv % Hk != 0 */
    GDN_ERR_UNSUPPORTED = 2,   /* a size outside the supported set above */
    GDN_ERR_CUDA = 3,          /* a CUDA launch or attribute call failed */
    GDN_ERR_TIMEOUT = 4,       /* a bounded on-device wait gave up (see gdn_device_status) */
    GDN_ERR_BAD_PAGE = 5,      /* a cache position had no valid page (see gdn_device_status) */
    GDN_ERR_BAD_OFFSETS = 6    /* offsets of packed sequences not in order (see gdn_device_status) */
} gdn_status;

/* Problem sizes: the fields of GatedDeltaConfig (mlex gated_delta.rs) plus the
 * batch B and the number of time steps T of this call.  eps_qk is the q/k
 * rms-norm epsilon (1e-6 on the pages). */
typedef struct gdn_dims {
    int32_t B, T, Hk, Hv, Dk, Dv, K;
    float eps_qk;
} gdn_dims;

/* Causal depthwise conv + SiLU + q/k rms-norm and scaling, with the rolling
 * conv state.  (mlex gated_delta.rs, GatedDeltaNet::forward: the conv_state
 * concat/slice, conv1d with groups = conv_dim, silu, split into q/k/v, rms_norm
 * and the inv_scale factors.)
 *   qkv        bf16 [B, T, C]      pre-conv input (in)
 *   conv_w     bf16 [C, K]         depthwise weights, tap K-1 = current token (in)
 *   conv_state bf16 [B, K-1, C]    in/out: the K-1 most recent valid raw inputs,
 *                                  oldest first; NULL = zeros and not returned
 *   mask       u8   [B, T]         nonzero = valid step; NULL = all valid
 *   q, k       bf16 [B, T, Hk, Dk] out; v bf16 [B, T, Hv, Dv] out.  One
 *                                  round-to-nearest-even rounding of the f32
 *                                  result; masked steps are written as zeros.
 * qkv must not alias any output. */
GDN_API gdn_status gdn_conv_update(const gdn_dims *dims, const uint16_t *qkv, const uint16_t *conv_w,
                           uint16_t *conv_state, const uint8_t *mask,
                           uint16_t *q, uint16_t *k, uint16_t *v, gdn_stream stream);

/* Gates. (mlex gated_delta.rs, GatedDeltaNet::forward: beta and g; mlx-bun
 * qwen3-delta.ts, computeG.)
 *   a, b        bf16 [B, T, Hv] (in);  A_log, dt_bias f32 [Hv] (in)
 *   g, beta     f32  [B, T, Hv] (out): g = exp(-exp(A_log) softplus(a + dt_bias)),
 *               beta = sigmoid(b), softplus(x) = max(x,0) + log1p(exp(-|x|)). */
GDN_API gdn_status gdn_gating(const gdn_dims *dims, const uint16_t *a, const uint16_t *b,
                      const float *A_log, const float *dt_bias, float *g, float *beta,
                      gdn_stream stream);

/* One decode step (dims->T must be 1), fully fused: conv window + conv + SiLU
 * + q/k norm, gates, and the recurrence step, in one kernel that streams the
 * f32 state once.  (mlx-bun qwen3-delta.ts, gated_delta_step at T = 1;
 * mlex gated_delta.rs, GatedDeltaNet::forward with a one-token input.)
 *   qkv        bf16 [B, C] (in)            conv_w bf16 [C, K] (in)
 *   conv_state bf16 [B, K-1, C] in/out (required)
 *   a, b       bf16 [B, Hv] (in)           A_log, dt_bias f32 [Hv] (in)
 *   state      f32  [B, Hv, Dv, Dk] in/out, updated in place
 *   row_mask   u8   [B] or NULL: a zero row writes y = 0 and leaves both of its
 *              states untouched
 *   y          bf16 [B, Hv, Dv] (out)
 * Supports Hv/Hk <= 16. */
GDN_API gdn_status gdn_recurrent_decode(const gdn_dims *dims, const uint16_t *qkv, const uint16_t *conv_w,
                                uint16_t *conv_state, const uint16_t *a, const uint16_t *b,
                                const float *A_log, const float *dt_bias, float *state,
                                const uint8_t *row_mask, uint16_t *y, gdn_stream stream);

/* Decode steps fed from and returned to host memory: n_steps consecutive
 * tokens of gdn_recurrent_decode (same arithmetic, same kernel), with each
 * step's inputs copied in from host buffers and its y copied out to a host
 * buffer inside the call, as a serving loop does.  (Same definitions as
 * gdn_recurrent_decode.)
 *   qkv_h      bf16 [n_steps, B, C]       host (in), step i's qkv at row i
 *   a_h, b_h   bf16 [n_steps, B, Hv]      host (in)
 *   y_h        bf16 [n_steps, B, Hv, Dv]  host (out)
 *   conv_w, conv_state, A_log, dt_bias, state, row_mask: device, as in
 *              gdn_recurrent_decode (row_mask applies to every step)
 *   staging    device workspace of gdn_decode_host_staging_size(dims) bytes,
 *              16-byte aligned: four slots of qkv, a, b and y, so that the
 *              next steps' inputs travel and earlier steps' y return while
 *              step i runs
 * Host buffers should be page-locked (cudaHostAlloc / pinned): pageable
 * memory is accepted but its copies do not overlap the kernels.  The copies
 * run on two copy streams of the library (cudaMemcpyAsync, one per tensor and
 * step) and are ordered against `stream` with events; the streams and events
 * are created on a device's first call and kept until the process exits, and
 * calls from several host threads enqueue one after the other (a lock per
 * device; their copies then share the two streams).  Everything is enqueued
 * before the call returns and `stream` completes after the last y has
 * arrived, so synchronise `stream` before reading y_h.  Neither host buffer
 * may be written (inputs) or read (y_h) before that.  n_steps = 0 is a no-op.
 * Errors: GDN_ERR_INVALID_ARG for a bad argument or a short staging buffer,
 * GDN_ERR_CUDA for a failed CUDA call (work already enqueued still runs). */
GDN_API gdn_status gdn_recurrent_decode_host_steps(const gdn_dims *dims, int n_steps, const uint16_t *qkv_h,
                                                   const uint16_t *a_h, const uint16_t *b_h, uint16_t *y_h,
                                                   const uint16_t *conv_w, uint16_t *conv_state,
                                                   const float *A_log, const float *dt_bias, float *state,
                                                   const uint8_t *row_mask, void *staging, size_t staging_bytes,
                                                   gdn_stream stream);

/* Bytes of device staging gdn_recurrent_decode_host_steps needs (0 for bad
 * dims). */
GDN_API size_t gdn_decode_host_staging_size(const gdn_dims *dims);

/* gdn_recurrent_decode followed by the layer's RMSNormGated.  The norm runs
 * in the decode kernel's epilogue when one CTA holds all Dv rows of a head
 * (for example Hv/Hk = 16 or Dv = 32 with few heads); when a head's rows are
 * spread over several CTAs, the decode kernel writes y into `out` and a
 * second kernel normalises it in place, which measured faster than an
 * exchange of partial sums between the CTAs.  (mlex gated_delta.rs,
 * GatedDeltaNet::forward: the f32 rms_norm of y over Dv with norm_eps, times
 * the norm weight, times silu(z), cast to bf16.)  Per (b, hv):
 *   out = bf16( silu(z) * norm_w * yb / sqrt(mean_Dv(yb^2) + norm_eps) )
 * where yb is the bf16-rounded recurrence output (the y gdn_recurrent_decode
 * would write), so the result equals gdn_recurrent_decode followed by
 * gdn_rmsnorm_gated up to f32 summation order.
 *   z          bf16 [B, Hv, Dv] (in): the in_proj_z output of the token
 *   norm_w     f32  [Dv] (in);  norm_eps >= 0
 *   out        bf16 [B, Hv, Dv] (out); a zero row of row_mask gives zeros
 *              (its y is 0; the sign of a zero follows silu(z) * norm_w)
 * Other arguments and limits as gdn_recurrent_decode. */
GDN_API gdn_status gdn_recurrent_decode_gated(const gdn_dims *dims, const uint16_t *qkv,
                                              const uint16_t *conv_w, uint16_t *conv_state,
                                              const uint16_t *a, const uint16_t *b, const float *A_log,
                                              const float *dt_bias, float *state, const uint8_t *row_mask,
                                              const uint16_t *z, const float *norm_w, float norm_eps,
                                              uint16_t *out, gdn_stream stream);

/* Multi-token decode window for speculative verification: dims->T (1..8)
 * new tokens per row, fused like gdn_recurrent_decode (one pass over the f32
 * state).  y is written for all T tokens; conv_state and state are advanced by
 * exactly keep[b] leading tokens of row b, so a verify call with keep = NULL
 * (all tokens) or a commit call with the accepted counts gives the state after
 * the accepted prefix.  (mlx-bun qwen3-delta.ts, SsmSpecRound and
 * specRoundRollback: a window of S tokens whose first `keep` are kept, the
 * state after them being the same arithmetic prefix; gated_delta_step.)
 *   qkv        bf16 [B, T, C] (in)          conv_w bf16 [C, K] (in)
 *   conv_state bf16 [B, K-1, C] in/out      a, b bf16 [B, T, Hv] (in)
 *   A_log, dt_bias f32 [Hv] (in)            state f32 [B, Hv, Dv, Dk] in/out
 *   keep       int32 [B] or NULL (= T); values are clamped to [0, T]; 0 leaves
 *              both states untouched (y is still produced)
 *   y          bf16 [B, T, Hv, Dv] (out)
 * Supports Hv/Hk <= 16; dims->T outside 1..8 gives GDN_ERR_UNSUPPORTED. */
GDN_API gdn_status gdn_decode_window(const gdn_dims *dims, const uint16_t *qkv, const uint16_t *conv_w,
                                     uint16_t *conv_state, const uint16_t *a, const uint16_t *b,
                                     const float *A_log, const float *dt_bias, float *state,
                                     const int32_t *keep, uint16_t *y, gdn_stream stream);

/* The recurrence over T steps (prefill).  (mlx-bun qwen3-delta.ts,
 * gatedDeltaUpdate and the gated_delta_step kernel with its masked
 * specialization; mlex gated_delta.rs, the per-timestep loop.)
 *   q, k       bf16 [B, T, Hk, Dk] (in)    v bf16 [B, T, Hv, Dv] (in)
 *   g, beta    f32  [B, T, Hv] (in)
 *   state_in   f32  [B, Hv, Dv, Dk] or NULL (= zeros)
 *   state_out  f32  [B, Hv, Dv, Dk] (out); may equal state_in
 *   mask       u8   [B, T] or NULL
 *   y          bf16 [B, T, Hv, Dv] (out)
 *   chunk      0 = sequential form (state resident on chip across all T);
 *              64 = chunked (WY / UT-transform) form on the tensor cores
 *   workspace  optional device scratch of at least gdn_prefill_workspace_size()
 *              bytes, 16-byte aligned, or NULL.  With a mask, the call first
 *              writes there the order in which rows are handed to the kernel's
 *              CTAs (most chunks holding a valid step first), so that the
 *              longest rows of a ragged batch do not start last; with NULL the
 *              rows go in index order.  With chunk = 64 and fewer heads
 *              (B * Hv) than the GPU has SMs, the size also covers the
 *              two-pass chunked form (about 145 KiB per head and chunk of 64
 *              steps): the state-independent work of all chunks first runs
 *              over the whole GPU and is kept there, then one pass per head
 *              applies it to the state.  The results are the same, bit for
 *              bit, whichever way the call runs.  A workspace smaller than
 *              the two-pass size but at least the row-order size runs the
 *              single pass; a smaller or misaligned one gives
 *              GDN_ERR_INVALID_ARG.  It must not be in use by another call
 *              still running on another stream.
 * Wholly masked 64-step chunks cost only their zero y stores.
 * The chunked form reads q, k, v of masked steps (their contribution is then
 * cancelled exactly), so those entries must hold finite values; the zeros
 * gdn_conv_update writes there qualify.  It supports every Dk, Dv in
 * {32, 64, 128}: smaller heads run in the same 128-wide tiles, the channels
 * past the head read as zeros and are never written, so a chunk costs what it
 * costs at 128 and the results are those of the true sizes.
 */
GDN_API gdn_status gdn_prefill(const gdn_dims *dims, const uint16_t *q, const uint16_t *k,
                       const uint16_t *v, const float *g, const float *beta,
                       const float *state_in, float *state_out, const uint8_t *mask,
                       uint16_t *y, int chunk, void *workspace, size_t ws_bytes,
                       gdn_stream stream);

/* gdn_prefill with the layer's RMSNormGated applied to y before it is
 * stored.  (mlex gated_delta.rs, GatedDeltaNet::forward: the f32 rms_norm of
 * y over Dv with norm_eps, times the norm weight, times silu(z), cast to bf16.)
 * Per (b, t, hv):
 *   out = bf16( silu(z) * norm_w * yb / sqrt(mean_Dv(yb^2) + norm_eps) )
 * with yb the bf16 y that gdn_prefill would write (so a masked step, yb = 0,
 * gives a zero).  chunk = 64 runs the norm in the chunked kernel's epilogue
 * (y never goes to memory) when B * Hv is at least the GPU's SM count; with
 * fewer heads, and for chunk = 0 (whose kernel spreads a head's rows over
 * several CTAs), y is written to `out` and a second kernel normalises it in
 * place, which measured faster there.
 *   z          bf16 [B, T, Hv, Dv] (in): the in_proj_z output
 *   norm_w     f32  [Dv] (in);  norm_eps >= 0
 *   out        bf16 [B, T, Hv, Dv] (out)
 * Other arguments, the workspace and the limits as gdn_prefill. */
GDN_API gdn_status gdn_prefill_gated(const gdn_dims *dims, const uint16_t *q, const uint16_t *k,
                                     const uint16_t *v, const float *g, const float *beta,
                                     const float *state_in, float *state_out, const uint8_t *mask,
                                     const uint16_t *z, const float *norm_w, float norm_eps, uint16_t *out,
                                     int chunk, void *workspace, size_t ws_bytes, gdn_stream stream);

/* RMSNormGated output of the layer, applied to the recurrence output y.
 * (mlex gated_delta.rs, GatedDeltaNet::forward: rms_norm of y in f32 with
 * norm_eps, times the norm weight, times silu(z), cast to the activation dtype.)
 *   y, z       bf16 [B, T, Hv, Dv] (in); z is the in_proj_z output
 *   norm_w     f32  [Dv] (in)
 *   out        bf16 [B, T, Hv, Dv] (out), per (b, t, hv) row:
 *              out = bf16( silu(z) * w * y / sqrt(mean_Dv(y^2) + norm_eps) )
 * Only dims->B, T, Hv, Dv are used (the others must still be valid).  out may
 * alias y. */
GDN_API gdn_status gdn_rmsnorm_gated(const gdn_dims *dims, const uint16_t *y, const uint16_t *z,
                                     const float *norm_w, float norm_eps, uint16_t *out, gdn_stream stream);

/* The recurrence with vectorized gating: one decay factor per key channel,
 * S <- S diag(g_t) in place of S <- g_t S (the variant the qwen3-delta.ts
 * page of mlx-bun names beside the scalar one; the rest of the step as in
 * gdn_prefill).  Sequential form.
 *   g_vec      f32  [B, T, Hv, Dk] (in): the per-channel decay factors
 *   other arguments as gdn_prefill (q, k, v, beta, state_in, state_out, mask, y) */
GDN_API gdn_status gdn_prefill_vec(const gdn_dims *dims, const uint16_t *q, const uint16_t *k,
                                   const uint16_t *v, const float *g_vec, const float *beta,
                                   const float *state_in, float *state_out, const uint8_t *mask,
                                   uint16_t *y, gdn_stream stream);

/* gdn_prefill for callers that cannot allocate device memory.  Not an
 * operation of the method (the pages have no counterpart): a variant of the
 * call above for code that may not call cudaMalloc, such as a runtime that
 * hands out all device memory from its own pool, a loop that must never
 * synchronise the device, or a binding with no device allocator.  Same
 * arguments, results and errors as gdn_prefill, minus the workspace: the
 * row-order scratch lives in a fixed 32 KiB array inside the library, held on
 * every GPU that loads the library until the process exits.
 *   dims->B above GDN_NOALLOC_MAX_ROWS gives GDN_ERR_UNSUPPORTED.
 * The first call on each device looks up that array's device address
 * (cudaGetSymbolAddress, with that device current); make it before capturing
 * any stream.  The address is kept for the life of the process: a device
 * reset (cudaDeviceReset, or a reset of the primary context) between calls
 * leaves it stale and is not supported.  All calls share the array: calls that
 * overlap on the GPU (other streams, other host threads) race on it, so order
 * them.  Nothing in it needs clearing between calls.  No allocation is made by
 * this call.
 * Speed: the array holds only the row order, not the per-chunk images of the
 * two-pass chunked form, so with chunk = 64 this call always runs the single
 * pass.  Results are bit-identical to gdn_prefill's, but when B * Hv is below
 * the number of SMs the single pass keeps only B * Hv SMs busy: at B = 1,
 * Hv = 32, T = 8192 it takes about 3.1 times as long as gdn_prefill given
 * its full workspace (1.25 against 0.40 ms).  With B * Hv at or above the SM count both calls run
 * the same kernels. */
#define GDN_NOALLOC_MAX_ROWS 4096
GDN_API gdn_status gdn_prefill_noalloc(const gdn_dims *dims, const uint16_t *q, const uint16_t *k,
                                       const uint16_t *v, const float *g, const float *beta,
                                       const float *state_in, float *state_out, const uint8_t *mask,
                                       uint16_t *y, int chunk, gdn_stream stream);

/* Backward pass of the recurrence (training): the gradients of y and of the
 * final state with respect to q, k, v, g, beta and the initial state.  The
 * pages define the forward step only (mlex gated_delta.rs, the per-timestep
 * loop; mlx-bun qwen3-delta.ts, gated_delta_step); this is its exact
 * derivative.  A masked step has zero gradients for its inputs and passes the
 * state gradient through.  Sequential form, every step in f32.
 *   q, k, v, g, beta, state_in, mask  as gdn_prefill (the forward inputs)
 *   dy         bf16 [B, T, Hv, Dv] (in): gradient of y
 *   dstate_out f32  [B, Hv, Dv, Dk] (in) or NULL (= 0): gradient of the final state
 *   dq, dk     f32  [B, T, Hk, Dk] (out): summed over the Hv/Hk v-heads of each k-head
 *   dv         f32  [B, T, Hv, Dv] (out)
 *   dg, dbeta  f32  [B, T, Hv] (out)
 *   dstate_in  f32  [B, Hv, Dv, Dk] (out): gradient of the initial state (also
 *              when state_in is NULL); may equal dstate_out
 *   workspace  device scratch of gdn_prefill_backward_workspace_size() bytes,
 *              16-byte aligned (required when B * T > 0): a longest-first
 *              row order for masked batches, the forward state
 *              at the start of every 32-step chunk (16 KiB per 32 state rows
 *              and chunk at Dk = 128), for batches with fewer than two row
 *              slices of 32 rows per SM also its gradient at every chunk's
 *              end, and one 32-step history per CTA of the pass that
 *              reverses the chunks (one per row slice, or at most two per SM
 *              of the current device, so query the size on the device that
 *              runs it)
 * The outputs are summed with atomics, so for Hv/Hk > 2 or Dv > 32 their
 * last bits can differ between runs.  Supports Dk, Dv in {32, 64, 128}. */
GDN_API size_t gdn_prefill_backward_workspace_size(const gdn_dims *dims);
GDN_API gdn_status gdn_prefill_backward(const gdn_dims *dims, const uint16_t *q, const uint16_t *k,
                                        const uint16_t *v, const float *g, const float *beta,
                                        const float *state_in, const uint8_t *mask, const uint16_t *dy,
                                        const float *dstate_out, float *dq, float *dk, float *dv, float *dg,
                                        float *dbeta, float *dstate_in, void *workspace, size_t ws_bytes,
                                        gdn_stream stream);

/* The same gradients in chunked form on the tensor cores (Dk, Dv in {32, 64,
 * 128}, all on 128-wide tiles whose padding is exact zeros): the derivative of the chunked
 * forward's products (chunks of 64 steps, tf32 operands with f32
 * accumulation, like gdn_prefill with chunk = 64), with the gradient of the
 * state carried backwards from chunk to chunk.  The call runs the chunked
 * forward first, keeping every chunk's start state and D^T, then the chain
 * images and the reverse chain (one cooperative launch when B * Hv is at
 * most a quarter of the SM count, else two) and two gradient passes.
 * Arguments, outputs and mask semantics as gdn_prefill_backward; the
 * gradients agree with the sequential form within the tf32 rounding of the
 * products (about 3e-4 relative L2 against an f64 reference).
 *   workspace  device scratch of gdn_prefill_backward_chunked_workspace_size()
 *              bytes, 16-byte aligned (required when B * T > 0): the row
 *              order, then per chunk of each (b, hv) head
 *              161 KiB of chain images and 192 KiB of f32 records (start
 *              state, D^T, state gradient, dZ^T), and, when B * Hv is below
 *              the SM count, the two-pass forward's chunk images (sharing
 *              space with the chain images), and a ready flag per chunk.
 *              About 353 KiB per 64 steps of each head: 1.4 GB at B = 1,
 *              Hv = 32, T = 8192.
 * The outputs are summed with atomics (dq, dk over the Hv/Hk v-heads of each
 * k-head); dv, dg, dbeta and dstate_in are written once. */
GDN_API size_t gdn_prefill_backward_chunked_workspace_size(const gdn_dims *dims);
GDN_API gdn_status gdn_prefill_backward_chunked(const gdn_dims *dims, const uint16_t *q, const uint16_t *k,
                                                const uint16_t *v, const float *g, const float *beta,
                                                const float *state_in, const uint8_t *mask, const uint16_t *dy,
                                                const float *dstate_out, float *dq, float *dk, float *dv,
                                                float *dg, float *dbeta, float *dstate_in, void *workspace,
                                                size_t ws_bytes, gdn_stream stream);

/* Bytes of the optional gdn_prefill workspace for these sizes and this chunk
 * mode (0 or 64): about 8 bytes per batch row, rounded up to 256.  Returns 0
 * for invalid or unsupported arguments. */
GDN_API size_t gdn_prefill_workspace_size(const gdn_dims *dims, int chunk);

/* Human-readable name of a status code (static storage). */
GDN_API const char *gdn_status_string(gdn_status status);

/* Synchronises `stream`, then reads and clears the current device's error
 * word, which a kernel sets when one of its bounded waits (on an mbarrier or
 * a tensor-core commit) gives up, or when a position of a paged cache has no
 * page (a page-table entry outside [0, n_pages), a negative position, or one
 * past the table), or when the offsets of packed sequences decrease or leave
 * their buffer.  Returns GDN_OK, GDN_ERR_TIMEOUT (whatever else was recorded),
 * GDN_ERR_BAD_OFFSETS (also when a bad page was recorded), GDN_ERR_BAD_PAGE, or
 * GDN_ERR_CUDA if the synchronisation itself failed. */
GDN_API gdn_status gdn_device_status(gdn_stream stream);

/* Self-test of the failure path: launches a kernel whose bounded wait (on an
 * mbarrier nothing arrives on) runs out after a few thousand probes, and
 * checks that the error word reports it (GDN_ERR_TIMEOUT) and is cleared
 * again.  Returns GDN_OK when the timeout was reported, GDN_ERR_CUDA when it
 * was not (or the device failed).  No fault or unbounded wait is involved;
 * the context stays usable. */
GDN_API gdn_status gdn_selftest_timeout(gdn_stream stream);

/* ------------------------------------------------------------------------
 * Full-attention layers
 * ------------------------------------------------------------------------
 * Sizes of one attention layer's core: B rows of T tokens, Hq query heads,
 * Hkv key/value heads (Hq % Hkv == 0, query head h reads key head
 * h / (Hq/Hkv)), D channels per head, of which the first Drot are rotated.
 * Supported: D in {64, 128, 256}; Drot a multiple of 16 in [0, D];
 * Hq/Hkv <= 16; Hq, Hkv <= 1024; B <= 65535; B, T >= 0 (a zero size is a
 * no-op).  Others give GDN_ERR_UNSUPPORTED.
 *   interleaved  0: channel i < Drot/2 turns with channel i + Drot/2;
 *                1: channel 2i turns with channel 2i + 1
 *   eps          epsilon of the per-head RMS norm, >= 0
 *
 * Inputs marked "heads" may be views of a packed projection: element
 * (b, t, h, d) lies at ptr[(b*T + t)*token_stride + h*head_stride + d], both
 * strides in elements, non-negative and multiples of 8 (so that every head
 * starts on a 16-byte boundary).  Outputs are dense.  Index arrays (pos,
 * n_new, page_table) need only 4-byte, masks no alignment.
 *
 * Rotation: `freqs` u64 [Drot/2] holds each pair's frequency in turns per
 * position as a 64-bit binary fraction, round(f / (2 pi) * 2^64) mod 2^64 for
 * f in radians.  The angle of position p is p * freqs[i] mod 2^64, exact to
 * p * 2^-65 turns at any position.  NULL is allowed when Drot = 0. */
typedef struct gdn_attn_dims {
    int32_t B, T, Hq, Hkv, D, Drot, interleaved;
    float eps;
} gdn_attn_dims;

/* A paged cache of keys and values: pages of page_size tokens, each page
 * [Hkv, page_size, D], so that one head's tokens of a page are contiguous.
 *   format     0: bf16.  1: e4m3 with one e8m0 scale byte per token and head,
 *              [n_pages, Hkv, page_size]: the value is code * 2^(byte - 127),
 *              byte 255 is NaN.  A row x of D values is written with the
 *              smallest power of two s >= 2^-127 such that max|x| <= 448 s, as
 *              codes rne(x / s); a row holding an infinity or NaN reads back
 *              as NaN.  (A power of two costs an e4m3 code no precision but at
 *              its subnormal end, and makes x / s and code * s exact.)
 *   page_size  16, 32, 64, 128 or 256; n_pages * Hkv * page_size < 2^31
 *   k_scale, v_scale are NULL for format 0.
 * A page table i32 [B, table_width] names each row's pages in order: position
 * p of row b lies in page page_table[b][p / page_size].  Rows may share pages.
 * Entries that no accessed position needs are not looked at.  A position
 * without a valid page is not written, reads as zeros and is not attended to;
 * the device error word records it (GDN_ERR_BAD_PAGE). */
typedef struct gdn_kv_cache {
    void *k, *v;
    uint8_t *k_scale, *v_scale;
    int64_t n_pages;
    int32_t page_size, format;
} gdn_kv_cache;

/* Per-head RMS norm and rotary embedding of q and k in one pass.  Per head
 * row x:  z = w x / sqrt(mean(x^2) + eps);  pair (a, b) of z at angle th:
 * y_a = z_a cos th - z_b sin th, y_b = z_b cos th + z_a sin th; the channels
 * from Drot on are z.  f32 arithmetic, one rounding to bf16.
 *   q      bf16 heads [B, T, Hq, D] (in);  k bf16 heads [B, T, Hkv, D] (in)
 *   wq, wk f32 [D] (in), or both NULL: no norm, z = x.  (A model that stores
 *          its weights around zero passes 1 + w.)
 *   pos    i32 [B, T] (in): the position of every token (may be negative)
 *   mask   u8 [B, T] or NULL: a step with mask 0 writes zeros
 *   q_out  bf16 [B, T, Hq, D] (out);  k_out bf16 [B, T, Hkv, D] (out); may be
 *          q and k themselves if those are dense */
GDN_API gdn_status gdn_qk_norm_rope(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                    int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                    int64_t k_head_stride, const float *wq, const float *wk, const uint64_t *freqs,
                                    const int32_t *pos, const uint8_t *mask, uint16_t *q_out, uint16_t *k_out,
                                    gdn_stream stream);

/* Its gradients.  dz = the inverse rotation of dy, xhat = x rstd:
 *   dw = sum over tokens and heads of dz xhat
 *   dx = rstd (w dz - xhat mean(w dz xhat))          (no norm: dx = dz)
 * A masked step has zero gradients and does not enter dw.
 *   q, k, wq, wk, freqs, pos, mask as above (the forward inputs)
 *   dq_out bf16 [B, T, Hq, D], dk_out bf16 [B, T, Hkv, D] (in)
 *   dq, dk bf16, dense, shaped alike (out): they feed the projections'
 *          bf16 products, so they are rounded once here
 *   dwq, dwk f32 [D] (out); NULL when wq, wk are
 *   workspace  device scratch of gdn_qk_norm_rope_backward_workspace_size()
 *          bytes on the device that runs the call (required with weights)
 * The sums over tokens run in a fixed order: equal calls give equal bits. */
GDN_API size_t gdn_qk_norm_rope_backward_workspace_size(const gdn_attn_dims *dims);
GDN_API gdn_status gdn_qk_norm_rope_backward(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                             int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                             int64_t k_head_stride, const float *wq, const float *wk,
                                             const uint64_t *freqs, const int32_t *pos, const uint8_t *mask,
                                             const uint16_t *dq_out, const uint16_t *dk_out, uint16_t *dq,
                                             uint16_t *dk, float *dwq, float *dwk, void *workspace, size_t ws_bytes,
                                             gdn_stream stream);

/* New tokens of every row: norm and rotation of q and k as gdn_qk_norm_rope,
 * keys and values quantised and written into the cache in the same pass.
 *   q, k   as above; v bf16 heads [B, T, Hkv, D] (in)
 *   pos    i32 [B] (in): tokens already in row b's cache; token t has
 *          position pos[b] + t
 *   n_new  i32 [B] or NULL (= T): row b's valid new tokens, clamped to [0, T];
 *          the others are not written and give zero q
 *   q_out  bf16 [B, T, Hq, D] (out)
 * Keys and values are rounded to the cache's type once, from f32. */
GDN_API gdn_status gdn_kv_append(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                 int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                 int64_t k_head_stride, const uint16_t *v, int64_t v_token_stride,
                                 int64_t v_head_stride, const float *wq, const float *wk, const uint64_t *freqs,
                                 const gdn_kv_cache *cache, const int32_t *page_table, int32_t table_width,
                                 const int32_t *pos, const int32_t *n_new, uint16_t *q_out, gdn_stream stream);

/* gdn_qk_norm_rope, its gradients and gdn_kv_append with positions on several axes
 * (the time, height and width of an image's or a video's patches): pair i turns
 * by the token's position on axis axes[i].
 *   axes   u8 [Drot/2] (in): values from n_axes on count as n_axes - 1; not NULL
 *          when Drot > 0
 *   n_axes 1..8
 *   pos    i32 [n_axes, B, T] (in): the position of every token on every axis;
 *          rope_pos likewise, beside gdn_kv_append's pos, which says where in
 *          the cache the tokens go
 * Everything else as above; one axis gives the same bits. */
GDN_API gdn_status gdn_qk_norm_rope_axes(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                         int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                         int64_t k_head_stride, const float *wq, const float *wk, const uint64_t *freqs,
                                         const uint8_t *axes, int32_t n_axes, const int32_t *pos, const uint8_t *mask,
                                         uint16_t *q_out, uint16_t *k_out, gdn_stream stream);
GDN_API gdn_status gdn_qk_norm_rope_axes_backward(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                                  int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                                  int64_t k_head_stride, const float *wq, const float *wk,
                                                  const uint64_t *freqs, const uint8_t *axes, int32_t n_axes,
                                                  const int32_t *pos, const uint8_t *mask, const uint16_t *dq_out,
                                                  const uint16_t *dk_out, uint16_t *dq, uint16_t *dk, float *dwq,
                                                  float *dwk, void *workspace, size_t ws_bytes, gdn_stream stream);
GDN_API gdn_status gdn_kv_append_axes(const gdn_attn_dims *dims, const uint16_t *q, int64_t q_token_stride,
                                      int64_t q_head_stride, const uint16_t *k, int64_t k_token_stride,
                                      int64_t k_head_stride, const uint16_t *v, int64_t v_token_stride,
                                      int64_t v_head_stride, const float *wq, const float *wk, const uint64_t *freqs,
                                      const uint8_t *axes, int32_t n_axes, const int32_t *rope_pos,
                                      const gdn_kv_cache *cache, const int32_t *page_table, int32_t table_width,
                                      const int32_t *pos, const int32_t *n_new, uint16_t *q_out, gdn_stream stream);

/* Positions start[b] .. start[b] + T - 1 of every row read back as bf16 (of an
 * e4m3 cache exactly: code * 2^e is a bf16 value, but where it underflows).
 *   start  i32 [B] (in);  n i32 [B] or NULL (= T): steps from n[b] on are zeros
 *   k_out, v_out bf16 [B, T, Hkv, D] (out)
 * dims->Hq, Drot are not used (but must be valid). */
GDN_API gdn_status gdn_kv_read(const gdn_attn_dims *dims, const gdn_kv_cache *cache, const int32_t *page_table,
                               int32_t table_width, const int32_t *start, const int32_t *n, uint16_t *k_out,
                               uint16_t *v_out, gdn_stream stream);

/* Attention of dims->T (1..8) new tokens per row over the paged cache, which
 * already holds them (gdn_kv_append): token t of row b sees the positions
 * 0 .. pos[b] + t.  Per query row: s_j = scale q.k_j, out = softmax(s) V,
 * lse = log sum_j exp(s_j).
 *   q      bf16 [B, T, Hq, D] (in), dense: gdn_kv_append's q_out
 *   pos, n_new as gdn_kv_append; a token past n_new[b], or one that sees no
 *          key, gives zeros and lse = -inf, whatever its gate holds
 *   gate   bf16 heads [B, T, Hq, D] or NULL: out is multiplied by
 *          sigmoid(gate), in f32 before its one rounding to bf16
 *   scale  of the scores (usually 1/sqrt(D)); finite
 *   out    bf16 [B, T, Hq, D] (out);  lse f32 [B, T, Hq] (out) or NULL
 *   workspace  device scratch of gdn_attn_decode_workspace_size() bytes on the
 *          device that runs the call: the partial results of rows whose
 *          length is split over several CTAs.  They are joined in a fixed
 *          order: equal calls give equal bits.
 * Scores and sums are f32.  Softmax weights are rounded to 16 bits for the
 * product with V: bf16, or with an e4m3 cache f16 (those that, times their
 * value's scale, are below 2^-39 of the largest such product are 0).  Values and keys at positions that a token does not see do
 * not enter its results, whatever they hold; a NaN among the scores that it
 * does see makes its output and lse NaN, and scores that are all -inf make its
 * output NaN (0 / 0) and lse -inf. */
GDN_API size_t gdn_attn_decode_workspace_size(const gdn_attn_dims *dims);
GDN_API gdn_status gdn_attn_decode(const gdn_attn_dims *dims, const uint16_t *q, const gdn_kv_cache *cache,
                                   const int32_t *page_table, int32_t table_width, const int32_t *pos,
                                   const int32_t *n_new, const uint16_t *gate, int64_t gate_token_stride,
                                   int64_t gate_head_stride, float scale, uint16_t *out, float *lse, void *workspace,
                                   size_t ws_bytes, gdn_stream stream);

/* ------------------------------------------------------------------------
 * Whole prompts
 * ------------------------------------------------------------------------
 * Causal attention of dims->B sequences of different lengths, queries and keys
 * from buffers of q_rows and k_rows tokens.  Sequence s holds the tokens
 * cu_q[s] .. cu_q[s + 1] - 1 of the queries' buffer (its slot) and cu_k[s] ..
 * cu_k[s + 1] - 1 of the keys'; of these the first n_q[s] and n_k[s] (clamped to
 * the slot) are there, the others are padding.  The last query sees the last
 * key: query t sees the keys 0 .. t + (keys - queries), so that keys before the
 * queries' own are a kept prefix; a query that sees no key gives zeros and lse =
 * -inf.  dims->T and dims->Drot are not used (but must be valid).
 *   cu_q, cu_k i32 [B + 1] or NULL: slots of q_rows / B (k_rows / B) tokens, which
 *          must be whole numbers.  Offsets that decrease or leave the buffer are
 *          found on the device: the call then writes nothing and the device
 *          error word records GDN_ERR_BAD_OFFSETS.
 *   n_q, n_k i32 [B] or NULL (the whole slots)
 * Padding of a slot gives zeros (and lse = -inf); rows of the outputs in no slot
 * are left as they were.  What lies in keys and values that a query does not
 * see, in padding and in no slot does not enter its results, whatever it is.
 *
 * Inputs marked "heads" are [rows, H, D] views as above (element (n, h, d) at
 * ptr[n*token_stride + h*head_stride + d]); here a stride of 0 over more than
 * one token or head gives GDN_ERR_UNSUPPORTED, as do more than 2^31 - 2^16 rows. */

/* Per query row: s_j = scale q.k_j, out = softmax(s) V, lse = log sum_j exp(s_j).
 *   q      bf16 heads [q_rows, Hq, D];  k, v bf16 heads [k_rows, Hkv, D] (in)
 *   gate   bf16 heads [q_rows, Hq, D] or NULL: out is multiplied by
 *          sigmoid(gate), in f32 before its one rounding to bf16
 *   scale  of the scores (usually 1/sqrt(D)); finite
 *   out    bf16 [q_rows, Hq, D] (out);  lse f32 [q_rows, Hq] (out) or NULL
 *   workspace  device scratch of gdn_attn_prefill_workspace_size() bytes on the
 *          device that runs the call: the work list, and the partial results
 *          of tiles that are split over several CTAs.  They are joined in a
 *          fixed order: equal calls give equal bits.
 * Scores, sums and accumulators are f32; softmax weights are rounded to bf16 for
 * the product with V.  A NaN or +inf among the scores that a query sees makes
 * its output and lse NaN; scores that are all -inf make its output NaN (0 / 0)
 * and lse -inf. */
GDN_API size_t gdn_attn_prefill_workspace_size(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows);
GDN_API gdn_status gdn_attn_prefill(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows, const uint16_t *q,
                                    int64_t q_token_stride, int64_t q_head_stride, const uint16_t *k,
                                    int64_t k_token_stride, int64_t k_head_stride, const uint16_t *v,
                                    int64_t v_token_stride, int64_t v_head_stride, const int32_t *cu_q,
                                    const int32_t *cu_k, const int32_t *n_q, const int32_t *n_k, const uint16_t *gate,
                                    int64_t gate_token_stride, int64_t gate_head_stride, float scale, uint16_t *out,
                                    float *lse, void *workspace, size_t ws_bytes, gdn_stream stream);

/* Its gradients.  P = exp(s - lse), dO = dout sigmoid(gate), delta = sum of dO O
 * over a row's channels:  dv = P^T dO;  dS = P (dO v^T - delta);  dq = scale dS k;
 * dk = scale dS^T q, both summed over the query heads of a key head;
 * dgate = dout out (1 - sigmoid(gate)).
 *   q, k, v, cu_q, cu_k, n_q, n_k, gate, scale  as above (the forward inputs)
 *   out    bf16 [q_rows, Hq, D], lse f32 [q_rows, Hq] (in): the forward results
 *   dout   bf16 [q_rows, Hq, D] (in), dense
 *   dq     bf16 [q_rows, Hq, D], dk, dv bf16 [k_rows, Hkv, D] (out), dense: they
 *          feed bf16 products, so they are rounded once here
 *   dgate  bf16 [q_rows, Hq, D] (out); NULL when gate is
 *   workspace  device scratch of gdn_attn_prefill_backward_workspace_size()
 *          bytes (gated: whether there is a gate) on the device that runs the
 *          call: work lists, delta, dO and partial sums
 * P and dS are rounded to bf16 for their products, dO too where there is a gate;
 * delta is taken from out, for queries that see no more than 64 keys from P and
 * dP themselves, where out's rounding would be too coarse.  Sums are f32 in a
 * fixed order: equal calls give equal bits.  Padding gives zeros, rows in no
 * slot are left as they were; a query that sees no key has no gradient. */
GDN_API size_t gdn_attn_prefill_backward_workspace_size(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows,
                                                        int32_t gated);
GDN_API gdn_status gdn_attn_prefill_backward(const gdn_attn_dims *dims, int64_t q_rows, int64_t k_rows, const uint16_t *q,
                                             int64_t q_token_stride, int64_t q_head_stride, const uint16_t *k,
                                             int64_t k_token_stride, int64_t k_head_stride, const uint16_t *v,
                                             int64_t v_token_stride, int64_t v_head_stride, const int32_t *cu_q,
                                             const int32_t *cu_k, const int32_t *n_q, const int32_t *n_k,
                                             const uint16_t *gate, int64_t gate_token_stride, int64_t gate_head_stride,
                                             float scale, const uint16_t *out, const float *lse, const uint16_t *dout,
                                             uint16_t *dq, uint16_t *dk, uint16_t *dv, uint16_t *dgate, void *workspace,
                                             size_t ws_bytes, gdn_stream stream);

/* ------------------------------------------------------------------------
 * Drafted tokens
 * ------------------------------------------------------------------------
 * Which of a row's drafted tokens stand, and the token after them, by given
 * random numbers, so that what comes out is distributed as the target's own:
 * drafted token x_t stands while all before it do and u_t q_t(x_t) < p_t(x_t).
 * With a of n standing, the next token is drawn from max(p_a - q_a, 0) (from p_a
 * itself where that is all zeros), or for a = n from p_n: the first token whose
 * cumulative sum is above u_T times the whole row's.  (a = the accepted tokens of
 * a window of gdn_decode_window or gdn_attn_decode that held the last token and
 * the drafts: a + 1 of its tokens are kept.)
 *   target f32 [B, T + 1, V] (in): the target's probabilities p_0 .. p_T
 *   draft  f32 [B, T, V] or NULL: the draft's q_0 .. q_(T-1); NULL: tokens from a
 *          lookup, certain to the draft (q = 1 at the token, 0 elsewhere)
 *   tokens i32 [B, T] (in): a token outside [0, V) does not stand
 *   u      f32 [B, T + 1] (in): in [0, 1); the last one draws the next token,
 *          whatever n is
 *   n      i32 [B] or NULL (= T): drafted tokens of a row, clamped to [0, T]
 *   tokens_out i32 [B, T + 1] (out): the standing tokens, the next one, then -1
 *   keep   i32 [B] (out): a + 1, the tokens of tokens_out that are there and
 *          gdn_decode_window's keep
 * 0 <= T <= 1023, 1 <= V <= 2^24, else GDN_ERR_UNSUPPORTED.  Rows are dense and
 * need only 4-byte alignment.  Probabilities count as their nearest value in [0,
 * 1] (NaN as 0); a row's sum must be below 16, else its token is some token in
 * [0, V).  A row of zeros draws token 0.  Comparisons are exact, sums are exact
 * in units of 2^-60: equal calls give equal tokens. */
GDN_API gdn_status gdn_spec_verify(int32_t B, int32_t T, int32_t V, const float *target, const float *draft,
                                   const int32_t *tokens, const float *u, const int32_t *n, int32_t *tokens_out,
                                   int32_t *keep, gdn_stream stream);

/* ABI version of this header (incremented on any signature change). */
GDN_API int gdn_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
