// One query row of a prompt's attention by the definition, key by key, in a
// warp: for rows whose result on the tensor cores is not finite.  There a
// masked weight of 0 meets whatever value lies in an unseen slot, and 0 times
// an infinity or NaN is NaN; here unseen keys are not touched.  Some 0.7 us a
// key: not for warps beside which others wait with a limit.
#pragma once

#include "prompt.cuh"

namespace gdn {
namespace prompt {

// out[d0 .. d1) of the row that sees the first `keys` keys at k, v (> 0);
// returns its lse (`want_lse`; else a row that has become NaN ends there).
template <int D>
__device__ __noinline__ float exact_row(const uint16_t *q, const uint16_t *k, long long k_ts, const uint16_t *v,
                                       long long v_ts, int keys, float scale, const uint16_t *gate, uint16_t *out, int d0,
                                        int d1, bool want_lse) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    float qx[N], o[N], l = 0.0f, m = -INFINITY;
    lane_row<D>(q, qx);
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = 0.0f;
    for (int j = 0; j < keys; ++j) {
        float x[N];
        lane_row<D>(k + j * k_ts, x);
        const float s = row_dot<D>(qx, x) * scale;
        if (s != s) {
            l = s;
            break;
        }
        const float top = fmaxf(m, s), f = m == top ? 1.0f : expf(m - top), w = s == -INFINITY ? 0.0f : expf(s - top);
        m = top;
        l = fmaf(l, f, w);
        lane_row<D>(v + j * v_ts, x);
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = fmaf(w, x[i], o[i] * f);
        if (!want_lse && all_nan(o)) break;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const int d = lane * N + i;
        if (d < d0 || d >= d1) continue;
        float y = o[i] / l;   // (0 / 0: every score is -infinity)
        if (gate != nullptr) y *= sigmoid(bf16_to_f32(gate[d]));
        out[d] = f32_to_bf16(y);
    }
    return m + logf(l);
}

}  // namespace prompt
}  // namespace gdn
