// Per-head RMS norm and rotary embedding of queries and keys: forward,
// backward, and the serving form that writes keys and values into the paged
// cache.
//
// Per head row x of D channels: z = w x / sqrt(mean(x^2) + eps); each pair
// (a, b) of the first R channels turns by its angle, y_a = z_a cos - z_b sin,
// y_b = z_b cos + z_a sin.  The rotation is orthogonal, so the backward pass
// turns dy by the opposite angle (dz), and with xhat = x rstd
//   dw = sum dz xhat,   dx = rstd (w dz - xhat mean(w dz xhat)).
//
// Every element is read and written once: HBM-bound.  D/8 lanes hold one head
// row, eight channels (16 bytes) a lane, so a warp holds 32 / (D/8) rows; the
// partner of a channel in the half-split form sits R/16 lanes away.
#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

constexpr int kThreads = 256;

struct RowParams {
    HeadsIn q, k, v;
    const float *wq, *wk;
    const uint64_t *freqs;
    const int32_t *pos;     // dense: [B, T]; append: [B]
    const uint8_t *mask;
    const int32_t *n_new;
    const uint16_t *dq_out, *dk_out;
    uint16_t *q_out, *k_out;   // backward: dq, dk
    float *partial;            // backward: [2][gridDim.x][D]
    PagedCache c;
    unsigned *err;
    int B, T, Hq, Hkv, R;
    float eps;
};

template <int LPR>
__device__ __forceinline__ float row_sum(float x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}

template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// cos and sin of the lane's eight channels (interleaved: of its four pairs).
template <bool INTER>
__device__ __forceinline__ void lane_angles(const RowParams &p, int d0, long long pos, float (&c)[8], float (&s)[8]) {
    const int half = p.R / 2;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.0f;
        s[i] = 0.0f;
    }
    if (d0 >= p.R) return;
    if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) rope_angle(pos, p.freqs[d0 / 2 + i], c[i], s[i]);
    } else {
        const int i0 = d0 < half ? d0 : d0 - half;
#pragma unroll
        for (int i = 0; i < 8; ++i) rope_angle(pos, p.freqs[i0 + i], c[i], s[i]);
    }
}

// Turns the lane's channels by the angles (sign = -1: back).
template <int LPR, bool INTER>
__device__ __forceinline__ void rotate(float (&z)[8], const float (&c)[8], const float (&s)[8], int d0, int R,
                                       float sign) {
    if (INTER) {
        if (d0 < R) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float a = z[2 * i], b = z[2 * i + 1], sn = sign * s[i];
                z[2 * i] = a * c[i] - b * sn;
                z[2 * i + 1] = b * c[i] + a * sn;
            }
        }
        return;
    }
    const int lane = threadIdx.x & 31;
    const bool low = d0 < R / 2;
    const int partner = d0 >= R ? lane : low ? lane + R / 16 : lane - R / 16;
    const float sg = low ? -sign : sign;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, z[i], partner);
        if (d0 < R) z[i] = z[i] * c[i] + sg * o * s[i];
    }
}

enum { kDense = 0, kAppend = 1 };

// One warp per 32/LPR head rows.
template <int D, bool INTER, int MODE>
__global__ void __launch_bounds__(kThreads) row_forward_kernel(const RowParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const int H = p.Hq + p.Hkv * (MODE == kAppend ? 2 : 1);
    const long long rows = (long long)p.B * p.T * H;
    const long long row = (((long long)blockIdx.x * kThreads + threadIdx.x) >> 5) * RPW + lane / LPR;
    const int d0 = (lane % LPR) * 8;
    const bool live = row < rows;
    const long long bt = live ? row / H : 0;
    const int h = live ? (int)(row % H) : 0;
    const int b = (int)(bt / p.T), t = (int)(bt % p.T);
    const bool isq = h < p.Hq, isv = MODE == kAppend && h >= p.Hq + p.Hkv;
    const int hh = isq ? h : isv ? h - p.Hq - p.Hkv : h - p.Hq;
    const HeadsIn &in = isq ? p.q : isv ? p.v : p.k;

    const bool on = MODE == kAppend ? t < clamp_new(p.n_new, b, p.T) : p.mask == nullptr || p.mask[bt] != 0;
    const long long pos = MODE == kAppend ? (long long)p.pos[b] + t : p.pos[bt];
    float x[8];
    unpack8(live && on ? *reinterpret_cast<const uint4 *>(in.p + bt * in.ts + hh * in.hs + d0) : make_uint4(0, 0, 0, 0),
            x);
    float ss = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
    const float *w = isq ? p.wq : p.wk;
    if (!isv && w != nullptr) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = x[i] * rstd * w[d0 + i];
    }
    float c[8], s[8], z[8];
    lane_angles<INTER>(p, d0, pos, c, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = x[i];
    rotate<LPR, INTER>(z, c, s, d0, p.R, 1.0f);
    if (!isv) {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = z[i];
    }
    uint32_t amax = 0;
    if (MODE == kAppend && p.c.fp8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
        amax = row_max<LPR>(amax);
    }
    if (!live) return;
    if (isq || MODE == kDense) {
        if (!on) {
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = 0.0f;
        }
        uint16_t *out = isq ? p.q_out + (bt * p.Hq + hh) * D : p.k_out + (bt * p.Hkv + hh) * D;
        *reinterpret_cast<uint4 *>(out + d0) = pack8(x);
        return;
    }
    if (!on) return;
    const long long at = cache_row(p.c, p.Hkv, p.c.table + (long long)b * p.c.width, pos, hh);
    if (at < 0) {
        if (d0 == 0) atomicOr(p.err, kErrBadPage);
        return;
    }
    void *pages = isv ? p.c.v : p.c.k;
    if (!p.c.fp8) {
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(pages) + at * D + d0) = pack8(x);
        return;
    }
    const uint32_t byte = e8m0_for(amax);
    const float inv = e8m0_inverse(byte);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= inv;
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(pages) + at * D + d0) = pack8_e4m3(x);
    if (d0 == 0) (isv ? p.c.vs : p.c.ks)[at] = (uint8_t)byte;
}

// Backward: each CTA takes head rows of q (CTAs below nq) or of k, sums its
// share of dw and leaves it in `partial`.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads) row_backward_kernel(const RowParams p, int nq) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ float sum[kThreads / 32 * RPW][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d0 = (lane % LPR) * 8;
    const bool isq = (int)blockIdx.x < nq;
    const HeadsIn &in = isq ? p.q : p.k;
    const int H = isq ? p.Hq : p.Hkv;
    const uint16_t *dy_p = isq ? p.dq_out : p.dk_out;
    uint16_t *dx_p = isq ? p.q_out : p.k_out;
    const float *wp = isq ? p.wq : p.wk;
    const bool norm = wp != nullptr;
    float w[8], acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = norm ? wp[d0 + i] : 1.0f;
        acc[i] = 0.0f;
    }
    const long long rows = (long long)p.B * p.T * H;
    const int cta = isq ? blockIdx.x : blockIdx.x - nq, ctas = isq ? nq : gridDim.x - nq;
    const long long step = (long long)ctas * (kThreads / 32) * RPW;
    for (long long r0 = ((long long)cta * (kThreads / 32) + warp) * RPW; r0 < rows; r0 += step) {
        const long long row = r0 + lane / LPR;
        const bool live = row < rows;
        const long long bt = live ? row / H : 0;
        const int h = live ? (int)(row % H) : 0;
        const bool on = live && (p.mask == nullptr || p.mask[bt] != 0);
        float x[8], dz[8], c[8], s[8];
        const uint4 zero = make_uint4(0, 0, 0, 0);
        unpack8(on ? *reinterpret_cast<const uint4 *>(in.p + bt * in.ts + h * in.hs + d0) : zero, x);
        unpack8(on ? *reinterpret_cast<const uint4 *>(dy_p + (bt * H + h) * D + d0) : zero, dz);
        lane_angles<INTER>(p, d0, p.pos[bt], c, s);
        rotate<LPR, INTER>(dz, c, s, d0, p.R, -1.0f);
        if (norm) {
            float ss = 0.0f, dot = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            float rstd = rsqrtf(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
            if (!on) rstd = 0.0f;   // (eps = 0 would make it an infinity)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                x[i] *= rstd;
                acc[i] = fmaf(dz[i], x[i], acc[i]);
                dz[i] *= w[i];
                dot = fmaf(dz[i], x[i], dot);
            }
            dot = row_sum<LPR>(dot) * (1.0f / D);
#pragma unroll
            for (int i = 0; i < 8; ++i) dz[i] = on ? rstd * (dz[i] - x[i] * dot) : 0.0f;
        }
        if (live) *reinterpret_cast<uint4 *>(dx_p + (bt * H + h) * D + d0) = pack8(dz);
    }
    if (!norm) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[warp * RPW + lane / LPR][d0 + i] = acc[i];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float t = 0.0f;
        for (int i = 0; i < kThreads / 32 * RPW; ++i) t += sum[i][d];
        p.partial[(size_t)blockIdx.x * D + d] = t;
    }
}

// dw = the CTAs' shares in their order.
__global__ void weight_sum_kernel(const float *partial, int nq, int n, int D, float *dwq, float *dwk) {
    const bool isq = blockIdx.x == 0;
    const int d = threadIdx.x;
    float t = 0.0f;
    for (int i = isq ? 0 : nq; i < (isq ? nq : n); ++i) t += partial[(size_t)i * D + d];
    (isq ? dwq : dwk)[d] = t;
}

template <int D, int MODE>
cudaError_t launch_forward(const RowParams &p, bool inter, cudaStream_t st) {
    const long long rows = (long long)p.B * p.T * (p.Hq + p.Hkv * (MODE == kAppend ? 2 : 1));
    const long long per_cta = kThreads / 32 * (32 / (D / 8));
    const long long grid = (rows + per_cta - 1) / per_cta;
    if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
    if (inter)
        row_forward_kernel<D, true, MODE><<<(unsigned)grid, kThreads, 0, st>>>(p);
    else
        row_forward_kernel<D, false, MODE><<<(unsigned)grid, kThreads, 0, st>>>(p);
    return cudaGetLastError();
}

template <int MODE>
cudaError_t launch_forward_d(const RowParams &p, int D, bool inter, cudaStream_t st) {
    switch (D) {
        case 64: return launch_forward<64, MODE>(p, inter, st);
        case 128: return launch_forward<128, MODE>(p, inter, st);
        case 256: return launch_forward<256, MODE>(p, inter, st);
        default: return cudaErrorInvalidValue;
    }
}

RowParams row_params(const AttnSizes &s, const HeadsIn &q, const HeadsIn &k, const float *wq, const float *wk,
                     const uint64_t *freqs, const int32_t *pos) {
    RowParams p = {};
    p.q = q;
    p.k = k;
    p.wq = wq;
    p.wk = wk;
    p.freqs = freqs;
    p.pos = pos;
    p.B = s.B;
    p.T = s.T;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.R = s.Drot;
    p.eps = s.eps;
    return p;
}

// CTAs of the backward pass for q and for k: in proportion to their rows.
void backward_grid(const AttnSizes &s, int *nq, int *nk) {
    const int total = 4 * num_sms();
    *nk = total * s.Hkv / (s.Hq + s.Hkv);
    if (*nk < 1) *nk = 1;
    *nq = total - *nk;
}

}  // namespace

cudaError_t launch_qk_norm_rope(const AttnSizes &s, const HeadsIn &q, const HeadsIn &k, const float *wq,
                                const float *wk, const uint64_t *freqs, const int32_t *pos, const uint8_t *mask,
                                uint16_t *q_out, uint16_t *k_out, cudaStream_t st) {
    RowParams p = row_params(s, q, k, wq, wk, freqs, pos);
    p.mask = mask;
    p.q_out = q_out;
    p.k_out = k_out;
    return launch_forward_d<kDense>(p, s.D, s.inter, st);
}

cudaError_t launch_kv_append(const AttnSizes &s, const HeadsIn &q, const HeadsIn &k, const HeadsIn &v,
                             const float *wq, const float *wk, const uint64_t *freqs, const PagedCache &c,
                             const int32_t *pos, const int32_t *n_new, uint16_t *q_out, unsigned *err,
                             cudaStream_t st) {
    RowParams p = row_params(s, q, k, wq, wk, freqs, pos);
    p.v = v;
    p.c = c;
    p.n_new = n_new;
    p.q_out = q_out;
    p.err = err;
    return launch_forward_d<kAppend>(p, s.D, s.inter, st);
}

size_t qk_norm_rope_backward_workspace(const AttnSizes &s) {
    int nq, nk;
    backward_grid(s, &nq, &nk);
    return (size_t)(nq + nk) * s.D * sizeof(float);
}

cudaError_t launch_qk_norm_rope_backward(const AttnSizes &s, const HeadsIn &q, const HeadsIn &k, const float *wq,
                                         const float *wk, const uint64_t *freqs, const int32_t *pos,
                                         const uint8_t *mask, const uint16_t *dq_out, const uint16_t *dk_out,
                                         uint16_t *dq, uint16_t *dk, float *dwq, float *dwk, void *ws,
                                         cudaStream_t st) {
    RowParams p = row_params(s, q, k, wq, wk, freqs, pos);
    p.mask = mask;
    p.dq_out = dq_out;
    p.dk_out = dk_out;
    p.q_out = dq;
    p.k_out = dk;
    p.partial = static_cast<float *>(ws);
    int nq, nk;
    backward_grid(s, &nq, &nk);
    auto run = [&](auto kernel) { kernel<<<nq + nk, kThreads, 0, st>>>(p, nq); };
    if (s.D == 64) s.inter ? run(row_backward_kernel<64, true>) : run(row_backward_kernel<64, false>);
    else if (s.D == 128) s.inter ? run(row_backward_kernel<128, true>) : run(row_backward_kernel<128, false>);
    else s.inter ? run(row_backward_kernel<256, true>) : run(row_backward_kernel<256, false>);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || wq == nullptr) return e;
    weight_sum_kernel<<<2, s.D, 0, st>>>(p.partial, nq, nq + nk, s.D, dwq, dwk);
    return cudaGetLastError();
}

}  // namespace gdn
