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
// row, eight channels (16 bytes) a lane, so a warp holds RPW = 32 / (D/8) rows
// at once; the partner of a channel in the half-split form sits R/16 lanes
// away.  A warp takes one token and up to ROWS * RPW heads of one kind: all
// their loads go out first, then the token's angles are computed once (one or
// more per lane, shared through shared memory), then the rows.
// At B = 1, T = 8192, 16 + 2 heads of 256 channels (151 MB): XXF us.
#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

constexpr int kThreads = 256, kWarps = kThreads / 32;

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
    int cq, ck;                // chunks of heads of a token: of q, of k (and of v)
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

// The warp's table of a position's angles, then cos and sin of the lane's eight
// channels (interleaved: of its four pairs); channels past R do not turn.
template <bool INTER>
__device__ __forceinline__ void lane_angles(const RowParams &p, float2 *table, int d0, long long pos, float (&c)[8],
                                            float (&s)[8]) {
    const int lane = threadIdx.x & 31, half = p.R / 2;
    __syncwarp();   // (the previous token's readers)
    for (int i = lane; i < half; i += 32) {
        float2 a;
        rope_angle(pos, p.freqs[i], a.x, a.y);
        table[i] = a;
    }
    __syncwarp();
    const int first = INTER ? d0 / 2 : d0 < half ? d0 : d0 - half;
#pragma unroll
    for (int i = 0; i < (INTER ? 4 : 8); ++i) {
        const float2 a = d0 < p.R ? table[first + i] : make_float2(1.0f, 0.0f);
        c[i] = a.x;
        s[i] = a.y;
    }
}

// Turns the lane's channels by the angles (sign = -1: back).
template <bool INTER>
__device__ __forceinline__ void rotate(float (&z)[8], const float (&c)[8], const float (&s)[8], int d0, int R,
                                       float sign) {
    if (INTER) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = z[2 * i], b = z[2 * i + 1], sn = sign * s[i];
            z[2 * i] = a * c[i] - b * sn;
            z[2 * i + 1] = b * c[i] + a * sn;
        }
        return;
    }
    if (R == 0) return;
    const int lane = threadIdx.x & 31;
    const bool low = d0 < R / 2;
    const int partner = d0 >= R ? lane : low ? lane + R / 16 : lane - R / 16;
    const float sg = low ? -sign : sign;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, z[i], partner);
        z[i] = z[i] * c[i] + sg * s[i] * o;
    }
}

enum { kDense = 0, kAppend = 1, kAppendE4M3 = 2 };

template <int D, bool INTER, int MODE, int ROWS>
__global__ void __launch_bounds__(kThreads) row_forward_kernel(const RowParams p, unsigned items) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    __shared__ float2 tables[kWarps][D / 2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const unsigned chunks = p.cq + p.ck * (MODE == kDense ? 1 : 2);
    const unsigned item = blockIdx.x * kWarps + warp;
    if (item >= items) return;
    const unsigned bt = item / chunks, chunk = item - bt * chunks;
    const int b = (int)(bt / (unsigned)p.T), t = (int)(bt - (unsigned)b * p.T);
    const bool isq = chunk < (unsigned)p.cq, isv = MODE != kDense && chunk >= (unsigned)(p.cq + p.ck);
    const int h0 = (int)(isq ? chunk : isv ? chunk - p.cq - p.ck : chunk - p.cq) * ROWS * RPW + lane / LPR;
    const int H = isq ? p.Hq : p.Hkv, d0 = (lane % LPR) * 8;
    const HeadsIn &in = isq ? p.q : isv ? p.v : p.k;
    const bool on = MODE == kDense ? p.mask == nullptr || p.mask[bt] != 0 : t < clamp_new(p.n_new, b, p.T);

    uint4 raw[ROWS];
    const uint16_t *src = in.p + (long long)bt * in.ts + d0;
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        raw[u] = make_uint4(0, 0, 0, 0);
        if (on && h0 + u * RPW < H) raw[u] = *reinterpret_cast<const uint4 *>(src + (h0 + u * RPW) * in.hs);
    }
    uint16_t *out = nullptr;
    if (isq || MODE == kDense) {
        out = (isq ? p.q_out + (long long)bt * p.Hq * D : p.k_out + (long long)bt * p.Hkv * D) + d0;
        if (!on) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                if (h0 + u * RPW < H) *reinterpret_cast<uint4 *>(out + (h0 + u * RPW) * D) = make_uint4(0, 0, 0, 0);
            return;
        }
    } else if (!on) {
        return;
    }
    const long long pos = MODE == kDense ? p.pos[bt] : (long long)p.pos[b] + t;
    long long page_row = -1;   // of head 0
    if (MODE != kDense && !isq) {
        page_row = cache_row(p.c, p.Hkv, p.c.table + (long long)b * p.c.width, pos, 0);
        if (page_row < 0) {
            if (lane == 0) atomicOr(p.err, kErrBadPage);
            return;
        }
    }
    float w[8], c[8], s[8];
    const float *wp = isq ? p.wq : p.wk;
    const bool norm = !isv && wp != nullptr;
    if (norm) {
        const float4 w0 = *reinterpret_cast<const float4 *>(wp + d0), w1 = *reinterpret_cast<const float4 *>(wp + d0 + 4);
        w[0] = w0.x, w[1] = w0.y, w[2] = w0.z, w[3] = w0.w, w[4] = w1.x, w[5] = w1.y, w[6] = w1.z, w[7] = w1.w;
    }
    if (!isv) lane_angles<INTER>(p, tables[warp], d0, pos, c, s);
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int h = h0 + u * RPW;
        if (u > 0 && h0 - lane / LPR + u * RPW >= H) break;   // (no row of the warp)
        float x[8];
        unpack8(raw[u], x);
        if (norm) {
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
            const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.0f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= rstd * w[i];
        }
        if (!isv) rotate<INTER>(x, c, s, d0, p.R, 1.0f);
        if (isq || MODE == kDense) {
            if (h < H) *reinterpret_cast<uint4 *>(out + h * D) = pack8(x);
            continue;
        }
        const long long at = page_row + ((long long)h << p.c.shift);
        if (MODE == kAppend) {
            if (h < H) *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(isv ? p.c.v : p.c.k) + at * D + d0) = pack8(x);
            continue;
        }
        uint32_t amax = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) amax = max(amax, __float_as_uint(x[i]) & 0x7fffffffu);
        amax = row_max<LPR>(amax);
        const uint32_t byte = e8m0_for(amax);
        const float inv = e8m0_inverse(byte);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] *= inv;
        if (h < H) {
            *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(isv ? p.c.v : p.c.k) + at * D + d0) = pack8_e4m3(x);
            if (d0 == 0) (isv ? p.c.vs : p.c.ks)[at] = (uint8_t)byte;
        }
    }
}

// Backward: CTAs below nq take head rows of q, the others of k (in proportion),
// each warp one token and ROWS * RPW heads at a time; a CTA sums its share of
// dw and leaves it in `partial`.
template <int D, bool INTER>
__global__ void __launch_bounds__(kThreads, 2) row_backward_kernel(const RowParams p, int nq) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = 4;
    __shared__ float2 tables[kWarps][D / 2];
    __shared__ float sum[kWarps * RPW][D];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int d0 = (lane % LPR) * 8;
    const bool isq = (int)blockIdx.x < nq;
    const HeadsIn &in = isq ? p.q : p.k;
    const int H = isq ? p.Hq : p.Hkv;
    const uint16_t *dy_p = (isq ? p.dq_out : p.dk_out) + d0;
    uint16_t *dx_p = (isq ? p.q_out : p.k_out) + d0;
    const float *wp = isq ? p.wq : p.wk;
    const bool norm = wp != nullptr;
    float w[8], acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        w[i] = norm ? wp[d0 + i] : 1.0f;
        acc[i] = 0.0f;
    }
    const unsigned chunks = isq ? p.cq : p.ck, items = (unsigned)p.B * p.T * chunks;
    const unsigned cta = isq ? blockIdx.x : blockIdx.x - nq, ctas = isq ? nq : gridDim.x - nq;
    for (unsigned item = cta * kWarps + warp; item < items; item += ctas * kWarps) {
        const unsigned bt = item / chunks, chunk = item - bt * chunks;
        const int h0 = (int)chunk * ROWS * RPW + lane / LPR;
        const long long row0 = (long long)bt * H;
        if (p.mask != nullptr && p.mask[bt] == 0) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                if (h0 + u * RPW < H)
                    *reinterpret_cast<uint4 *>(dx_p + (row0 + h0 + u * RPW) * D) = make_uint4(0, 0, 0, 0);
            continue;
        }
        uint4 rx[ROWS], rdy[ROWS];
        const uint16_t *src = in.p + (long long)bt * in.ts + d0;
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const int h = h0 + u * RPW;
            rx[u] = rdy[u] = make_uint4(0, 0, 0, 0);
            if (h < H) {
                if (norm) rx[u] = *reinterpret_cast<const uint4 *>(src + h * in.hs);
                rdy[u] = *reinterpret_cast<const uint4 *>(dy_p + (row0 + h) * D);
            }
        }
        float c[8], s[8];
        lane_angles<INTER>(p, tables[warp], d0, p.pos[bt], c, s);
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const int h = h0 + u * RPW;
            if (u > 0 && h0 - lane / LPR + u * RPW >= H) break;   // (no row of the warp)
            float x[8], dz[8];
            unpack8(rx[u], x);
            unpack8(rdy[u], dz);
            rotate<INTER>(dz, c, s, d0, p.R, -1.0f);
            if (norm) {
                // two sums at once: x.x, and (w dz).x, which times rstd is (w dz).xhat
                float ss = 0.0f, dot = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    ss = fmaf(x[i], x[i], ss);
                    dot = fmaf(w[i] * dz[i], x[i], dot);
                }
                ss = row_sum<LPR>(ss);
                dot = row_sum<LPR>(dot);
                float rstd = rsqrtf(ss * (1.0f / D) + p.eps);
                if (h >= H) rstd = 0.0f;   // (a row that is not there; eps = 0 would make it an infinity)
                const float k = dot * rstd * rstd * (1.0f / D);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc[i] = fmaf(dz[i], x[i] * rstd, acc[i]);
                    dz[i] = rstd * fmaf(-k, x[i], w[i] * dz[i]);
                }
            }
            if (h < H) *reinterpret_cast<uint4 *>(dx_p + (row0 + h) * D) = pack8(dz);
        }
    }
    grid_dep_launch();
    if (!norm) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[warp * RPW + lane / LPR][d0 + i] = acc[i];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float t = 0.0f;
        for (int i = 0; i < kWarps * RPW; ++i) t += sum[i][d];
        p.partial[(size_t)blockIdx.x * D + d] = t;
    }
}

// dw = the CTAs' shares, every eighth one by one thread, then those sums in
// order.  Blocks: (q or k, 32 channels).
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float *partial, int nq, int n, int D, float *dwq,
                                                          float *dwk) {
    __shared__ float sum[32][33];
    grid_dep_wait();
    const bool isq = blockIdx.x == 0;
    const int d = blockIdx.y * 32 + threadIdx.x, part = threadIdx.y;
    float t = 0.0f;
    for (int i = (isq ? 0 : nq) + part; i < (isq ? nq : n); i += 32) t += partial[(size_t)i * D + d];
    sum[part][threadIdx.x] = t;
    __syncthreads();
    if (part != 0) return;
    t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += sum[i][threadIdx.x];
    (isq ? dwq : dwk)[d] = t;
}

int chunks_of(int heads, int rows) { return (heads + rows - 1) / rows; }

template <int D, int MODE, int ROWS>
cudaError_t launch_forward_rows(RowParams p, bool inter, cudaStream_t st) {
    constexpr int RPW = 32 / (D / 8);
    p.cq = chunks_of(p.Hq, ROWS * RPW);
    p.ck = chunks_of(p.Hkv, ROWS * RPW);
    const unsigned long long items = (unsigned long long)p.B * p.T * (p.cq + p.ck * (MODE == kDense ? 1 : 2));
    if (items > 0xffffff00ull) return cudaErrorNotSupported;
    const unsigned grid = (unsigned)((items + kWarps - 1) / kWarps);
    if (inter)
        row_forward_kernel<D, true, MODE, ROWS><<<grid, kThreads, 0, st>>>(p, (unsigned)items);
    else
        row_forward_kernel<D, false, MODE, ROWS><<<grid, kThreads, 0, st>>>(p, (unsigned)items);
    return cudaGetLastError();
}

// Four rows a warp hide each other's latency when there are warps enough to
// fill the GPU; with few tokens (B = 128, T = 1: XXA against XXB us) one row a
// warp spreads wider.
template <int D, int MODE>
cudaError_t launch_forward(const RowParams &p, bool inter, cudaStream_t st) {
    constexpr int RPW = 32 / (D / 8);
    const long long warps = (long long)p.B * p.T * (p.Hq + 2 * p.Hkv) / RPW;
    return warps >= 64LL * num_sms() ? launch_forward_rows<D, MODE, 4>(p, inter, st)
                                     : launch_forward_rows<D, MODE, 1>(p, inter, st);
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

// CTAs of the backward pass for q and for k: in proportion to their rows, and
// no more than there is work for.
void backward_grid(const AttnSizes &s, int *nq, int *nk) {
    const int rows = 4 * (32 / (s.D / 8));
    const long long tokens = (long long)s.B * s.T;
    const long long wq = (tokens * chunks_of(s.Hq, rows) + kWarps - 1) / kWarps;
    const long long wk = (tokens * chunks_of(s.Hkv, rows) + kWarps - 1) / kWarps;
    const int total = 2 * num_sms();
    const int k = (int)((long long)total * s.Hkv / (s.Hq + s.Hkv));
    *nk = k < 1 ? 1 : k;
    *nq = total - *nk;
    if (*nk > wk) *nk = wk < 1 ? 1 : (int)wk;
    if (*nq > wq) *nq = wq < 1 ? 1 : (int)wq;
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
    return c.fp8 ? launch_forward_d<kAppendE4M3>(p, s.D, s.inter, st) : launch_forward_d<kAppend>(p, s.D, s.inter, st);
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
    const int rows = 4 * (32 / (s.D / 8));
    p.cq = chunks_of(s.Hq, rows);
    p.ck = chunks_of(s.Hkv, rows);
    if ((unsigned long long)s.B * s.T * p.cq > 0x7fffffffull) return cudaErrorNotSupported;
    int nq, nk;
    backward_grid(s, &nq, &nk);
    auto run = [&](auto kernel) { kernel<<<nq + nk, kThreads, 0, st>>>(p, nq); };
    if (s.D == 64) s.inter ? run(row_backward_kernel<64, true>) : run(row_backward_kernel<64, false>);
    else if (s.D == 128) s.inter ? run(row_backward_kernel<128, true>) : run(row_backward_kernel<128, false>);
    else s.inter ? run(row_backward_kernel<256, true>) : run(row_backward_kernel<256, false>);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || wq == nullptr) return e;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2, s.D / 32);
    cfg.blockDim = dim3(32, 32);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, weight_sum_kernel, (const float *)p.partial, nq, nq + nk, (int)s.D, dwq, dwk);
}

}  // namespace gdn
