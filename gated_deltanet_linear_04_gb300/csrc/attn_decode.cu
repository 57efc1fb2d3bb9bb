// Attention of 1..8 new tokens per row over the paged cache.
//
// Per query row: s_j = scale q.k_j over the visible positions, out =
// sum_j exp(s_j - m) v_j / sum_j exp(s_j - m), held as a running maximum, sum
// and weighted sum over tiles of keys (one pass over the cache).
//
// One CTA per (row, key head) takes its T * Hq/Hkv query rows through all
// keys, a tile of 64 at a time, scores and the running sums in shared memory.
#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

constexpr int kThreads = 256, kTile = 64;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

struct DecodeAttnParams {
    const uint16_t *q;
    PagedCache c;
    const int32_t *pos, *n_new;
    HeadsIn gate;
    uint16_t *out;
    float *lse;
    unsigned *err;
    int T, Hq, Hkv, G;
    float scale2;   // scale * log2(e)
};

template <int D>
__device__ __forceinline__ void load_row8(const void *pages, const uint8_t *scale, bool fp8, long long at, int d0,
                                          float (&x)[8]) {
    if (!fp8) {
        unpack8(*reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(pages) + at * D + d0), x);
        return;
    }
    unpack8_e4m3(*reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pages) + at * D + d0), x);
    const float s = e8m0_value(scale[at]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= s;
}

template <int D>
__global__ void __launch_bounds__(kThreads) attn_decode_kernel(const DecodeAttnParams p) {
    extern __shared__ float smem[];
    const int b = blockIdx.y, h = blockIdx.x, R = p.T * p.G;
    float *acc = smem, *sc = acc + R * D, *m = sc + R * kTile, *l = m + R, *corr = l + R;
    long long *at = reinterpret_cast<long long *>(corr + R + (R & 1));
    const int n = clamp_new(p.n_new, b, p.T);
    const long long pos = p.pos[b];
    const long long keys = n == 0 ? 0 : min(max(pos + n, 0LL), (long long)p.c.width << p.c.shift);
    if (threadIdx.x == 0 && n > 0 && (pos < 0 || pos + n > keys)) atomicOr(p.err, kErrBadPage);
    for (int i = threadIdx.x; i < R * D; i += kThreads) acc[i] = 0.0f;
    for (int r = threadIdx.x; r < R; r += kThreads) {
        m[r] = -INFINITY;
        l[r] = 0.0f;
    }
    for (long long j0 = 0; j0 < keys; j0 += kTile) {
        __syncthreads();
        if (threadIdx.x < kTile) {
            const long long j = j0 + threadIdx.x;
            long long a = -1;
            if (j < keys) {
                a = cache_row(p.c, p.Hkv, p.c.table + (long long)b * p.c.width, j, h);
                if (a < 0) atomicOr(p.err, kErrBadPage);
            }
            at[threadIdx.x] = a;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < R * kTile; i += kThreads) {
            const int r = i / kTile, j = i % kTile, t = r / p.G;
            const uint16_t *q = p.q + (((long long)b * p.T + t) * p.Hq + h * p.G + r % p.G) * D;
            float s = -INFINITY;
            if (at[j] >= 0 && t < n && j0 + j <= pos + t) {
                s = 0.0f;
                for (int d = 0; d < D; d += 8) {
                    float x[8], y[8];
                    load_row8<D>(p.c.k, p.c.ks, p.c.fp8, at[j], d, x);
                    unpack8(*reinterpret_cast<const uint4 *>(q + d), y);
#pragma unroll
                    for (int e = 0; e < 8; ++e) s = fmaf(x[e], y[e], s);
                }
                s *= p.scale2;
            }
            sc[i] = s;
        }
        __syncthreads();
        for (int r = threadIdx.x; r < R; r += kThreads) {
            float mx = m[r];
            for (int j = 0; j < kTile; ++j) mx = fmaxf(mx, sc[r * kTile + j]);
            const float base = mx == -INFINITY ? 0.0f : mx;
            corr[r] = exp2f(m[r] - base);
            float sum = l[r] * corr[r];
            for (int j = 0; j < kTile; ++j) {
                const float e = exp2f(sc[r * kTile + j] - base);
                sc[r * kTile + j] = e;
                sum += e;
            }
            m[r] = mx;
            l[r] = sum;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < R * (D / 8); i += kThreads) {
            const int r = i / (D / 8), d0 = i % (D / 8) * 8, t = r / p.G;
            float a[8], x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) a[e] = acc[r * D + d0 + e] * corr[r];
            for (int j = 0; j < kTile; ++j) {
                if (at[j] < 0 || t >= n || j0 + j > pos + t) continue;
                load_row8<D>(p.c.v, p.c.vs, p.c.fp8, at[j], d0, x);
#pragma unroll
                for (int e = 0; e < 8; ++e) a[e] = fmaf(sc[r * kTile + j], x[e], a[e]);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[r * D + d0 + e] = a[e];
        }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < R * D; i += kThreads) {
        const int r = i / D, d = i % D, t = r / p.G, hq = h * p.G + r % p.G;
        const long long bt = (long long)b * p.T + t;
        float o = l[r] == 0.0f ? 0.0f : acc[i] / l[r];
        if (p.gate.p != nullptr) o *= sigmoid(bf16_to_f32(p.gate.p[bt * p.gate.ts + hq * p.gate.hs + d]));
        p.out[(bt * p.Hq + hq) * D + d] = f32_to_bf16(o);
        if (d == 0 && p.lse != nullptr) p.lse[bt * p.Hq + hq] = (m[r] + log2f(l[r])) * kLn2;
    }
}

template <int D>
cudaError_t launch_t(const DecodeAttnParams &p, int B, cudaStream_t st) {
    const int R = p.T * p.G;
    const size_t smem = (size_t)(R * D + R * kTile + 3 * R + 1) * sizeof(float) + kTile * sizeof(long long) + 8;
    static unsigned long long done = 0;
    cudaError_t e = set_max_smem(done, attn_decode_kernel<D>, 128 * (D + kTile + 3) * sizeof(float) + 1024);
    if (e != cudaSuccess) return e;
    attn_decode_kernel<D><<<dim3(p.Hkv, B), kThreads, smem, st>>>(p);
    return cudaGetLastError();
}

}  // namespace

size_t attn_decode_workspace(const AttnSizes &) { return 256; }

cudaError_t launch_attn_decode(const AttnSizes &s, const uint16_t *q, const PagedCache &c, const int32_t *pos,
                               const int32_t *n_new, const HeadsIn &gate, float scale, uint16_t *out, float *lse,
                               void *, unsigned *err, cudaStream_t st) {
    const DecodeAttnParams p{q, c, pos, n_new, gate, out, lse, err, s.T, s.Hq, s.Hkv, s.Hq / s.Hkv, scale * kLog2e};
    if (s.D == 64) return launch_t<64>(p, s.B, st);
    if (s.D == 128) return launch_t<128>(p, s.B, st);
    return launch_t<256>(p, s.B, st);
}

}  // namespace gdn
