// Reading a paged cache back as bf16: positions start[b] .. start[b] + T - 1
// of every row.  A copy (and, of an e4m3 cache, one exact multiplication by
// the row's power of two): HBM-bound.  A warp takes one token: its page is
// looked up once, then up to ROWS * RPW key rows and the value rows beside
// them are asked for before the first is written (eight channels a lane).
// B = 8, up to 4093 positions of 2 heads of 256 channels from e4m3 (92 MB): 16.5 us.
#include <type_traits>

#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

struct ReadParams {
    PagedCache c;
    const int32_t *start, *n;
    uint16_t *k_out, *v_out;
    unsigned *err;
    int B, T, Hkv;
};

template <int D, bool FP8, int ROWS>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadParams p, unsigned items, unsigned chunks) {
    constexpr int LPR = D / 8, RPW = 32 / LPR;
    const int lane = threadIdx.x & 31;
    const unsigned item = blockIdx.x * 8 + (threadIdx.x >> 5);
    grid_dep_enter();
    if (item >= items) return;
    const unsigned bt = item / chunks, chunk = item - bt * chunks;
    const int b = (int)(bt / (unsigned)p.T), t = (int)(bt - (unsigned)b * p.T);
    const int h0 = (int)chunk * ROWS * RPW + lane / LPR, d0 = (lane % LPR) * 8;
    long long at = -1;   // the cache row of head 0
    if (t < clamp_new(p.n, b, p.T)) {
        at = cache_row(p.c, p.Hkv, p.c.table + (long long)b * p.c.width, (long long)p.start[b] + t, 0);
        if (at < 0 && lane == 0) atomicOr(p.err, kErrBadPage);
    }
    using Raw = typename std::conditional<FP8, uint2, uint4>::type;
    Raw raw[2][ROWS];
    uint32_t scale[2][ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int h = h0 + u * RPW;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            raw[v][u] = Raw{};
            scale[v][u] = 127;
            if (at >= 0 && h < p.Hkv) {
                const long long row = at + ((long long)h << p.c.shift);
                const char *pages = static_cast<const char *>(v ? p.c.v : p.c.k);
                raw[v][u] = *reinterpret_cast<const Raw *>(pages + (row * D + d0) * (FP8 ? 1 : 2));
                if (FP8) scale[v][u] = (v ? p.c.vs : p.c.ks)[row];
            }
        }
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
        const int h = h0 + u * RPW;
        if (h >= p.Hkv) break;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
            uint4 o;
            if constexpr (FP8) {
                float x[8];
                unpack8_e4m3(raw[v][u], x);
                const float s = e8m0_value(scale[v][u]);
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] *= s;
                o = pack8(x);
            } else {
                o = raw[v][u];
            }
            *reinterpret_cast<uint4 *>((v ? p.v_out : p.k_out) + ((long long)bt * p.Hkv + h) * D + d0) = o;
        }
    }
}

template <int D, bool FP8>
cudaError_t launch_read(const ReadParams &p, cudaStream_t st) {
    constexpr int ROWS = 2, RPW = 32 / (D / 8);
    const unsigned chunks = (p.Hkv + ROWS * RPW - 1) / (ROWS * RPW);
    const unsigned long long items = (unsigned long long)p.B * p.T * chunks;
    if (items > 0xffffff00ull) return cudaErrorNotSupported;
    return DependentLaunch(dim3((unsigned)((items + 7) / 8)), dim3(256), 0, st)(kv_read_kernel<D, FP8, ROWS>, p,
                                                                                (unsigned)items, chunks);
}

template <int D>
cudaError_t launch_d(const ReadParams &p, cudaStream_t st) {
    return p.c.fp8 ? launch_read<D, true>(p, st) : launch_read<D, false>(p, st);
}

}  // namespace

cudaError_t launch_kv_read(const AttnSizes &s, const PagedCache &c, const int32_t *start, const int32_t *n,
                           uint16_t *k_out, uint16_t *v_out, unsigned *err, cudaStream_t st) {
    const ReadParams p{c, start, n, k_out, v_out, err, s.B, s.T, s.Hkv};
    if (s.D == 64) return launch_d<64>(p, st);
    if (s.D == 128) return launch_d<128>(p, st);
    return launch_d<256>(p, st);
}

}  // namespace gdn
