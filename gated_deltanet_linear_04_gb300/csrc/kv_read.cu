// Reading a paged cache back as bf16: positions start[b] .. start[b] + T - 1
// of every row.  A copy (and, of an e4m3 cache, one exact multiplication by
// the row's power of two): HBM-bound.  One thread per eight channels of a key
// and of the value beside it.
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

template <int D>
__device__ __forceinline__ uint4 load8(const void *pages, const uint8_t *scale, bool fp8, long long at, int d0) {
    if (!fp8) return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(pages) + at * D + d0);
    float x[8];
    unpack8_e4m3(*reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(pages) + at * D + d0), x);
    const float s = e8m0_value(scale[at]);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= s;
    return pack8(x);
}

template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const ReadParams p) {
    constexpr int LPR = D / 8;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    const long long row = i / LPR;   // (b, t, h)
    const int d0 = (int)(i % LPR) * 8;
    if (row >= (long long)p.B * p.T * p.Hkv) return;
    const int h = (int)(row % p.Hkv);
    const long long bt = row / p.Hkv;
    const int b = (int)(bt / p.T), t = (int)(bt % p.T);
    uint4 k = make_uint4(0, 0, 0, 0), v = k;
    if (t < clamp_new(p.n, b, p.T)) {
        const long long at = cache_row(p.c, p.Hkv, p.c.table + (long long)b * p.c.width, (long long)p.start[b] + t, h);
        if (at < 0) {
            if (d0 == 0) atomicOr(p.err, kErrBadPage);
        } else {
            k = load8<D>(p.c.k, p.c.ks, p.c.fp8, at, d0);
            v = load8<D>(p.c.v, p.c.vs, p.c.fp8, at, d0);
        }
    }
    *reinterpret_cast<uint4 *>(p.k_out + row * D + d0) = k;
    *reinterpret_cast<uint4 *>(p.v_out + row * D + d0) = v;
}

}  // namespace

cudaError_t launch_kv_read(const AttnSizes &s, const PagedCache &c, const int32_t *start, const int32_t *n,
                           uint16_t *k_out, uint16_t *v_out, unsigned *err, cudaStream_t st) {
    const ReadParams p{c, start, n, k_out, v_out, err, s.B, s.T, s.Hkv};
    const long long threads = (long long)s.B * s.T * s.Hkv * (s.D / 8);
    const long long grid = (threads + 255) / 256;
    if (grid > 0x7fffffffLL) return cudaErrorNotSupported;
    if (s.D == 64) kv_read_kernel<64><<<(unsigned)grid, 256, 0, st>>>(p);
    else if (s.D == 128) kv_read_kernel<128><<<(unsigned)grid, 256, 0, st>>>(p);
    else kv_read_kernel<256><<<(unsigned)grid, 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace gdn
