// Drafted tokens against the target's probabilities, from given random
// numbers.  A drafted token x stands while u q(x) < p(x) (that is, with the
// probability min(1, p / q)); the token after the last one that stands is drawn
// from what the target has above the draft, max(p - q, 0), or from the target's
// next row where all stand: the first token whose cumulative sum is above u
// times the whole.  Tokens so kept and drawn are distributed as the target's.
//
// Two numbers are read for each drafted token; then one row of V probabilities
// (two where a token fell) per batch row: HBM-bound.  A row is spread over a
// cluster of CTAs, each warp has a contiguous piece and sums it; the sums meet
// in distributed shared memory, and the warp whose piece holds the drawn token
// goes over its piece once more.
//
// Sums are 64-bit integers in units of 2^-60: exact whatever their order, so
// that a token does not depend on how a row is split.  Probabilities from 2^-37
// on enter exactly, smaller ones rounded to the unit.
//
// B = 128, four drafts, V = 131072, half of the rows with a draft's row to read
// (125 MB): 29.1 us, 4.3 TB/s.  The reads' own time is 18.5 us.  About half of the
// rest is the launch, the chain of three loads before a row is known, the clusters'
// meeting and the second look at a piece (what one row takes, 5.4 us); the other
// half is that a thread has eight loads (sixteen with a draft) in flight, 32 to
// 64 KB an SM, and none while it sums their digits.  One row of 32003: 5.4 us, a
// launch and a chain of five loads.
#include <cooperative_groups.h>

#include "attn.cuh"

namespace gdn {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32, kAhead = 8, kBatch = 32 * kAhead, kMostCtas = 8;

struct Params {
    const float *target, *draft, *u;
    const int32_t *tokens, *n;
    int32_t *out, *keep;
    int T, V;
};

using Sum = unsigned long long;

// Two f32 in one register pair.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 pair(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ F2 add(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 less(F2 a, F2 b) {   // a - b
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(b.v), "l"(pair(-1.0f, -1.0f).v), "l"(a.v));
    return r;
}
__device__ __forceinline__ int bits_apart(F2 x) {   // the first's bits less the second's
    int a, b;
    asm("mov.b64 {%0, %1}, %2;" : "=r"(a), "=r"(b) : "l"(x.v));
    return a - b;
}

// What a number counts as: its nearest value in [0, 1], NaN as 0.
__device__ __forceinline__ float probability(float x) { return fminf(fmaxf(x, 0.0f), 1.0f); }

// p - min(p, q) in whole units of 2^-60 (each of the two rounded to them), as
// three digits: of 2^-23, 2^-46 and 2^-60.  Adding 1 (1.5 2^-23, 1.5 2^-37) to a
// value below it leaves the value's multiple of 2^-23 (2^-46, 2^-60) in the
// sum's bits and, taken off again, an exact rest for the next digit; of p and
// min(p, q) at once, so that what was added cancels.  NaN and what is below 0
// count as 0, what is above 1 as 1.  (A conversion to 64-bit integers runs on
// this GPU's few double-precision units, shifts take three times as many
// instructions: 73 and 38 us for the largest case.)
struct Digits {
    int a, b, c;
    __device__ __forceinline__ void add_above(float p, float q) {
        p = probability(p);
        const F2 one = pair(1.0f, 1.0f), next = pair(1.5f * 0x1p-23f, 1.5f * 0x1p-23f), last = pair(1.5f * 0x1p-37f, 1.5f * 0x1p-37f);
        const F2 x = pair(p, fminf(p, fmaxf(q, 0.0f)));
        const F2 s = add(x, one), rest = less(x, less(s, one));
        const F2 s2 = add(rest, next), rest2 = less(rest, less(s2, next));
        a += bits_apart(s);
        b += bits_apart(s2);
        c += bits_apart(add(rest2, last));
    }
    __device__ __forceinline__ Sum value() const {
        return (Sum)(((long long)a << 37) + ((long long)b << 14) + (long long)c);
    }
};

// What is drawn from: p, or p above q, or p without one token.
struct Rest {
    const float *p, *q;
    int without;
};

__device__ __forceinline__ Sum warp_total(Sum v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// The sum of the lanes before.
__device__ __forceinline__ Sum warp_before(Sum v) {
    Sum s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const Sum y = __shfl_up_sync(0xffffffffu, s, o);
        if ((threadIdx.x & 31) >= o) s += y;
    }
    return s - v;
}

// The largest integer not above u * total, below total: a cumulative sum is
// above u * total if it is above this.
__device__ __forceinline__ Sum threshold(float u, Sum total) {
    if (!(u > 0.0f)) return 0ull;
    if (u >= 1.0f) return total - 1;
    const uint32_t bits = __float_as_uint(u);
    const int e = (int)(bits >> 23);
    const Sum m = e == 0 ? bits : (bits & 0x7fffffu) | 0x800000u;
    const int s = 150 - (e == 0 ? 1 : e);   // u = m 2^-s, s >= 24
    const Sum hi = __umul64hi(m, total), lo = m * total;
    if (s < 64) return (hi << (64 - s)) | (lo >> s);
    return s < 128 ? hi >> (s - 64) : 0ull;
}

__global__ void __launch_bounds__(kThreads, 2) spec_verify_kernel(const Params p) {
    cg::cluster_group cluster = cg::this_cluster();
    __shared__ Sum sums[kMostCtas][kWarps];   // of all warps of the row's CTAs
    __shared__ int stands;
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank(), warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long b = blockIdx.x / ctas;
    const int T = p.T, V = p.V;
    cluster_arrive_relaxed();   // (this CTA runs: the others may write its sums; they wait for that before they do)
    attn::grid_dep_enter();
    const float *target = p.target + b * (T + 1) * V, *draft = p.draft == nullptr ? nullptr : p.draft + b * T * V;
    const int32_t *tokens = p.tokens + b * T;
    const int n = p.n == nullptr ? T : min(max(p.n[b], 0), T);
    if (warp == 0) {
        int a = 0;
        for (int t0 = 0; t0 < n; t0 += 32) {
            const int t = t0 + lane;
            bool ok = false;
            if (t < n) {
                const int x = tokens[t];
                if (x >= 0 && x < V) {
                    const float q = draft == nullptr ? 1.0f : probability(draft[(long long)t * V + x]);
                    // (both sides exact in 64 bits)
                    ok = (double)p.u[b * (T + 1) + t] * (double)q < (double)probability(target[(long long)t * V + x]);
                }
            }
            const unsigned m = __ballot_sync(0xffffffffu, ok);
            const int run = __ffs(~m) - 1;   // (-1: all 32)
            a += run < 0 ? 32 : run;
            if (run >= 0) break;
        }
        if (lane == 0) stands = a < n ? a : n;
    }
    __syncthreads();
    const int a = stands;
    if (rank == 0) {
        for (int t = threadIdx.x; t <= T; t += kThreads)
            p.out[b * (T + 1) + t] = t < a ? tokens[t] : t == a ? 0 : -1;   // (what is drawn comes after the clusters have met)
        if (threadIdx.x == 0) p.keep[b] = a + 1;
    }
    Rest rest{target + (long long)a * V, a < n && draft != nullptr ? draft + (long long)a * V : nullptr,
              a < n && draft == nullptr ? tokens[a] : -1};
    // the warp's piece, in up to 32 chunks of whole batches; lane c remembers chunk c's sum
    const int pieces = ctas * kWarps, piece = rank * kWarps + warp;
    const int batches = (V + kBatch - 1) / kBatch, each = (batches + pieces - 1) / pieces;
    const int chunk = (each + 31) / 32 * kBatch;
    const long long start = (long long)piece * each * kBatch;
    const int first = (int)min(start, (long long)V), last = (int)min(start + (long long)each * kBatch, (long long)V);
    // the batch of 32 x kAhead tokens from i: token i + 32 k + lane by use(k, p, q)
    auto batch = [&](int i, auto &&use) {
        float x[kAhead], y[kAhead];
        const float *p0 = rest.p + i + lane, *q0 = rest.q + i + lane;
        if (i + kBatch <= last) {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) x[k] = p0[k * 32];
            if (rest.q != nullptr) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) y[k] = q0[k * 32];
            } else {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) y[k] = 0.0f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const bool there = i + k * 32 + lane < last;
                x[k] = there ? p0[k * 32] : 0.0f;
                y[k] = there && rest.q != nullptr ? q0[k * 32] : 0.0f;
            }
        }
        if (rest.without >= i && rest.without < i + kBatch)
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (i + k * 32 + lane == rest.without) x[k] = 0.0f;
#pragma unroll
        for (int k = 0; k < kAhead; ++k) use(k, x[k], y[k]);
    };
    Sum total = 0, before = 0, mine = 0, of_chunk = 0;
    for (int round = 0; round < 2; ++round) {
        of_chunk = 0;
        for (int c = 0, i = first; i < last; ++c) {
            Sum s = 0;
            for (const int end = min(i + chunk, last); i < end; i += kBatch) {
                Digits d{0, 0, 0};
                batch(i, [&](int, float p, float q) { d.add_above(p, q); });
                s += d.value();
            }
            s = warp_total(s);
            if (lane == c) of_chunk = s;
        }
        mine = warp_total(of_chunk);
        if (round == 0) cluster_wait_acquire();
        if (lane < ctas) *cluster.map_shared_rank(&sums[rank][warp], lane) = mine;
        cluster.sync();
        total = before = 0;
        for (int k = lane; k < pieces; k += 32) {
            const Sum v = sums[k / kWarps][k % kWarps];
            total += v;
            if (k < piece) before += v;
        }
        total = warp_total(total);
        before = warp_total(before);
        cluster.sync();   // (the sums' readers, and no CTA leaves before its sums are written)
        if (total != 0 || (rest.q == nullptr && rest.without < 0)) break;
        rest.q = nullptr;   // nothing above the draft: the target itself
        rest.without = -1;
    }
    int32_t *to = p.out + b * (T + 1) + a;
    if (total == 0) return;
    const Sum x = threshold(p.u[b * (T + 1) + T], total);
    if (x < before || x >= before + mine) return;
    // this piece: the chunk, then the batch's lines of 32, then the lane
    Sum c = before + warp_before(of_chunk);
    const int hit = __ffs(__ballot_sync(0xffffffffu, x >= c && x < c + of_chunk)) - 1;
    if (hit < 0) return;   // (sums that passed 64 bits, of rows that are no probabilities: token 0 stands)
    c = __shfl_sync(0xffffffffu, c, hit);
    const int end = min(first + (hit + 1) * chunk, last);
    for (int i = first + hit * chunk; i < end; i += kBatch) {
        Sum v[kAhead];
        batch(i, [&](int k, float p, float q) {
            Digits d{0, 0, 0};
            d.add_above(p, q);
            v[k] = d.value();
        });
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const Sum line = warp_total(v[k]);
            if (x < c + line) {
                const Sum upto = c + warp_before(v[k]);
                if (x >= upto && x < upto + v[k]) *to = i + k * 32 + lane;
                return;
            }
            c += line;
        }
    }
}

}  // namespace

cudaError_t launch_spec_verify(int B, int T, int V, const float *target, const float *draft, const int32_t *tokens,
                               const float *u, const int32_t *n, int32_t *tokens_out, int32_t *keep, cudaStream_t st) {
    const Params p{target, draft, u, tokens, n, tokens_out, keep, T, V};
    // One wave of two CTAs an SM, a batch for every warp at least (128 rows of 131072: 29.4 us; two waves 33.5, CTAs of half the
    // size, four an SM, 29.7, three an SM with half the loads ahead 35.9).
    const int room = 2 * num_sms() / B, full = (V + kWarps * kBatch - 1) / (kWarps * kBatch);
    int ctas = room < full ? room : full;
    ctas = ctas < 1 ? 1 : ctas > kMostCtas ? kMostCtas : ctas;
    if ((long long)B * ctas > 0x7fffffffLL) return cudaErrorNotSupported;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(B * ctas));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, spec_verify_kernel, p);
}

}  // namespace gdn

extern "C" gdn_status gdn_spec_verify(int32_t B, int32_t T, int32_t V, const float *target, const float *draft,
                                      const int32_t *tokens, const float *u, const int32_t *n, int32_t *tokens_out,
                                      int32_t *keep, gdn_stream stream) {
    auto ok = [](const void *p, bool needed) { return (reinterpret_cast<uintptr_t>(p) & 3) == 0 && (!needed || p != nullptr); };
    if (B < 0 || T < 0 || V <= 0) return GDN_ERR_INVALID_ARG;
    if (T > 1023 || V > (1 << 24)) return GDN_ERR_UNSUPPORTED;
    const bool some = B > 0;
    if (!ok(target, some) || !ok(draft, false) || !ok(tokens, some && T > 0) || !ok(u, some) || !ok(n, false) ||
        !ok(tokens_out, some) || !ok(keep, some))
        return GDN_ERR_INVALID_ARG;
    if (!some) return GDN_OK;
    const cudaError_t e = gdn::launch_spec_verify(B, T, V, target, draft, tokens, u, n, tokens_out, keep, (cudaStream_t)stream);
    return e == cudaSuccess ? GDN_OK : e == cudaErrorNotSupported ? GDN_ERR_UNSUPPORTED : GDN_ERR_CUDA;
}
