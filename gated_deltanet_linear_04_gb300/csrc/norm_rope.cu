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
// Every element is read and written once: HBM-bound, if a row of 256 channels
// takes a warp fewer than about 90 instructions (a load and a store of 512
// bytes take an SM 46 clocks).  So:
//   - D/8 lanes hold one head row, RPW = 32 / (D/8) rows a warp; a lane holds
//     two pieces of four channels (8 bytes each) that turn with each other: in
//     the half-split form i .. i+3 and R/2 + i .. R/2 + i+3, so no lane needs
//     another's channels.  The pieces of neighbouring lanes are adjacent.
//   - a warp takes one token and up to eight (backward: four) times RPW heads of
//     one kind: all their rows are asked for at once, into its shared memory
//     (cp.async), while it computes the token's angles (one or more per lane,
//     shared through shared memory) and multiplies them with the weights; then
//     each head row is y = rstd (x A + x' B), x' the partners.
//   - four rows' sums go over the lanes together; arithmetic goes two channels
//     at a time (f32x2 instructions).
// At B = 1, T = 8192, 16 + 2 heads of 256 channels (151 MB): 27.9 us forward (a plain
// copy of as much takes 23.5), 43.6 backward (227 MB).  Steps on the way: a warp per
// head row 89 us; four rows a warp, into registers, partners by shuffle, sincospi
// 31.4 (164 instructions a row, most of them a token's angles and addresses).
#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

constexpr int kThreads = 256, kWarps = kThreads / 32;

struct RowParams {
    HeadsIn q, k, v;
    const float *wq, *wk;
    const uint64_t *freqs;
    const int32_t *pos;     // dense: [B, T], not read with several axes; append: [B]
    const uint8_t *mask;
    const int32_t *n_new;
    const uint16_t *dq_out, *dk_out;
    uint16_t *q_out, *k_out;   // backward: dq, dk
    float *partial;            // backward: [2][gridDim.x][D]
    PagedCache c;
    unsigned *err;
    AxesIn axes;               // of a pair's position, if there are several
    int B, T, Hq, Hkv, R;
    int cq, ck;                // parts of a token's heads: of q, of k (and of v)
    int aq, ak;                // backward: CTAs of a part of q, of k
    float eps;
};

// Four sums over the LPR lanes of a head row at once: the first two exchanges
// halve the values as well as the lanes, so that 6 exchanges do what 20 would;
// f is applied to each sum by the lanes that end up with it.
template <int LPR, typename F>
__device__ __forceinline__ void row_sums4(float (&v)[4], F &&f) {
    const int lane = threadIdx.x & 31;
    constexpr int O1 = LPR / 2, O2 = LPR / 4;
    const bool b1 = lane & O1, b2 = lane & O2;
    const float s0 = (b1 ? v[2] : v[0]) + __shfl_xor_sync(0xffffffffu, b1 ? v[0] : v[2], O1);
    const float s1 = (b1 ? v[3] : v[1]) + __shfl_xor_sync(0xffffffffu, b1 ? v[1] : v[3], O1);
    float t = (b2 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, b2 ? s0 : s1, O2);
#pragma unroll
    for (int o = LPR / 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    t = f(t);
    const int base = lane & ~(LPR - 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __shfl_sync(0xffffffffu, t, base + (i & 2 ? O1 : 0) + (i & 1 ? O2 : 0));
}

template <int LPR>
__device__ __forceinline__ uint32_t row_max(uint32_t x) {
    if constexpr (LPR == 32) {
        return __reduce_max_sync(0xffffffffu, x);
    } else {
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
        return x;
    }
}

// max(a, |b|, |c|), a >= 0; a NaN if one of them is
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two f32 in one register pair.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 parts(F2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 swap2(F2 a) {
    const float2 x = parts(a);
    return f2(x.y, x.x);
}

// The eight channels of a lane: piece 0 is x[0], x[1], piece 1 is x[2], x[3].
struct Row {
    F2 x[4];
};
struct RawRow {
    uint2 p[2];
};

__device__ __forceinline__ Row unpack_row(const RawRow &r) {
    Row o;
    const uint32_t w[4] = {r.p[0].x, r.p[0].y, r.p[1].x, r.p[1].y};
#pragma unroll
    for (int i = 0; i < 4; ++i) o.x[i] = f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    return o;
}

__device__ __forceinline__ RawRow pack_row(const Row &x) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = parts(x.x[i]);
        w[i] = pack2(v.x, v.y);
    }
    return {{make_uint2(w[0], w[1]), make_uint2(w[2], w[3])}};
}

// Where a lane's pieces are: channels c[0] .. + 3 and c[1] .. + 3 of its row.
struct Pieces {
    int c[2];
    bool turns;
    template <int LPR, bool INTER>
    static __device__ __forceinline__ Pieces of(int R) {
        constexpr int D = LPR * 8;
        const int l = (threadIdx.x & 31) % LPR, r = R / 8;   // the first R/8 lanes turn
        Pieces p;
        p.turns = l < r;
        const int first = p.turns ? 0 : R, n = p.turns ? R : D - R, m = p.turns ? l : l - r;
        p.c[0] = first + 4 * m;
        p.c[1] = first + n / 2 + 4 * m;
        return p;
    }
};

// A turned channel is own * a + partner * b.  The partners of a lane's pair k:
// the other piece's (half-split), or its own two swapped (interleaved).
template <bool INTER>
__device__ __forceinline__ F2 partners(const Row &x, int k) {
    return INTER ? swap2(x.x[k]) : x.x[k ^ 2];
}

// a = cos and b = the sine with the sign of the channel's place in its pair
// (`back`: of the opposite turn) of the lane's channels at a position; 1 and 0
// for channels that do not turn.  The warp computes the angles together, into
// its table; four entries behind them hold (1, 0).  With several axes a pair
// turns by the token's position on its own.
template <bool INTER, bool AXES>
__device__ __forceinline__ void lane_angles(const RowParams &p, float2 *table, const Pieces &pc, unsigned bt,
                                            long long pos, bool back, Row &a, Row &b) {
    const int lane = threadIdx.x & 31, half = p.R / 2;
    __syncwarp();   // (the previous token's readers)
    for (int i = lane; i < half; i += 32) {
        long long at = pos;
        if (AXES) at = p.axes.pos[(long long)min((int)p.axes.axis[i], p.axes.n - 1) * p.B * p.T + bt];
        rope_angle(at, p.freqs[i], table[i].x, table[i].y);
    }
    if (lane < 4) table[half + lane] = make_float2(1.0f, 0.0f);
    __syncwarp();
    const float sg = back ? -1.0f : 1.0f;
    const float4 *t4 = reinterpret_cast<const float4 *>(table);
    if (INTER) {
        // a piece is two pairs: two entries, in order
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 t = t4[(pc.turns ? pc.c[i] / 2 : half) / 2];
            a.x[2 * i] = f2(t.x, t.x);
            a.x[2 * i + 1] = f2(t.z, t.z);
            b.x[2 * i] = f2(-sg * t.y, sg * t.y);
            b.x[2 * i + 1] = f2(-sg * t.w, sg * t.w);
        }
    } else {
        // the two pieces are four pairs: four entries
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 t = t4[(pc.turns ? pc.c[0] : half) / 2 + i];
            a.x[i] = a.x[2 + i] = f2(t.x, t.z);
            b.x[i] = f2(-sg * t.y, -sg * t.w);
            b.x[2 + i] = f2(sg * t.y, sg * t.w);
        }
    }
}

// y += partners * b in the lanes whose channels turn; in the others nothing is
// added (an infinity times a sine of 0 is not 0).
template <bool INTER>
__device__ __forceinline__ void add_turned(Row &y, const Row &x, const Row &b, bool turns) {
    asm("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %12, 0;\n\t"
        "@p fma.rn.f32x2 %0, %4, %8, %0;\n\t@p fma.rn.f32x2 %1, %5, %9, %1;\n\t"
        "@p fma.rn.f32x2 %2, %6, %10, %2;\n\t@p fma.rn.f32x2 %3, %7, %11, %3;\n\t}"
        : "+l"(y.x[0].v), "+l"(y.x[1].v), "+l"(y.x[2].v), "+l"(y.x[3].v)
        : "l"(partners<INTER>(x, 0).v), "l"(partners<INTER>(x, 1).v), "l"(partners<INTER>(x, 2).v),
          "l"(partners<INTER>(x, 3).v), "l"(b.x[0].v), "l"(b.x[1].v), "l"(b.x[2].v), "l"(b.x[3].v),
          "r"((uint32_t)turns));
}

__device__ __forceinline__ Row load_weights(const float *w, const Pieces &pc) {
    Row r;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float4 v = *reinterpret_cast<const float4 *>(w + pc.c[i]);
        r.x[2 * i] = f2(v.x, v.y);
        r.x[2 * i + 1] = f2(v.z, v.w);
    }
    return r;
}

// The sum of the products of two rows' channels, over the lanes of a head row.
__device__ __forceinline__ float dot_lane(const Row &a, const Row &b) {
    F2 s = mul2(a.x[0], b.x[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s = fma2(a.x[k], b.x[k], s);
    const float2 v = parts(s);
    return v.x + v.y;
}

enum { kDense = 0, kAppend = 1, kAppendE4M3 = 2 };

__device__ __forceinline__ void cp_async16(void *dst, const void *src, bool there) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(there ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int LEFT>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory");
}

template <int D, bool INTER, int MODE, int ROWS, bool AXES>
__global__ void __launch_bounds__(kThreads, 3) row_forward_kernel(const RowParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, GROUP = ROWS < 4 ? ROWS : 4;
    extern __shared__ __align__(16) uint16_t stages[];
    __shared__ __align__(16) float2 tables[kWarps][D / 2 + 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
    const unsigned bt = blockIdx.x * kWarps + warp, part = blockIdx.y;
    grid_dep_enter();
    if (bt >= (unsigned)(p.B * p.T)) return;
    const bool isq = part < (unsigned)p.cq, isv = MODE != kDense && part >= (unsigned)(p.cq + p.ck);
    const int h0 = (int)(isq ? part : isv ? part - p.cq - p.ck : part - p.cq) * ROWS * RPW + sub;
    const int H = isq ? p.Hq : p.Hkv, rows = H - h0;   // (of this lane's, RPW apart)
    int b = 0, t = 0;
    bool on;
    if (MODE == kDense) {
        on = p.mask == nullptr || p.mask[bt] != 0;
    } else {
        b = (int)(bt / (unsigned)p.T);
        t = (int)(bt - (unsigned)b * p.T);
        on = t < clamp_new(p.n_new, b, p.T);
    }
    uint16_t *ring = stages + warp * (ROWS * RPW * D);
    if (on) {
        const HeadsIn &in = isq ? p.q : isv ? p.v : p.k;
        const uint16_t *src = in.p + (long long)bt * in.ts + (long long)h0 * in.hs + (lane % LPR) * 8;
        const long long hop = RPW * in.hs;
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            if (u * RPW < rows + sub) {   // (a row of the warp)
                cp_async16(ring + u * RPW * D + lane * 8, src, u * RPW < rows);
                if (u * RPW + RPW < rows) src += hop;
            }
            if ((u + 1) % GROUP == 0) cp_async_commit();
        }
    }
    const Pieces pc = Pieces::of<LPR, INTER>(p.R);
    uint16_t *out = nullptr;
    if (isq || MODE == kDense) {
        out = (isq ? p.q_out + (long long)bt * p.Hq * D : p.k_out + (long long)bt * p.Hkv * D) + h0 * D;
        if (!on) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                if (u * RPW < rows)
                    *reinterpret_cast<uint4 *>(out + u * RPW * D + (lane % LPR) * 8) = make_uint4(0, 0, 0, 0);
            return;
        }
    } else if (!on) {
        return;
    }
    const long long pos = MODE != kDense ? (long long)p.pos[b] + t : AXES ? 0 : p.pos[bt];
    long long at = -1;   // the cache row of head h0
    if (MODE != kDense && !isq) {
        at = cache_row(p.c, p.Hkv, p.c.table + (long long)b * p.c.width, pos, 0);
        if (at < 0) {
            if (lane == 0) atomicOr(p.err, kErrBadPage);
            cp_async_wait<0>();
            return;
        }
        at += (long long)h0 << p.c.shift;
    }
    // y = rstd (x A + x' B), x' the partners' x: A = w cos, B = +- w' sin
    Row A, B;
    const float *wp = isq ? p.wq : p.wk;
    const bool norm = !isv && wp != nullptr;
    if (!isv) lane_angles<INTER, AXES>(p, tables[warp], pc, bt, pos, false, A, B);
    if (norm) {
        const Row w = load_weights(wp, pc);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            A.x[k] = mul2(A.x[k], w.x[k]);
            B.x[k] = mul2(B.x[k], partners<INTER>(w, k));
        }
    }
#pragma unroll
    for (int u0 = 0; u0 < ROWS; u0 += GROUP) {
        if (u0 + GROUP < ROWS)
            cp_async_wait<1>();
        else
            cp_async_wait<0>();
        __syncwarp();
        const int n = (rows + sub - u0 * RPW + RPW - 1) / RPW;   // rows of the group that hold a head
        if (n <= 0) break;
        Row xs[GROUP];
        float rstd[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
            if (u >= n) break;
            const uint16_t *src = ring + ((u0 + u) * RPW + sub) * D;
            RawRow raw;
#pragma unroll
            for (int i = 0; i < 2; ++i) raw.p[i] = *reinterpret_cast<const uint2 *>(src + pc.c[i]);
            xs[u] = unpack_row(raw);
            if (norm) rstd[u] = dot_lane(xs[u], xs[u]);
        }
        if (norm) row_sums4<LPR>(rstd, [&](float ss) { return rsqrtf(ss * (1.0f / D) + p.eps); });
#pragma unroll
        for (int u = 0; u < GROUP; ++u) {
            if (u >= n) break;
            const bool there = (u0 + u) * RPW < rows;
            Row &x = xs[u];
            if (!isv) {
                Row y;
#pragma unroll
                for (int k = 0; k < 4; ++k) y.x[k] = mul2(x.x[k], A.x[k]);
                add_turned<INTER>(y, x, B, pc.turns);
                x = y;
                if (norm) {
                    const F2 r2 = f2(rstd[u], rstd[u]);
#pragma unroll
                    for (int k = 0; k < 4; ++k) x.x[k] = mul2(y.x[k], r2);
                }
            }
            const long long row = at + ((long long)((u0 + u) * RPW) << p.c.shift);
            if (isq || MODE != kAppendE4M3) {
                const RawRow o = pack_row(x);
                uint16_t *dst = isq || MODE == kDense ? out + (u0 + u) * RPW * D
                                                      : static_cast<uint16_t *>(isv ? p.c.v : p.c.k) + row * D;
                if (there) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) *reinterpret_cast<uint2 *>(dst + pc.c[i]) = o.p[i];
                }
                continue;
            }
            float2 v[4];
            float most = 0.0f;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                v[k] = parts(x.x[k]);
                most = max_abs(most, v[k].x, v[k].y);
            }
            const uint32_t amax = row_max<LPR>(__float_as_uint(most));
            const uint32_t byte = e8m0_for(amax);
            const float inv = e8m0_inverse(byte);
            const float y[8] = {v[0].x * inv, v[0].y * inv, v[1].x * inv, v[1].y * inv,
                                v[2].x * inv, v[2].y * inv, v[3].x * inv, v[3].y * inv};
            const uint2 codes = pack8_e4m3(y);
            if (there) {
                uint8_t *dst = static_cast<uint8_t *>(isv ? p.c.v : p.c.k) + row * D;
                *reinterpret_cast<uint32_t *>(dst + pc.c[0]) = codes.x;
                *reinterpret_cast<uint32_t *>(dst + pc.c[1]) = codes.y;
                if (lane % LPR == 0) (isv ? p.c.vs : p.c.ks)[row] = (uint8_t)byte;
            }
        }
    }
}

constexpr int kCtasPerSm = 2;
constexpr int kStages = 2;   // backward: tokens of a warp in shared memory, one in work, one on its way
constexpr int kBwdRows = 4;

// Backward: a CTA belongs to one part of the heads (p.aq CTAs to each of q's, the
// first; p.ak to each of k's), its warps go from token to token; it sums its share
// of dw and leaves it in `partial`.
template <int D, bool INTER, bool AXES>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) row_backward_kernel(const RowParams p) {
    constexpr int LPR = D / 8, RPW = 32 / LPR, ROWS = kBwdRows, HALF = ROWS * RPW * D, STAGE = 2 * HALF;
    extern __shared__ __align__(16) uint16_t stages[];
    __shared__ __align__(16) float2 tables[kWarps][D / 2 + 4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, sub = lane / LPR;
    uint16_t *ring = stages + warp * kStages * STAGE;
    const int nq = p.cq * p.aq;
    const bool isq = (int)blockIdx.x < nq;
    const HeadsIn &in = isq ? p.q : p.k;
    const int H = isq ? p.Hq : p.Hkv, cta = isq ? blockIdx.x : blockIdx.x - nq, parts_n = isq ? p.cq : p.ck;
    const int h0 = cta % parts_n * ROWS * RPW + sub, rows = H - h0;
    const float *wp = isq ? p.wq : p.wk;
    const bool norm = wp != nullptr;
    const Pieces pc = Pieces::of<LPR, INTER>(p.R);
    grid_dep_enter();
    Row w, acc;
    if (norm) w = load_weights(wp, pc);
#pragma unroll
    for (int k = 0; k < 4; ++k) acc.x[k] = f2(0.0f, 0.0f);
    const unsigned tokens = (unsigned)(p.B * p.T), step = (isq ? p.aq : p.ak) * kWarps;
    const uint16_t *x_p = in.p + (long long)h0 * in.hs + (lane % LPR) * 8;
    const uint16_t *dy_p = (isq ? p.dq_out : p.dk_out) + (long long)h0 * D + (lane % LPR) * 8;
    uint16_t *dx_p = (isq ? p.q_out : p.k_out) + (long long)h0 * D;

    auto ask = [&](unsigned bt, int stage) {
        if (p.mask != nullptr && p.mask[bt] == 0) return;
        const uint16_t *src = x_p + (long long)bt * in.ts, *dy = dy_p + (long long)bt * H * D;
        uint16_t *dst = ring + stage * STAGE + lane * 8;
#pragma unroll
        for (int u = 0; u < ROWS; ++u) {
            const bool there = u * RPW < rows;
            cp_async16(dst + u * RPW * D, there ? src + u * RPW * in.hs : in.p, there && norm);
            cp_async16(dst + HALF + u * RPW * D, there ? dy + u * RPW * D : dy_p, there);
        }
    };
    unsigned bt = cta / parts_n * kWarps + warp;
    if (bt < tokens) ask(bt, 0);
    cp_async_commit();
    for (int stage = 0; bt < tokens; bt += step, stage ^= 1) {
        if (bt + step < tokens) ask(bt + step, stage ^ 1);
        cp_async_commit();
        uint16_t *out = dx_p + (long long)bt * H * D;
        if (p.mask != nullptr && p.mask[bt] == 0) {
#pragma unroll
            for (int u = 0; u < ROWS; ++u)
                if (u * RPW < rows)
                    *reinterpret_cast<uint4 *>(out + u * RPW * D + (lane % LPR) * 8) = make_uint4(0, 0, 0, 0);
            continue;
        }
        Row a, b;
        lane_angles<INTER, AXES>(p, tables[warp], pc, bt, AXES ? 0 : p.pos[bt], true, a, b);
        cp_async_wait<1>();
        __syncwarp();
        const uint16_t *src = ring + stage * STAGE + sub * D;
#pragma unroll
        for (int u0 = 0; u0 < ROWS; u0 += 2) {
            if (u0 > 0 && u0 * RPW - sub >= rows) break;   // (no row of the warp)
            Row x[2], dz[2];
            float sums[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                RawRow rx, rdy;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    rx.p[i] = *reinterpret_cast<const uint2 *>(src + (u0 + u) * RPW * D + pc.c[i]);
                    rdy.p[i] = *reinterpret_cast<const uint2 *>(src + HALF + (u0 + u) * RPW * D + pc.c[i]);
                }
                const Row dy = unpack_row(rdy);
                x[u] = unpack_row(rx);
                // (channels that do not turn: a = 1)
#pragma unroll
                for (int k = 0; k < 4; ++k) dz[u].x[k] = mul2(dy.x[k], a.x[k]);
                add_turned<INTER>(dz[u], dy, b, pc.turns);
                if (!norm) continue;
                Row g;
#pragma unroll
                for (int k = 0; k < 4; ++k) g.x[k] = mul2(w.x[k], dz[u].x[k]);
                // x.x, and (w dz).x, which times rstd is (w dz).xhat
                sums[2 * u] = dot_lane(x[u], x[u]);
                sums[2 * u + 1] = dot_lane(g, x[u]);
            }
            if (norm) row_sums4<LPR>(sums, [](float t) { return t; });
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const bool there = (u0 + u) * RPW < rows;
                if (norm) {
                    float rstd = rsqrtf(sums[2 * u] * (1.0f / D) + p.eps);
                    if (!there) rstd = 0.0f;   // (a row that is not there; eps = 0 would make it an infinity)
                    const float m = -sums[2 * u + 1] * rstd * (1.0f / D);
                    const F2 r2 = f2(rstd, rstd), m2 = f2(m, m);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const F2 xhat = mul2(x[u].x[k], r2);
                        acc.x[k] = fma2(dz[u].x[k], xhat, acc.x[k]);
                        dz[u].x[k] = mul2(fma2(xhat, m2, mul2(w.x[k], dz[u].x[k])), r2);
                    }
                }
                const RawRow o = pack_row(dz[u]);
                if (there) {
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        *reinterpret_cast<uint2 *>(out + (u0 + u) * RPW * D + pc.c[i]) = o.p[i];
                }
            }
        }
        __syncwarp();   // (the stage is free for the next rows)
    }
    cp_async_wait<0>();
    if (!norm) return;
    __syncthreads();
    float *sum = reinterpret_cast<float *>(stages);   // [kWarps * RPW][D]: no more than the stages
    static_assert(kWarps * RPW * D * 4 <= kWarps * kStages * STAGE * 2, "");
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 v = parts(acc.x[k]);
        *reinterpret_cast<float2 *>(sum + (warp * RPW + sub) * D + pc.c[k >> 1] + 2 * (k & 1)) = v;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float t = 0.0f;
        for (int i = 0; i < kWarps * RPW; ++i) t += sum[i * D + d];
        p.partial[(size_t)blockIdx.x * D + d] = t;
    }
}

// dw = the CTAs' shares: 32 threads per channel, each sums every 32nd of them, then
// their sums are added in order.  Blocks: (q or k, 32 channels).
__global__ void __launch_bounds__(1024) weight_sum_kernel(const float *partial, int nq, int n, int D, float *dwq,
                                                          float *dwk) {
    __shared__ float sum[32][33];
    grid_dep_enter();
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

template <int D, bool INTER, int MODE, int ROWS, bool AXES>
cudaError_t launch_forward_axes(RowParams p, cudaStream_t st) {
    constexpr int RPW = 32 / (D / 8);
    constexpr size_t smem = (size_t)kWarps * ROWS * RPW * D * 2;
    p.cq = chunks_of(p.Hq, ROWS * RPW);
    p.ck = chunks_of(p.Hkv, ROWS * RPW);
    const long long tokens = (long long)p.B * p.T, ctas = (tokens + kWarps - 1) / kWarps;
    if (tokens > 0x7fffffffLL - kWarps) return cudaErrorNotSupported;
    static unsigned long long done = 0;
    cudaError_t e = set_max_smem(done, row_forward_kernel<D, INTER, MODE, ROWS, AXES>, smem);
    if (e != cudaSuccess) return e;
    return DependentLaunch(dim3((unsigned)ctas, p.cq + p.ck * (MODE == kDense ? 1 : 2)), dim3(kThreads), smem,
                           st)(row_forward_kernel<D, INTER, MODE, ROWS, AXES>, p);
}

// (Positions on one axis have kernels of their own: asked at run time it takes a token 1 % longer, 2.5 % in the gradients.)
template <int D, bool INTER, int MODE, int ROWS>
cudaError_t launch_forward_rows(const RowParams &p, cudaStream_t st) {
    return p.axes.axis != nullptr ? launch_forward_axes<D, INTER, MODE, ROWS, true>(p, st)
                                  : launch_forward_axes<D, INTER, MODE, ROWS, false>(p, st);
}

// Eight rows a warp, or one where there are too few tokens to fill the GPU (16 +
// 2 heads of 256 channels: T = 128 3.5 and 2.7 us, 256 3.4 and 3.1, 512 3.8 and
// 4.8, 8192 26.7 and 46.0).
template <int D, int MODE>
cudaError_t launch_forward(const RowParams &p, bool inter, cudaStream_t st) {
    constexpr int RPW = 32 / (D / 8);
    const long long rows = (long long)p.B * p.T * (p.Hq + p.Hkv) / RPW;
    if (rows < 32LL * num_sms())
        return inter ? launch_forward_rows<D, true, MODE, 1>(p, st) : launch_forward_rows<D, false, MODE, 1>(p, st);
    return inter ? launch_forward_rows<D, true, MODE, 8>(p, st) : launch_forward_rows<D, false, MODE, 8>(p, st);
}

template <int D, bool INTER, bool AXES>
cudaError_t launch_backward_i(const RowParams &p, cudaStream_t st) {
    constexpr size_t smem = (size_t)kWarps * kStages * 2 * kBwdRows * 512;   // (a warp's rows: 512 bytes)
    static unsigned long long done = 0;
    cudaError_t e = set_max_smem(done, row_backward_kernel<D, INTER, AXES>, smem);
    if (e != cudaSuccess) return e;
    return DependentLaunch(dim3(p.cq * p.aq + p.ck * p.ak), dim3(kThreads), smem,
                           st)(row_backward_kernel<D, INTER, AXES>, p);
}

template <int D>
cudaError_t launch_backward_rows(const RowParams &p, bool inter, cudaStream_t st) {
    if (p.axes.axis != nullptr) return inter ? launch_backward_i<D, true, true>(p, st) : launch_backward_i<D, false, true>(p, st);
    return inter ? launch_backward_i<D, true, false>(p, st) : launch_backward_i<D, false, false>(p, st);
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
                     const uint64_t *freqs, const int32_t *pos, const AxesIn &axes) {
    RowParams p = {};
    p.q = q;
    p.k = k;
    p.wq = wq;
    p.wk = wk;
    p.freqs = freqs;
    p.axes = axes;
    p.pos = pos != nullptr ? pos : axes.pos;   // (several axes of which no pair turns: as one)
    p.B = s.B;
    p.T = s.T;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.R = s.Drot;
    p.eps = s.eps;
    return p;
}

// The backward pass's parts of the heads and the CTAs of each: in proportion to
// their work (a token's angles and addresses cost a warp as much as three rows),
// kCtasPerSm per SM in all, no more than there are tokens for.
struct BackwardGrid {
    int cq, ck, aq, ak;
    explicit BackwardGrid(const AttnSizes &s) {
        const int rows = kBwdRows * (32 / (s.D / 8));
        cq = chunks_of(s.Hq, rows);
        ck = chunks_of(s.Hkv, rows);
        const int rpw = 32 / (s.D / 8);
        const long long total = (long long)kCtasPerSm * num_sms();
        const long long work_q = 3 * cq + chunks_of(s.Hq, rpw), work_k = 3 * ck + chunks_of(s.Hkv, rpw);
        const long long most = ((long long)s.B * s.T + kWarps - 1) / kWarps;
        long long k = (2 * total * work_k / (work_q + work_k) + ck) / (2 * ck);   // (rounded)
        long long q = (total - (k < 1 ? 1 : k) * ck) / cq;
        if (k > most) k = most;
        if (q > most) q = most;
        aq = q < 1 ? 1 : (int)q;
        ak = k < 1 ? 1 : (int)k;
    }
};

}  // namespace

cudaError_t launch_qk_norm_rope(const AttnSizes &s, const HeadsIn &q, const HeadsIn &k, const float *wq,
                                const float *wk, const uint64_t *freqs, const int32_t *pos, const uint8_t *mask,
                                uint16_t *q_out, uint16_t *k_out, cudaStream_t st, const AxesIn &axes) {
    RowParams p = row_params(s, q, k, wq, wk, freqs, pos, axes);
    p.mask = mask;
    p.q_out = q_out;
    p.k_out = k_out;
    return launch_forward_d<kDense>(p, s.D, s.inter, st);
}

cudaError_t launch_kv_append(const AttnSizes &s, const HeadsIn &q, const HeadsIn &k, const HeadsIn &v,
                             const float *wq, const float *wk, const uint64_t *freqs, const PagedCache &c,
                             const int32_t *pos, const int32_t *n_new, uint16_t *q_out, unsigned *err,
                             cudaStream_t st, const AxesIn &axes) {
    RowParams p = row_params(s, q, k, wq, wk, freqs, pos, axes);
    p.v = v;
    p.c = c;
    p.n_new = n_new;
    p.q_out = q_out;
    p.err = err;
    return c.fp8 ? launch_forward_d<kAppendE4M3>(p, s.D, s.inter, st) : launch_forward_d<kAppend>(p, s.D, s.inter, st);
}

size_t qk_norm_rope_backward_workspace(const AttnSizes &s) {
    const BackwardGrid g(s);
    return (size_t)(g.cq * g.aq + g.ck * g.ak) * s.D * sizeof(float);
}

cudaError_t launch_qk_norm_rope_backward(const AttnSizes &s, const HeadsIn &q, const HeadsIn &k, const float *wq,
                                         const float *wk, const uint64_t *freqs, const int32_t *pos,
                                         const uint8_t *mask, const uint16_t *dq_out, const uint16_t *dk_out,
                                         uint16_t *dq, uint16_t *dk, float *dwq, float *dwk, void *ws,
                                         cudaStream_t st, const AxesIn &axes) {
    RowParams p = row_params(s, q, k, wq, wk, freqs, pos, axes);
    p.mask = mask;
    p.dq_out = dq_out;
    p.dk_out = dk_out;
    p.q_out = dq;
    p.k_out = dk;
    p.partial = static_cast<float *>(ws);
    const BackwardGrid g(s);
    p.cq = g.cq;
    p.ck = g.ck;
    p.aq = g.aq;
    p.ak = g.ak;
    const int nq = g.cq * g.aq, nk = g.ck * g.ak;
    if ((long long)s.B * s.T > 0x7fffffffLL - (long long)(g.aq + g.ak) * kWarps) return cudaErrorNotSupported;
    cudaError_t e = s.D == 64    ? launch_backward_rows<64>(p, s.inter, st)
                    : s.D == 128 ? launch_backward_rows<128>(p, s.inter, st)
                                 : launch_backward_rows<256>(p, s.inter, st);
    if (e != cudaSuccess || wq == nullptr) return e;
    return DependentLaunch(dim3(2, s.D / 32), dim3(32, 32), 0, st)(weight_sum_kernel, (const float *)p.partial, nq,
                                                                   nq + nk, (int)s.D, dwq, dwk);
}

}  // namespace gdn
