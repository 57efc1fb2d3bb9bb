// Attention of 1..8 new tokens per row over the paged cache.
//
// Per query row: s_j = scale q.k_j over the visible positions, out =
// sum_j 2^(s'_j - m) v_j / sum_j 2^(s'_j - m) with s' = s log2(e) and m a
// running maximum: one pass over the keys and values, HBM-bound (16 flop per
// byte for 8 query heads per key head, bf16).
//
// Work.  A unit is one (row b, key head h, block of at most 64 of its T * Hq/Hkv
// query rows); its keys come in tiles of KT.  The tiles of all units form one
// list, cut into equal shares for one CTA per SM, so ragged batches and a
// single long row both fill the GPU; each CTA finds its share from pos / n_new
// itself.  A unit that crosses shares leaves partial results (m, sum, weighted
// sum) in the workspace, and a second kernel joins them in share order.
//
// CTA.  One warp keeps a ring of tiles filled with TMA box loads (a box: the
// tokens of one page, or KT of them, 128-byte swizzled; a page that does not
// exist is skipped and marked).  Consumer warps are RG groups of 8*NT query
// rows times KL lanes: a tile goes to the RG warps of one lane, which keep
// their own running maximum, sum and weighted sum, so nothing but the ring's
// barriers is waited for inside a unit.  At its end the lanes are joined in
// order through shared memory.
//
// Products.  mma.sync m16n8k16 with keys (then channels) as the 16 and query
// rows as the 8: S^T = K Q^T, O^T = V^T P^T.  Eight heads per key head fill
// n = 8 exactly, where a 128-row tcgen05 tile would hold 8 rows of use, and
// the tensor work is far from the bound.  S^T becomes P^T's operand by one
// movmatrix per 8x8 block.  e4m3 codes are turned into f16 pairs on the way
// from shared memory to the operand (exactly); their scales go to the scores
// (keys) and into the exponent of the weights (values).
#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxRows = 64;      // query rows of a unit
constexpr int kMinTiles = 4;      // least tiles of a share
constexpr int kMaxStages = 24;
constexpr int kSmemLimit = 227 * 1024;

template <int D_, bool FP8_>
struct Geo {
    static constexpr int D = D_;
    static constexpr bool FP8 = FP8_;
    static constexpr int ROWB = FP8 ? D : 2 * D;               // bytes of a key
    static constexpr int SUBB = ROWB < 128 ? ROWB : 128;       // ... in sub-tiles of one swizzle span
    static constexpr int NSUB = ROWB / SUBB;
    static constexpr int KT = FP8 ? (D == 256 ? 32 : 64) : 4096 / D;   // keys of a tile
    static constexpr int MT = KT / 16;
    static constexpr int KV = KT * ROWB;                       // bytes of a tile's keys
    static constexpr int STAGE = 2 * KV;
    static constexpr int OSTR = D + 4;                         // row stride of a join buffer (floats)
};

struct Params {
    const uint16_t *q;
    PagedCache c;
    const int32_t *pos, *n_new;
    HeadsIn gate;
    uint16_t *out;
    float *lse;
    float *part_o;      // [2 * ctas][rows][D]
    float2 *part_ml;    // [2 * ctas][rows]
    int *meta;          // [ctas][3]: the unit that starts in the share and goes on (or -1), its last share, its slot
    unsigned *err;
    int B, T, Hq, Hkv, G, R;
    int RB, rows;       // row blocks of a (b, h), query rows of one
    int RG, KL, stages, box_log2, copies;
    float scale2;       // scale * log2(e)
};

// Offsets into dynamic shared memory (after the ring).
struct Layout {
    int qf, obuf, ml, qscale, scales, total;
};

template <class G>
__host__ __device__ Layout layout(int RG, int NT, int KL, int copies, int stages) {
    const int rows = RG * NT * 8;
    Layout l;
    l.qf = stages * G::STAGE;
    l.obuf = l.qf + rows * G::D * 2;
    l.ml = l.obuf + copies * rows * G::OSTR * 4;
    l.qscale = l.ml + KL * rows * 8;
    l.scales = l.qscale + rows * 4;
    l.total = l.scales + (G::FP8 ? stages * 2 * G::KT : 0);
    return l;
}

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// The 8x8 matrix of 16-bit values held by the warp, transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

// d += a (16x16) b (16x8); f16 operands for an e4m3 cache, else bf16.
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four e4m3 codes as two f16 pairs, exactly.
__device__ __forceinline__ void codes_f16(uint32_t x, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(x));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack16(float a, float b) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    return pack2(a, b);
}

template <class G>
__device__ __forceinline__ uint32_t sub_offset(int chunk, int substride) {
    return (uint32_t)(chunk / (G::SUBB / 16)) * substride;
}

__device__ __forceinline__ void consumer_sync(int threads) {
    asm volatile("bar.sync 1, %0;" ::"r"(threads) : "memory");
}

// The keys of row b (the new tokens' own included) and its tiles; a row
// without keys still has one, empty, tile, so that its outputs get written.
struct RowLen {
    long long pos, keys;
    int n, tiles;
    bool short_table;   // some of its positions have no page
};

template <class G>
__device__ __forceinline__ RowLen row_len(const Params &p, int b) {
    RowLen r;
    r.n = clamp_new(p.n_new, b, p.T);
    r.pos = p.pos[b];
    const long long want = r.n == 0 ? 0 : max(r.pos + r.n, 0LL);
    r.keys = min(min(want, (long long)p.c.width << p.c.shift), 0x7fffff00LL);   // (key indexes are 32 bits)
    r.short_table = r.n > 0 && (r.keys < want || r.pos < 0);
    r.tiles = (int)max((r.keys + G::KT - 1) / G::KT, 1LL);
    return r;
}

// The list of all units' tiles in `act` shares that differ by at most one
// tile, the longer ones first.
struct Shares {
    unsigned act, base, extra;   // base or base + 1 tiles; `extra` shares have one more

    __device__ Shares(unsigned total, unsigned ctas) {
        act = min(ctas, max(total / kMinTiles, 1u));
        base = total / act;
        extra = total - base * act;
    }
    __device__ unsigned start(unsigned c) const { return c * base + min(c, extra); }
    // the share that holds a tile
    __device__ unsigned of(unsigned tile) const {
        const unsigned cut = extra * (base + 1);
        return tile < cut ? tile / (base + 1) : extra + (tile - cut) / base;
    }
};

// Consumer warps at most: 11 and the producer leave 168 registers a thread,
// 7 leave 255, which the widest accumulators (16 rows of 256 channels) need.
template <class G, int NT>
constexpr int max_consumers() {
    return G::D * NT >= 512 ? 7 : 11;
}

template <class G, int NT>
__global__ void __launch_bounds__((max_consumers<G, NT>() + 1) * 32, 1) attn_decode_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                             const __grid_constant__ CUtensorMap tm_v,
                                                             const Params p) {
    constexpr int D = G::D, KT = G::KT, MT = G::MT;
    constexpr bool FP8 = G::FP8;
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) uint64_t full[kMaxStages], empty[kMaxStages];
    __shared__ uint32_t bad_boxes[kMaxStages];
    __shared__ unsigned warp_sum_sh[12], found_off;
    __shared__ int found_b;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int RG = p.RG, KL = p.KL, W = RG * KL, NST = p.stages;
    const Layout lay = layout<G>(RG, NT, KL, p.copies, NST);
    grid_dep_launch();
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], RG);
        }
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
        found_b = -1;
    }
    grid_dep_wait();

    // the share: prefix sums of the rows' tiles, blockDim rows at a time (twice, if that is not all of them)
    const int heads = p.Hkv * p.RB, nthr = blockDim.x, nwarp = nthr / 32;
    const bool once = p.B <= nthr;
    Shares sh(1, 1);
    unsigned start = 0;
    for (int pass = 0; pass < 2; ++pass) {
        unsigned run = 0;
        for (int base = 0; base < p.B; base += nthr) {
            const int b = base + tid;
            const unsigned v = b < p.B ? (unsigned)(row_len<G>(p, b).tiles * heads) : 0;
            unsigned x = v;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += y;
            }
            __syncthreads();   // (also: barrier initialisation, the previous chunk's readers)
            if (lane == 31) warp_sum_sh[warp] = x;
            __syncthreads();
            unsigned before = run, all = 0;
            for (int w = 0; w < nwarp; ++w) {
                if (w < warp) before += warp_sum_sh[w];
                all += warp_sum_sh[w];
            }
            if (once) {
                sh = Shares(all, gridDim.x);
                start = sh.start(blockIdx.x);
            }
            if ((pass == 1 || once) && b < p.B && before + x - v <= start && start < before + x) {
                found_b = b;
                found_off = start - (before + x - v);
            }
            run += all;
        }
        if (once) break;
        if (pass == 0) {
            sh = Shares(run, gridDim.x);
            start = sh.start(blockIdx.x);
        }
    }
    __syncthreads();
    if (blockIdx.x >= sh.act) {
        if (tid == 0) p.meta[3 * blockIdx.x] = -1;
        return;
    }
    int b = found_b;
    RowLen len = row_len<G>(p, b);
    int ui = (int)(found_off / (unsigned)len.tiles), ta = (int)(found_off % (unsigned)len.tiles);
    int left = (int)(sh.start(blockIdx.x + 1) - start);
    const int boxrows = 1 << p.box_log2;
    bool dead = false;

    if (warp == W) {
        // ---- producer -----------------------------------------------------
        const int bpt = KT >> p.box_log2, page_sh = p.c.shift - p.box_log2;   // boxes per tile; pages = boxes >> page_sh
        const uint32_t box_bytes = (uint32_t)boxrows * G::ROWB;
        const uint32_t tx = 2 * box_bytes + (FP8 ? 2 * boxrows : 0);
        int st = 0;
        uint32_t ph = 1;
        uint32_t used = 0;
        while (left > 0) {
            const int n = min(len.tiles - ta, left);
            const int h = ui / p.RB;
            const int32_t *line = p.c.table + (long long)b * p.c.width;
            const int nbox = (int)((len.keys + boxrows - 1) >> p.box_log2);
            const int npage = (int)((len.keys + p.c.page - 1) >> p.c.shift);
            if (len.short_table && lane == 0) atomicOr(p.err, kErrBadPage);
            // page numbers, 32 at a time, the next 32 on their way
            int w0 = ((ta * bpt) >> page_sh) & ~31;
            int cur = w0 + lane < npage ? line[w0 + lane] : -1;
            int nxt = w0 + 32 + lane < npage ? line[w0 + 32 + lane] : -1;
            for (int i = 0; i < n; ++i) {
                const int box0 = (ta + i) * bpt;
                if ((box0 >> page_sh) >= w0 + 32) {
                    w0 += 32;
                    cur = nxt;
                    nxt = w0 + 32 + lane < npage ? line[w0 + 32 + lane] : -1;
                }
                const int box = box0 + lane;
                const int page = __shfl_sync(0xffffffffu, cur, ((lane < bpt ? box : box0) >> page_sh) - w0);
                const bool want = lane < bpt && box < nbox;
                const bool ok = want && page >= 0 && page < p.c.n_pages;
                if (want && !ok) atomicOr(p.err, kErrBadPage);
                const uint32_t good = __ballot_sync(0xffffffffu, ok);
                if (!dead && !mbar_wait(&empty[st], ph, p.err)) dead = true;
                dead = __any_sync(0xffffffffu, dead);
                if (!dead) {
                    if (lane == 0) {
                        bad_boxes[st] = ~good & ((1u << bpt) - 1);
                        if (good != 0)
                            mbar_expect_tx(&full[st], __popc(good) * tx);
                        else
                            mbar_arrive(&full[st]);
                        used |= 1u << st;
                    }
                    __syncwarp();
                    if (ok) {
                        const int row =
                            (int)((((long long)page * p.Hkv + h) << p.c.shift) + (((long long)box << p.box_log2) & (p.c.page - 1)));
                        unsigned char *dst = smem + st * G::STAGE + lane * box_bytes;
                        tma_load_3d(dst, &tm_k, 0, row, 0, &full[st]);
                        tma_load_3d(dst + G::KV, &tm_v, 0, row, 0, &full[st]);
                        if (FP8) {
                            unsigned char *sc = smem + lay.scales + st * 2 * KT + lane * boxrows;
                            bulk_load(sc, p.c.ks + row, boxrows, &full[st]);
                            bulk_load(sc + KT, p.c.vs + row, boxrows, &full[st]);
                        }
                    }
                    if (++st == NST) {
                        st = 0;
                        ph ^= 1;
                    }
                }
            }
            left -= n;
            ta = 0;
            if (left > 0 && ++ui == heads) {
                ui = 0;
                len = row_len<G>(p, ++b);
            }
        }
        // after a wait that gave up: let the copies in flight land before the CTA ends
        if (dead && lane == 0) {
            for (int i = 0; i < NST; ++i) {
                if ((used >> i & 1) == 0) continue;
                const uint32_t phase = i < st ? ph ^ 1 : ph;   // the parity of stage i's last fill
                for (uint32_t k = 0; k < kSpinLimit && !mbar_try_wait(&full[i], phase); ++k) {
                }
            }
        }
        return;
    }

    // ---- consumers -----------------------------------------------------------
    const int rg = warp % RG, kl = warp / RG, threads = W * 32;
    const int g = lane >> 2, j = lane & 3;
    const int rows_pad = RG * NT * 8;
    uint2 *qf = reinterpret_cast<uint2 *>(smem + lay.qf);
    float *obuf = reinterpret_cast<float *>(smem + lay.obuf);
    float2 *ml = reinterpret_cast<float2 *>(smem + lay.ml);        // [KL][rows_pad]
    float *qscale = reinterpret_cast<float *>(smem + lay.qscale);
    const uint32_t ring = smem_u32(smem);
    // ldmatrix rows and 16-byte chunks of this lane: matrix mi holds rows (mi & 1) * 8 .. and chunk + (mi >> 1)
    // (keys; e4m3 values), or rows (mi >> 1) * 8 .. and chunk + (mi & 1) (bf16 values)
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t swz = G::SUBB == 128 ? mr : mr >> 1;
    const uint32_t k_row = ((mi & 1) * 8 + mr) * G::SUBB, k_x = ((mi >> 1) ^ swz) << 4;
    const uint32_t v_row = FP8 ? k_row : (uint32_t)((mi >> 1) * 8 + mr) * G::SUBB;
    const uint32_t v_x = FP8 ? k_x : (uint32_t)((mi & 1) ^ swz) << 4;
    const int substride = boxrows * G::SUBB;
    constexpr uint32_t XMASK = G::SUBB - 16;

    int it = 0;                       // tiles of this CTA before the unit
    int st = kl;                      // this lane's next tile: its stage and parity
    uint32_t ph = 0;
    int next = kl;                    // ... its number in the CTA
    bool first = true;
    if (tid == 0) p.meta[3 * blockIdx.x] = -1;
    while (left > 0) {
        const int n = min(len.tiles - ta, left);
        const int h = ui / p.RB, r0 = (ui % p.RB) * p.rows;
        const int nrows = min(p.rows, p.R - r0);
        const int n_new = len.n;

        // queries to operand order: 8 channels of a row per thread
        for (int i = tid; i < rows_pad * (D / 8); i += threads) {
            const int r = i / (D / 8), d0 = (i % (D / 8)) * 8;
            float x[8];
            uint4 raw = make_uint4(0, 0, 0, 0);
            if (r < nrows) {
                const int rr = r0 + r, t = rr / p.G, hq = h * p.G + rr % p.G;
                raw = *reinterpret_cast<const uint4 *>(p.q + (((long long)b * p.T + t) * p.Hq + hq) * D + d0);
            }
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            if (FP8) {
                // a power of two per row brings the largest query to [1, 4): f16 then holds every bit but those
                // below 2^-24 of it
                unpack8(raw, x);
                uint32_t top = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) top = max(top, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
                for (int o = D / 16; o > 0; o >>= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                int e2 = (int)(top >> 23);
                e2 = e2 == 255 || top == 0 ? 127 : min(max(e2, 1), 253);
                const float inv = __uint_as_float((uint32_t)(254 - e2) << 23);
#pragma unroll
                for (int e = 0; e < 4; ++e) w[e] = pack16<true>(x[2 * e] * inv, x[2 * e + 1] * inv);
                if (d0 == 0) qscale[r] = __uint_as_float((uint32_t)e2 << 23);
            }
            const int rt = r >> 3, rr = r & 7, ks = d0 >> 4, hi = (d0 >> 3) & 1;
            uint32_t *base = reinterpret_cast<uint32_t *>(qf) + ((((rt / NT) * (D / 16) + ks) * 32) * NT + rt % NT) * 2;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // bf16: k = 2e (+8 hi) of the 16; e4m3: channels 4j .. 4j+3 are k = 2j, 2j+1, 2j+8, 2j+9
                const int ln = rr * 4 + (FP8 ? hi * 2 + (e >> 1) : e), reg = FP8 ? e & 1 : hi;
                base[ln * NT * 2 + reg] = w[e];
            }
        }
        consumer_sync(threads);

        float acc[D / 16][NT][4];
        float m[NT][2], l[NT][2], mv[NT][2], rs[NT][2];
        int lim[NT][2];               // visible keys of the lane's query rows (relative to 0), 0 for none
#pragma unroll
        for (int a = 0; a < NT; ++a) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                m[a][c] = mv[a][c] = -INFINITY;
                l[a][c] = 0.0f;
                const int r = rg * NT * 8 + a * 8 + 2 * j + c;
                const int t = (r0 + r) / p.G;
                lim[a][c] = r < nrows && t < n_new ? (int)min(max(len.pos + t + 1, 0LL), len.keys) : 0;
                rs[a][c] = p.scale2 * (FP8 ? qscale[r] : 1.0f);
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[i][a][c] = 0.0f;
        }
        const int all_see = (int)min(max(len.pos + 1, 0LL), len.keys);   // keys that every live row sees
        const uint2 *myq = qf + (size_t)rg * (D / 16) * 32 * NT;

        for (; next < it + n; next += KL) {
            const int tile = ta + next - it;
            if (!dead && !mbar_wait(&full[st], ph, p.err)) dead = true;
            dead = __any_sync(0xffffffffu, dead);
            if (!dead) {
                const uint32_t kbase = ring + st * G::STAGE, vbase = kbase + G::KV;
                const uint32_t bad = bad_boxes[st];
                const int key0 = tile * KT;
                const bool tail = bad != 0 || key0 + KT > all_see;
                float s[MT][NT][4];
#pragma unroll
                for (int a = 0; a < MT; ++a)
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[a][c][e] = 0.0f;
                uint32_t mrow[MT];
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    const int k0 = a * 16;
                    mrow[a] = (uint32_t)(k0 >> p.box_log2) * (boxrows * G::ROWB) + (k0 & (boxrows - 1)) * G::SUBB;
                }
                // S^T = K Q^T
                if constexpr (!FP8) {
#pragma unroll 4
                    for (int ks = 0; ks < D / 16; ++ks) {
                        uint2 q[NT];
#pragma unroll
                        for (int c = 0; c < NT; ++c) q[c] = myq[(ks * 32 + lane) * NT + c];
                        const uint32_t off = sub_offset<G>(2 * ks, substride) + k_row + (k_x ^ ((ks * 32) & XMASK));
#pragma unroll
                        for (int a = 0; a < MT; ++a) {
                            uint32_t k[4];
                            ldsm4(kbase + mrow[a] + off, k);
#pragma unroll
                            for (int c = 0; c < NT; ++c) mma<false>(s[a][c], k[0], k[1], k[2], k[3], q[c].x, q[c].y);
                        }
                    }
                } else {
#pragma unroll 2
                    for (int ks = 0; ks < D / 16; ks += 2) {
                        uint2 q[2][NT];
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int c = 0; c < NT; ++c) q[e][c] = myq[((ks + e) * 32 + lane) * NT + c];
                        const uint32_t off = sub_offset<G>(ks, substride) + k_row + (k_x ^ ((ks * 16) & XMASK));
#pragma unroll
                        for (int a = 0; a < MT; ++a) {
                            uint32_t k[4];
                            ldsm4(kbase + mrow[a] + off, k);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                uint32_t a0, a1, a2, a3;
                                codes_f16(k[2 * e], a0, a2);
                                codes_f16(k[2 * e + 1], a1, a3);
#pragma unroll
                                for (int c = 0; c < NT; ++c) mma<true>(s[a][c], a0, a1, a2, a3, q[e][c].x, q[e][c].y);
                            }
                        }
                    }
                }
                // scores in units of log2, the unseen ones -inf
                float ve[MT][2];
#pragma unroll
                for (int a = 0; a < MT; ++a) {
                    float ksc[2] = {1.0f, 1.0f};
                    if (FP8) {
                        const unsigned char *sc = smem + lay.scales + st * 2 * KT + a * 16 + g;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            ksc[e] = e8m0_value(sc[e * 8]);
                            const int vb = sc[KT + e * 8];
                            ve[a][e] = vb == 255 ? __uint_as_float(0x7fffffffu) : (float)(vb - 127);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[a][c][e] *= rs[c][e & 1] * ksc[e >> 1];
                    if (tail) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = a * 16 + e * 8 + g;
                            const bool there = (bad >> (key >> p.box_log2) & 1) == 0;
                            if (FP8 && (!there || key0 + key >= len.keys)) ve[a][e] = 0.0f;
#pragma unroll
                            for (int c = 0; c < NT; ++c)
#pragma unroll
                                for (int x = 0; x < 2; ++x)
                                    if (!there || key0 + key >= lim[c][x]) s[a][c][2 * e + x] = -INFINITY;
                        }
                    }
                }
                // running maxima
                bool moved = false;
                float mnew[NT][2], mvnew[NT][2];
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float t = s[0][c][x], tv = -INFINITY;
#pragma unroll
                        for (int a = 0; a < MT; ++a) t = fmaxf(t, fmaxf(s[a][c][x], s[a][c][2 + x]));
                        if (FP8) {
#pragma unroll
                            for (int a = 0; a < MT; ++a)
#pragma unroll
                                for (int e = 0; e < 2; ++e)
                                    tv = fmaxf(tv, tail && s[a][c][2 * e + x] == -INFINITY ? -INFINITY
                                                                                       : s[a][c][2 * e + x] + ve[a][e]);
                        }
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) {
                            t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, o));
                            if (FP8) tv = fmaxf(tv, __shfl_xor_sync(0xffffffffu, tv, o));
                        }
                        mnew[c][x] = fmaxf(m[c][x], t);
                        mvnew[c][x] = FP8 ? fmaxf(mv[c][x], tv) : mnew[c][x];
                        moved |= mnew[c][x] > m[c][x] || (FP8 && mvnew[c][x] > mv[c][x]);
                    }
                if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float f = mnew[c][x] == -INFINITY ? 1.0f : ex2(m[c][x] - mnew[c][x]);
                            const float fv = !FP8 ? f : mvnew[c][x] == -INFINITY ? 1.0f : ex2(mv[c][x] - mvnew[c][x]);
                            l[c][x] *= f;
                            m[c][x] = mnew[c][x];
                            mv[c][x] = mvnew[c][x];
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                acc[i][c][x] *= fv;
                                acc[i][c][2 + x] *= fv;
                            }
                        }
                }
                // weights, and P^T in operand order
                uint32_t pf[MT][NT][2];
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    float base[2], basev[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        base[x] = m[c][x] == -INFINITY ? 0.0f : m[c][x];
                        basev[x] = mv[c][x] == -INFINITY ? 0.0f : mv[c][x];
                    }
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            float w[2];
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const float v = s[a][c][2 * e + x], wl = ex2(v - base[x]);
                                l[c][x] += wl;
                                w[x] = !FP8 ? wl : tail && v == -INFINITY ? 0.0f : ex2(v + ve[a][e] - basev[x]);
                            }
                            pf[a][c][e] = transpose8x8(pack16<FP8>(w[0], w[1]));
                        }
                }
                // O^T += V^T P^T; values of slots that hold no key are zeroed (0 times NaN is NaN)
                uint32_t keep[MT][2];
                bool window = false;          // a NaN or infinity among the values that only later tokens see
                if (tail) {
#pragma unroll
                    for (int a = 0; a < MT; ++a)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int key = a * 16 + e * 8 + 2 * j;
                            const bool there = (bad >> (key >> p.box_log2) & 1) == 0;
                            keep[a][e] = there ? (key0 + key < len.keys ? 0xffffu : 0u) |
                                                     (key0 + key + 1 < len.keys ? 0xffff0000u : 0u)
                                               : 0u;
                        }
                    if (p.T > 1) {
                        for (int key = max(all_see - key0, 0); key < KT && key0 + key < len.keys; ++key) {
                            if (bad >> (key >> p.box_log2) & 1) continue;
                            const unsigned char *row = smem + st * G::STAGE + G::KV +
                                                       (key >> p.box_log2) * (boxrows * G::ROWB) +
                                                       (key & (boxrows - 1)) * G::SUBB;
                            for (int i = lane; i < G::ROWB / 4; i += 32) {
                                const uint32_t x = *reinterpret_cast<const uint32_t *>(
                                    row + (i / (G::SUBB / 4)) * substride + (i % (G::SUBB / 4)) * 4);
                                if (FP8) {
                                    const uint32_t y = x & 0x7f7f7f7fu;
                                    window |= (y & 0xff) == 0x7f || (y & 0xff00) == 0x7f00 ||
                                              (y & 0xff0000) == 0x7f0000 || (y >> 24) == 0x7f;
                                } else {
                                    window |= (x & 0x7f80u) == 0x7f80u || (x & 0x7f800000u) == 0x7f800000u;
                                }
                            }
                        }
                        window = __any_sync(0xffffffffu, window);
                    }
                }
                if (!window) {
#pragma unroll
                    for (int a = 0; a < MT; ++a) {
                        if constexpr (!FP8) {
#pragma unroll
                            for (int i = 0; i < D / 16; ++i) {
                                uint32_t v[4];
                                ldsm4t(vbase + mrow[a] + sub_offset<G>(2 * i, substride) + v_row + (v_x ^ ((i * 32) & XMASK)),
                                       v);
                                if (tail) {
                                    v[0] &= keep[a][0];
                                    v[1] &= keep[a][0];
                                    v[2] &= keep[a][1];
                                    v[3] &= keep[a][1];
                                }
#pragma unroll
                                for (int c = 0; c < NT; ++c)
                                    mma<false>(acc[i][c], v[0], v[1], v[2], v[3], pf[a][c][0], pf[a][c][1]);
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < D / 16; i += 2) {
                                uint32_t v[4];
                                ldsm4t(vbase + mrow[a] + sub_offset<G>(i, substride) + v_row + (v_x ^ ((i * 16) & XMASK)), v);
#pragma unroll
                                for (int e = 0; e < 2; ++e) {
                                    uint32_t lo = v[2 * e], hi = v[2 * e + 1];
                                    if (tail) {
                                        lo &= keep[a][0];
                                        hi &= keep[a][1];
                                    }
                                    lo = __byte_perm(lo, 0, 0x3120);   // (key, key + 1) of channel 2g, then of 2g + 1
                                    hi = __byte_perm(hi, 0, 0x3120);
                                    uint32_t a0, a1, a2, a3;
                                    codes_f16(lo, a0, a1);
                                    codes_f16(hi, a2, a3);
#pragma unroll
                                    for (int c = 0; c < NT; ++c)
                                        mma<true>(acc[i + e][c], a0, a1, a2, a3, pf[a][c][0], pf[a][c][1]);
                                }
                            }
                        }
                    }
                } else {
                    // one token at a time: its rows' products over the values it sees, the others' dropped
                    for (int t = 0; t < n_new; ++t) {
                        const int see = (int)min(max(len.pos + t + 1, 0LL), len.keys) - key0;
#pragma unroll
                        for (int a = 0; a < MT; ++a) {
                            uint32_t cut[2];
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = a * 16 + e * 8 + 2 * j;
                                cut[e] = keep[a][e] & ((key < see ? 0xffffu : 0u) | (key + 1 < see ? 0xffff0000u : 0u));
                            }
#pragma unroll
                            for (int i = 0; i < D / 16; i += FP8 ? 2 : 1) {
                                uint32_t v[4];
                                ldsm4t(vbase + mrow[a] + sub_offset<G>(FP8 ? i : 2 * i, substride) + v_row +
                                           (v_x ^ ((FP8 ? i * 16 : i * 32) & XMASK)),
                                       v);
#pragma unroll
                                for (int e = 0; e < (FP8 ? 2 : 1); ++e) {
                                    uint32_t a0, a1, a2, a3;
                                    if (FP8) {
                                        const uint32_t lo = __byte_perm(v[2 * e] & cut[0], 0, 0x3120);
                                        const uint32_t hi = __byte_perm(v[2 * e + 1] & cut[1], 0, 0x3120);
                                        codes_f16(lo, a0, a1);
                                        codes_f16(hi, a2, a3);
                                    } else {
                                        a0 = v[0] & cut[0];
                                        a1 = v[1] & cut[0];
                                        a2 = v[2] & cut[1];
                                        a3 = v[3] & cut[1];
                                    }
#pragma unroll
                                    for (int c = 0; c < NT; ++c) {
                                        float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                                        mma<FP8>(d, a0, a1, a2, a3, pf[a][c][0], pf[a][c][1]);
#pragma unroll
                                        for (int x = 0; x < 4; ++x) {
                                            const int r = r0 + rg * NT * 8 + c * 8 + 2 * j + (x & 1);
                                            if (r / p.G == t) acc[i + e][c][x] += d[x];
                                        }
                                    }
                                }
                            }
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[st]);
            }
            if ((st += KL) >= NST) {
                st = kl;
                ph ^= 1;
            }
        }
        it += n;

        // join the lanes, in their order
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) l[c][x] += __shfl_xor_sync(0xffffffffu, l[c][x], o);
                if (lim[c][x] == 0) {   // (a token that is not there saw what the first one sees)
                    m[c][x] = -INFINITY;
                    l[c][x] = 0.0f;
                }
                if (g == 0) ml[kl * rows_pad + rg * NT * 8 + c * 8 + 2 * j + x] = make_float2(m[c][x], l[c][x]);
            }
        consumer_sync(threads);
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int r = rg * NT * 8 + c * 8 + 2 * j + x;
                float top = -INFINITY;
                for (int k = 0; k < KL; ++k) top = fmaxf(top, ml[k * rows_pad + r].x);
                // this lane's sums in units of 2^top
                const float f = m[c][x] == -INFINITY ? 0.0f : ex2(m[c][x] - top) * (FP8 ? ex2(mv[c][x] - m[c][x]) : 1.0f);
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    acc[i][c][x] *= f;
                    acc[i][c][2 + x] *= f;
                }
            }
        // each round, one lane writes or adds to each copy of the join buffer
        float *mine = obuf + (size_t)(kl % p.copies) * rows_pad * G::OSTR;
        for (int round = 0; round * p.copies < KL; ++round) {
            if (kl / p.copies == round) {
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int i = 0; i < D / 16; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int r = rg * NT * 8 + c * 8 + 2 * j + (e & 1);
                            const int d = i * 16 + (FP8 ? 2 * g + (e >> 1) : g + 8 * (e >> 1));
                            float *o = mine + r * G::OSTR + d;
                            *o = round == 0 ? acc[i][c][e] : *o + acc[i][c][e];
                        }
            }
            consumer_sync(threads);
        }
        // the unit's output, or this share's part of it
        const bool whole = ta == 0 && n == len.tiles;
        const int slot = 2 * blockIdx.x + (first ? 0 : 1);
        for (int i = tid; i < nrows * (D / 8); i += threads) {
            const int r = i / (D / 8), d0 = (i % (D / 8)) * 8;
            float top = -INFINITY, sum = 0.0f, o[8];
            for (int k = 0; k < KL; ++k) top = fmaxf(top, ml[k * rows_pad + r].x);
            for (int k = 0; k < KL; ++k) {
                const float2 v = ml[k * rows_pad + r];
                sum += v.x == -INFINITY ? 0.0f : v.y * ex2(v.x - top);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = obuf[r * G::OSTR + d0 + e];
            for (int k = 1; k < p.copies; ++k)
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] += obuf[(k * rows_pad + r) * G::OSTR + d0 + e];
            if (whole) {
                const int rr = r0 + r, t = rr / p.G, hq = h * p.G + rr % p.G;
                const long long bt = (long long)b * p.T + t;
                const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = sum == 0.0f ? 0.0f : o[e] * inv;
                if (p.gate.p != nullptr) {
                    float z[8];
                    unpack8(*reinterpret_cast<const uint4 *>(p.gate.p + bt * p.gate.ts + hq * p.gate.hs + d0), z);
#pragma unroll
                    for (int e = 0; e < 8; ++e) o[e] *= sigmoid(z[e]);
                }
                *reinterpret_cast<uint4 *>(p.out + (bt * p.Hq + hq) * D + d0) = pack8(o);
                if (d0 == 0 && p.lse != nullptr) p.lse[bt * p.Hq + hq] = (top + log2f(sum)) * kLn2;
            } else {
                float4 *dst = reinterpret_cast<float4 *>(p.part_o + ((size_t)slot * p.rows + r) * D + d0);
                dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                if (d0 == 0) p.part_ml[(size_t)slot * p.rows + r] = make_float2(top, sum);
            }
        }
        if (ta == 0 && !whole && tid == 0) {
            // the unit goes on: its last tile lies in the last share that starts at or before it
            const unsigned last = start + (it - n) + len.tiles - 1;
            p.meta[3 * blockIdx.x] = b * heads + ui;
            p.meta[3 * blockIdx.x + 1] = (int)sh.of(last);
            p.meta[3 * blockIdx.x + 2] = slot;
        }
        first = false;
        left -= n;
        ta = 0;
        if (left > 0 && ++ui == heads) {
            ui = 0;
            len = row_len<G>(p, ++b);
        }
    }
}

// Joins the partial results of the unit that starts in share blockIdx.x and
// goes on, if there is one: rows blockIdx.y, + gridDim.y ...  D/4 threads take
// four channels each of a group of parts; a chain of few loads: what the
// parts hold is asked for before their weights are known.
template <int D>
__global__ void __launch_bounds__(512) attn_join_kernel(const Params p) {
    constexpr int COLS = D / 4, GROUPS = 512 / COLS, UNROLL = 4;
    __shared__ float4 sums[GROUPS][COLS];
    __shared__ float red_m[GROUPS], red_l[GROUPS];
    grid_dep_launch();
    grid_dep_wait();
    const int c0 = blockIdx.x, unit = p.meta[3 * c0];
    if (unit < 0) return;
    // its first part lies in that share's slot, the others in the first slots of the shares that follow
    const int n = p.meta[3 * c0 + 1] - c0 + 1, first_slot = p.meta[3 * c0 + 2];
    const int heads = p.Hkv * p.RB, b = unit / heads, h = unit % heads / p.RB, r0 = (unit % heads % p.RB) * p.rows;
    const int nrows = min(p.rows, p.R - r0);
    const int tid = threadIdx.x, col = tid % COLS, grp = tid / COLS;
    for (int r = blockIdx.y; r < nrows; r += gridDim.y) {
        // this group's parts, with a running maximum
        float m = -INFINITY, l = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i0 = grp; i0 < n; i0 += GROUPS * UNROLL) {
            float2 v[UNROLL];
            float4 x[UNROLL];
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                const int i = i0 + k * GROUPS;
                const size_t slot = i == 0 ? first_slot : 2 * (c0 + i);
                v[k] = make_float2(-INFINITY, 0.0f);
                x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                if (i < n) {
                    v[k] = p.part_ml[slot * p.rows + r];
                    x[k] = *reinterpret_cast<const float4 *>(p.part_o + (slot * p.rows + r) * D + col * 4);
                }
            }
            float top = m;
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) top = fmaxf(top, v[k].x);
            const float f = m == -INFINITY ? 0.0f : ex2(m - top);
            o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
            l *= f;
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                if (v[k].x == -INFINITY) continue;   // (a part in which the row saw nothing)
                const float w = ex2(v[k].x - top);
                l = fmaf(w, v[k].y, l);
                o.x = fmaf(w, x[k].x, o.x);
                o.y = fmaf(w, x[k].y, o.y);
                o.z = fmaf(w, x[k].z, o.z);
                o.w = fmaf(w, x[k].w, o.w);
            }
            m = top;
        }
        __syncthreads();   // (the previous row's readers)
        sums[grp][col] = o;
        if (col == 0) {
            red_m[grp] = m;
            red_l[grp] = l;
        }
        __syncthreads();
        if (tid < D) {
            float top = -INFINITY, acc = 0.0f, total = 0.0f;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) top = fmaxf(top, red_m[i]);
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) {
                if (red_m[i] == -INFINITY) continue;
                const float w = ex2(red_m[i] - top);
                acc = fmaf(w, reinterpret_cast<const float *>(sums[i])[tid], acc);
                total = fmaf(w, red_l[i], total);
            }
            const int rr = r0 + r, t = rr / p.G, hq = h * p.G + rr % p.G;
            const long long bt = (long long)b * p.T + t;
            float y = total == 0.0f ? 0.0f : acc / total;
            if (p.gate.p != nullptr) y *= sigmoid(bf16_to_f32(p.gate.p[bt * p.gate.ts + hq * p.gate.hs + tid]));
            p.out[(bt * p.Hq + hq) * D + tid] = f32_to_bf16(y);
            if (tid == 0 && p.lse != nullptr) p.lse[bt * p.Hq + hq] = (top + log2f(total)) * kLn2;
        }
    }
}

// Row blocks of a (b, h) and the query rows of one.
void row_blocks(const AttnSizes &s, int *blocks, int *rows) {
    const int R = s.T * (s.Hq / s.Hkv);
    *blocks = (R + kMaxRows - 1) / kMaxRows;
    *rows = (R + *blocks - 1) / *blocks;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Workspace {
    size_t o, ml, meta, total;
};

Workspace workspace(const AttnSizes &s) {
    int blocks, rows;
    row_blocks(s, &blocks, &rows);
    const size_t slots = 2 * (size_t)num_sms();
    Workspace w;
    w.o = 0;
    w.ml = up256(slots * rows * s.D * sizeof(float));
    w.meta = w.ml + up256(slots * rows * sizeof(float2));
    w.total = w.meta + up256((size_t)num_sms() * 3 * sizeof(int));
    return w;
}

template <class G, int NT>
cudaError_t launch_t(Params &p, cudaStream_t st) {
    p.RG = (p.rows + NT * 8 - 1) / (NT * 8);
    p.KL = max_consumers<G, NT>() / p.RG;
    p.copies = 64 * 1024 / (p.RG * NT * 8 * G::OSTR * 4);
    p.copies = p.copies < 1 ? 1 : p.copies > 4 ? 4 : p.copies;
    if (p.copies > p.KL) p.copies = p.KL;
    int lg = 0;
    while ((1 << lg) < G::KT) ++lg;
    p.box_log2 = p.c.shift < lg ? p.c.shift : lg;
    // A stage always belongs to the same lane (stages a multiple of KL): fills may land out of order, and a lane
    // that waits for a stage's fill k by its parity must have seen fill k - 1 land itself, or the parity of a fill
    // k - 1 still on its way would read as fill k.
    p.stages = p.KL;
    while (p.stages + p.KL <= kMaxStages &&
           layout<G>(p.RG, NT, p.KL, p.copies, p.stages + p.KL).total <= kSmemLimit - 1024)
        p.stages += p.KL;
    if (layout<G>(p.RG, NT, p.KL, p.copies, p.stages).total > kSmemLimit - 1024) return cudaErrorInvalidConfiguration;
    const int smem = layout<G>(p.RG, NT, p.KL, p.copies, p.stages).total;
    static unsigned long long done = 0;
    cudaError_t e = set_max_smem(done, attn_decode_kernel<G, NT>, kSmemLimit - 1024);
    if (e != cudaSuccess) return e;

    CUtensorMap maps[2];
    const bool none = p.c.n_pages == 0;   // (no page: nothing is ever loaded, but a map needs a tensor)
    const uint64_t rows = none ? 1 : ((uint64_t)p.c.n_pages * p.Hkv) << p.c.shift;
    const uint64_t dims[3] = {(uint64_t)(G::FP8 ? G::SUBB : G::SUBB / 2), rows, (uint64_t)G::NSUB};
    const uint64_t strides[2] = {(uint64_t)G::ROWB, (uint64_t)G::SUBB};
    const uint32_t box[3] = {(uint32_t)dims[0], 1u << p.box_log2, (uint32_t)G::NSUB};
    for (int i = 0; i < 2; ++i) {
        const void *base = none ? p.q : i == 0 ? p.c.k : p.c.v;
        if (!encode_tmap_strided(&maps[i], base, G::FP8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                 3, dims, strides, box,
                                 G::SUBB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
            return cudaErrorInvalidValue;
    }
    // the tiles of a call are counted in 32 bits
    if ((unsigned long long)p.B * p.Hkv * p.RB * (((unsigned long long)p.c.width << p.c.shift) / G::KT + 1) > 0x7fffffffULL)
        return cudaErrorNotSupported;
    const int ctas = num_sms();
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3((p.RG * p.KL + 1) * 32);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, attn_decode_kernel<G, NT>, maps[0], maps[1], p);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(ctas, p.rows < 8 ? p.rows : 8);
    cfg.blockDim = dim3(512);
    cfg.dynamicSmemBytes = 0;
    return cudaLaunchKernelEx(&cfg, attn_join_kernel<G::D>, p);
}

template <int D>
cudaError_t launch_d(Params &p, cudaStream_t st) {
    const bool one = p.rows <= 8;
    if (p.c.fp8) return one ? launch_t<Geo<D, true>, 1>(p, st) : launch_t<Geo<D, true>, 2>(p, st);
    return one ? launch_t<Geo<D, false>, 1>(p, st) : launch_t<Geo<D, false>, 2>(p, st);
}

}  // namespace

size_t attn_decode_workspace(const AttnSizes &s) { return workspace(s).total; }

cudaError_t launch_attn_decode(const AttnSizes &s, const uint16_t *q, const PagedCache &c, const int32_t *pos,
                               const int32_t *n_new, const HeadsIn &gate, float scale, uint16_t *out, float *lse,
                               void *ws, unsigned *err, cudaStream_t st) {
    Params p = {};
    p.q = q;
    p.c = c;
    p.pos = pos;
    p.n_new = n_new;
    p.gate = gate;
    p.out = out;
    p.lse = lse;
    p.err = err;
    p.B = s.B;
    p.T = s.T;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.G = s.Hq / s.Hkv;
    p.R = s.T * p.G;
    row_blocks(s, &p.RB, &p.rows);
    p.scale2 = scale * kLog2e;
    const Workspace w = workspace(s);
    char *base = static_cast<char *>(ws);
    p.part_o = reinterpret_cast<float *>(base + w.o);
    p.part_ml = reinterpret_cast<float2 *>(base + w.ml);
    p.meta = reinterpret_cast<int *>(base + w.meta);
    if (s.D == 64) return launch_d<64>(p, st);
    if (s.D == 128) return launch_d<128>(p, st);
    return launch_d<256>(p, st);
}

}  // namespace gdn
