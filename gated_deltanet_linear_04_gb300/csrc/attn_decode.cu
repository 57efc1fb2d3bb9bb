// Attention of 1..8 new tokens per row over the paged cache.
//
// Per query row: s_j = scale q.k_j over the visible positions, out =
// sum_j 2^(s'_j - m) v_j / sum_j 2^(s'_j - m) with s' = s log2(e) and m a
// running maximum: one pass over the keys and values, HBM-bound (16 flop per
// byte for 8 query heads per key head, bf16).
//
// Work.  A unit is one (row b, key head h, block of at most 32 of its T * Hq/Hkv
// query rows); its keys come in tiles of KT (32 KB of keys, 32 KB of values).
// The tiles of all units form one list (with blank slots before each unit's first
// tile, for what its start and end cost), cut into equal shares for one CTA per
// SM (two, with half the tile, for short tables), so ragged batches and a single
// long row both fill the GPU; each CTA finds its share from pos / n_new itself.
// A unit that crosses shares leaves partial results (m, sum, weighted sum) in the
// workspace, and a second kernel joins them in share order.
//
// CTA.  Producer warps keep two rings (keys, values) filled with TMA box loads
// (a box: the tokens of one page, or KT of them, 128-byte swizzled; a page
// that does not exist is skipped and marked).  Eight consumer warps go through
// a tile together: each takes 16 or 32 keys for S^T = K Q^T; each then takes
// every eighth query row for the softmax; each then takes 1/8 of the channels
// for O^T += V^T P^T.  S and P pass through shared memory, two barriers a tile.
// So a warp's accumulators are small (16 to 32 channels of all rows), nothing
// has to be joined at the end of a unit, and a tile is held only for the
// microsecond that it takes all warps together, while the next two are on
// their way.  (Warps that take whole tiles on their own, with all channels and
// a join at the end of each unit, held each tile three times as long and lost
// 5 us at each unit's end: 69 against 61 us for B = 128, e4m3, 2048 keys.)
// What it came to (16 query and 2 key heads of 256 channels; calls in a host loop
// over fresh inputs): one row of 262144 keys in bf16 86.5 us, 6.2 TB/s of keys and
// values; B = 128, up to 4096 keys in e4m3 51.0 us, 5.3 TB/s; B = 32, windows of 4
// tokens, 32 and 8 heads of 128 channels, bf16 56.7 us, 5.3 TB/s.  (With every key in
// the L2 cache the last two take 41 and 47 us.)  In between, a tile takes the consumers
// about 3100 clocks (with e4m3 its conversions alone take 770 of them), the memory 2990;
// the first data come after 5 us, and a unit's end and the next one's start cost 4000
// clocks more than a tile.
//
// Products.  mma.sync m16n8k16 with keys (then channels) as the 16 and query rows
// as the 8, which eight heads per key head fill exactly.  With up to 8 rows the
// products are far from the bound, and tcgen05 (128 keys by the rows, as full as
// these) would only add the way through tensor memory in front of the softmax.  With
// 32 and more rows they are the bound (B = 32, up to 4095 keys, 16 and 2 heads of 256,
// bf16: 8, 32 and 64 rows 31, 50 and 79 us): there these products are what holds the
// kernel back.  e4m3 codes are turned into f16 pairs on the way from shared memory to
// the operand (exactly); their scales go to the scores (keys) and into the exponent of
// the weights (values).
//
// Weights are rounded to the 16 bits of the operand beside them: f16 with e4m3 values,
// bf16 with bf16 values.  bf16 weights leave the output 0.0020 from the 64-bit result
// (2-norm) where its own rounding alone is 0.0017.  A high and a low bf16 part of each
// gives 0.0017 for twice the products: one row of 262144 keys 86.5 -> 86.7 us, windows
// of 16 rows 56.7 -> 58.7, 32 rows 49.7 -> 53.1, 64 rows of 128 channels 76 -> 87; one
// part was kept.
#include "attn.cuh"

namespace gdn {
namespace {

using namespace attn;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxStages = 4;
constexpr int kRowCache = 192;     // rows whose lengths a CTA keeps
// f16 softmax weights (e4m3 caches) are 2^14 at the largest: f16 ends at 2^16, and below 2^-14 it loses bits.  So a
// weight is whole down to 2^-28 of the largest and lost only below 2^-39; with 1 as the largest, 2^-14 and 2^-25, a few
// hundred thousand keys 17 nats below another lost a third of their share of the output.
constexpr float kWeightBits = 14.0f, kWeightUnit = 1.0f / 16384;
constexpr int kBlank = 2;         // blank slots of a unit in the list of tiles (B = 128, ragged, e4m3: 1, 2, 3 of
                                  // them 56.2, 53.6, 53.7 us)
constexpr int kSmemSM = 228 * 1024;   // shared memory of an SM
constexpr int kMaxCtas = 2;       // CTAs on an SM

// The geometry of a tile: eight consumer warps and 32 KB of keys, or (SMALL) two CTAs on an SM with half of both.
template <int D_, bool FP8_, bool SMALL_>
struct Geo {
    static constexpr int D = D_, W = SMALL_ ? 4 : 8, THREADS = W * 32, CTAS = SMALL_ ? 2 : 1;
    static constexpr int SMEM = kSmemSM / CTAS - 3072;         // (1 KB of a CTA is the system's; static shared memory)
    static constexpr bool FP8 = FP8_;
    static constexpr int ROWB = FP8 ? D : 2 * D;               // bytes of a key
    static constexpr int SUBB = ROWB < 128 ? ROWB : 128;       // ... in sub-tiles of one swizzle span
    static constexpr int NSUB = ROWB / SUBB;
    static constexpr int KT = 32768 / CTAS / ROWB > 256 ? 256 : 32768 / CTAS / ROWB;   // keys of a tile: 64, 128 or 256
    static constexpr int TILE = KT * ROWB;                     // bytes of a tile's keys, or values
    static constexpr int KB = KT / 16, DB = D / 16;            // blocks of 16 keys, of 16 channels
    static constexpr int SPLIT = W > KB ? W / KB : 1;          // S: warps that share 16 keys, part of the channels each
    static constexpr int MPW = KB > W ? KB / W : 1;            // ... or blocks of 16 keys of a warp
    static constexpr int KS = DB / SPLIT;                      // ... channel blocks of a warp
    // O: channel blocks of a warp (e4m3: pairs, which is what one ldmatrix brings), and warps that share them, part of
    // the keys each
    static constexpr int DPW = DB > W ? DB / W : FP8 ? 2 : 1;
    static constexpr int KSPL = W * DPW / DB;
    static constexpr int KK = KB / KSPL;                       // ... key blocks of a warp
    static constexpr int SSTR = KT + 4;                        // row stride of S (floats): banks 8 apart for rows 2 apart
    static constexpr int PSTR = KT + 8;                        // row stride of P (16-bit): banks 4 apart
    static constexpr int PRODUCERS = FP8 && !SMALL_ ? 4 : 2;   // warps: keys, values, key scales, value scales (or the first: all scales)
    static_assert(KS >= (FP8 ? 2 : 1) && KK >= 2 && KK % 2 == 0, "");
};

struct Params {
    const uint16_t *q;
    PagedCache c;
    const int32_t *pos, *n_new;
    HeadsIn gate;
    uint16_t *out;
    float *lse;
    float *part_o;      // [2 * ctas][rows][D]
    float2 *part_ml;    // [2 * ctas][rows]: m and the sum, which is -1 where the row saw no key of the part
    int *meta;          // [ctas][3]: the unit that starts in the share and goes on (or -1), its last share, its slot
    unsigned *err;
    int B, T, Hq, Hkv, G, R;
    int RB, rows;       // row blocks of a (b, h), query rows of one
    int g_mul;          // r / G = r * g_mul >> 16 for the r < 128 there are
    int box_log2;
    float scale2;       // scale * log2(e)
};

// Dynamic shared memory: the rings, then
template <class G, int NT>
struct Smem {
    static constexpr int rows = NT * 8;
    static constexpr int q_bytes = rows * G::D * 2;
    // S, and in its place at a unit's end the parts of O that went over other keys
    static constexpr int s_only = G::SPLIT * rows * G::SSTR * 4, o_parts = (G::KSPL - 1) * rows * G::D * 4;
    static constexpr int s_bytes = s_only > o_parts ? s_only : o_parts;
    static constexpr int p_bytes = rows * G::PSTR * 2;
    static constexpr int row_bytes = rows * 16;                // corr, qscale, fin
    static constexpr int sc_bytes = G::FP8 ? 2 * G::KT : 0;    // a stage's scales
    static constexpr int fixed = q_bytes + s_bytes + p_bytes + row_bytes;
    static constexpr int pair = 2 * G::TILE + sc_bytes;        // a stage of both rings
    static constexpr int fit = (G::SMEM - 1024 - fixed) / pair;
    static constexpr int stages = fit > kMaxStages ? kMaxStages : fit;
    static constexpr int q = stages * 2 * G::TILE, s = q + q_bytes, p = s + s_bytes, row = p + p_bytes,
                         sc = row + row_bytes, total = sc + stages * sc_bytes;
    static_assert(stages >= 2, "");
};

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

// sigmoid(x), a factor of an f32 that is rounded to bf16 next: the hardware's
// exponential and reciprocal are off by about 2^-21 (2^-17 at |x| = 80).
__device__ __forceinline__ float gate_value(float x) { return rcp_fast(1.0f + exp_fast(-x)); }

// The warp's largest value; a NaN is passed over.
__device__ __forceinline__ float warp_max(float x) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
    return r;
}

// The values of two e8m0 bytes.
__device__ __forceinline__ float2 e8m0_pair(uint32_t bytes) {
    uint32_t b;
    asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(b) : "h"((uint16_t)bytes));
    return make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
}

// L2 policy of keys and values, which a call reads once (rows that share pages, at
// about the same time): they go before what else the cache holds.  In calls one after
// the other the ragged batch took 50.2 instead of 53.0 us, windows 56.0 instead of
// 58.7; after a flush of the cache there is no difference, nor with shared pages.
__device__ __forceinline__ uint64_t read_once() {
    uint64_t policy;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
    return policy;
}

// A box of a page's keys or values: row `row` on, all channels.
__device__ __forceinline__ void load_box(void *dst, const CUtensorMap *map, int row, uint64_t *bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
        "[%1, {%2, %3, %2}], [%4], %5;" ::"r"(smem_u32(dst)),
        "l"(map), "r"(0), "r"(row), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
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

// The keys of row b (the new tokens' own included) and its tiles; a row
// without keys still has one, empty, tile, so that its outputs get written.
struct RowLen {
    long long pos, keys;
    int n, tiles;
    bool short_table;   // some of its positions have no page
};

template <class G>
__device__ __forceinline__ RowLen row_len(const Params &p, int pos, int n) {
    RowLen r;
    r.n = n;
    r.pos = pos;
    const long long want = r.n == 0 ? 0 : max(r.pos + r.n, 0LL);
    r.keys = min(min(want, (long long)p.c.width << p.c.shift), 0x7fffff00LL);   // (key indexes are 32 bits)
    r.short_table = r.n > 0 && (r.keys < want || r.pos < 0);
    r.tiles = (int)max((r.keys + G::KT - 1) / G::KT, 1LL);
    return r;
}

template <class G>
__device__ __forceinline__ RowLen row_len(const Params &p, int b) {
    return row_len<G>(p, p.pos[b], clamp_new(p.n_new, b, p.T));
}

// The list of all units' slots in `act` shares that differ by at most one slot,
// the longer ones first.
struct Shares {
    unsigned act, base, extra;   // base or base + 1 slots; `extra` shares have one more

    __device__ void set(unsigned total, unsigned ctas) {
        act = min(ctas, total);
        base = total / act;
        extra = total - base * act;
    }
    __device__ unsigned start(unsigned c) const { return c * base + min(c, extra); }
    // the share that holds a slot
    __device__ unsigned of(unsigned slot) const {
        const unsigned cut = extra * (base + 1);
        return slot < cut ? slot / (base + 1) : extra + (slot - cut) / base;
    }
};

// A stretch of one unit's tiles in a share.
struct Seg {
    int b, h, r0, ta, n;      // row, key head, first query row; tiles [ta, ta + n)
    RowLen len;
    unsigned first_slot;      // of the unit's first tile, in the list
    __device__ bool whole() const { return ta == 0 && n == len.tiles; }
};

// Goes through a share's stretches.
template <class G>
struct Walk {
    int b, ui, so, left;      // row; unit of it; slot of the unit; slots left of the share
    unsigned slot;
    RowLen len;
    // (pos, n) of the rows from `row0` on: with the memory's queues full a load takes microseconds
    const int2 *rows;
    int row0;

    __device__ bool next(const Params &p, Seg &s) {
        while (left > 0) {
            const int all = len.tiles + kBlank, take = min(all - so, left);
            s.b = b;
            s.h = p.RB == 1 ? ui : ui / p.RB;
            s.r0 = p.RB == 1 ? 0 : (ui - s.h * p.RB) * p.rows;
            s.ta = max(so - kBlank, 0);
            s.n = so + take - kBlank - s.ta;
            s.len = len;
            s.first_slot = slot - so + kBlank;
            left -= take;
            slot += take;
            so = 0;
            if (left > 0 && ++ui == p.Hkv * p.RB) {
                ui = 0;
                const int i = ++b - row0;
                len = i < kRowCache ? row_len<G>(p, rows[i].x, rows[i].y) : row_len<G>(p, b);
            }
            if (s.n > 0) return true;
        }
        return false;
    }
};

template <int THREADS>
__device__ __forceinline__ void consumer_sync() {
    asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

template <class G, int NT>
__global__ void __launch_bounds__((G::W + G::PRODUCERS) * 32, G::CTAS)
    attn_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const Params p) {
    using L = Smem<G, NT>;
    constexpr int D = G::D, KT = G::KT, W = G::W, NST = L::stages;
    constexpr bool FP8 = G::FP8;
    constexpr bool QREG = NT <= 2;           // query operands in registers; else read from shared memory each time
    extern __shared__ __align__(1024) unsigned char smem[];
    __shared__ __align__(8) uint64_t full_k[NST], full_v[NST], empty_k[NST], empty_v[NST];
    __shared__ uint32_t bad_boxes[NST], nan_tile;
    __shared__ unsigned warp_sum_sh[G::W + 4], found_off;
    __shared__ int found_b;
    __shared__ int2 row_cache[kRowCache];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (tid == 0) {
        nan_tile = 0;
#pragma unroll
        for (int i = 0; i < NST; ++i) {
            mbar_init(&full_k[i], G::PRODUCERS == 4 ? 3 : 1);
            mbar_init(&full_v[i], 1);
            mbar_init(&empty_k[i], W);
            mbar_init(&empty_v[i], W);
        }
        fence_mbar_init();
        prefetch_tmap(&tm_k);
        prefetch_tmap(&tm_v);
    }
    grid_dep_enter();

    // the share: prefix sums of the rows' tiles, blockDim rows at a time (twice, if that is not all of them)
    const int heads = p.Hkv * p.RB;
    constexpr int nthr = (W + G::PRODUCERS) * 32, nwarp = nthr / 32;
    const bool once = p.B <= nthr, keep = p.B <= kRowCache && once;   // (keep: all rows' lengths, as they come in)
    Shares sh;
    unsigned start = 0;
    for (int pass = 0; pass < 2; ++pass) {
        unsigned run = 0;
        for (int base = 0; base < p.B; base += nthr) {
            const int b = base + tid;
            unsigned v = 0;
            if (b < p.B) {
                const int pos = p.pos[b], n = clamp_new(p.n_new, b, p.T);
                if (keep) row_cache[b] = make_int2(pos, n);
                v = (unsigned)((row_len<G>(p, pos, n).tiles + kBlank) * heads);
            }
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
#pragma unroll
            for (int w = 0; w < nwarp; ++w) {
                if (w < warp) before += warp_sum_sh[w];
                all += warp_sum_sh[w];
            }
            run += all;
            if (once) {
                sh.set(all, gridDim.x);
                start = sh.start(blockIdx.x);
            }
            if ((pass == 1 || once) && b < p.B && before + x - v <= start && start < before + x) {
                found_b = b;
                found_off = start - (before + x - v);
            }
        }
        if (once) break;
        if (pass == 0) {
            sh.set(run, gridDim.x);
            start = sh.start(blockIdx.x);
        }
    }
    __syncthreads();
    if (tid == 0) p.meta[3 * blockIdx.x] = -1;
    if (blockIdx.x >= sh.act) return;
    Walk<G> walk;
    walk.b = found_b;
    walk.rows = row_cache;
    walk.row0 = keep ? 0 : found_b;
    if (!keep) {
        if (tid < kRowCache && found_b + tid < p.B)
            row_cache[tid] = make_int2(p.pos[found_b + tid], clamp_new(p.n_new, found_b + tid, p.T));
        __syncthreads();
    }
    {
        const int2 row = row_cache[found_b - walk.row0];
        walk.len = row_len<G>(p, row.x, row.y);
    }
    walk.slot = start;
    walk.left = (int)(sh.start(blockIdx.x + 1) - start);
    {
        const unsigned all = walk.len.tiles + kBlank;
        walk.ui = (int)(found_off / all);
        walk.so = (int)(found_off - walk.ui * all);
    }
    Seg seg;
    const int boxrows = 1 << p.box_log2;
    bool dead = false;
    int st = 0;           // the tile's stage, and the parity of its fill
    uint32_t ph = 0;

    if (warp >= W) {
        // ---- producers: lane i < bpt fills box i of every tile -------------------------------------------
        const int role = warp - W;                  // keys, values, key scales, value scales
        const int bpt = KT >> p.box_log2, page_sh = p.c.shift - p.box_log2;   // boxes per tile; pages = boxes >> page_sh
        constexpr bool all_scales = FP8 && G::PRODUCERS == 2;
        const uint32_t bytes = role < 2 ? (uint32_t)boxrows * G::ROWB : (uint32_t)boxrows;
        const uint32_t box_bytes = bytes + (all_scales && role == 0 ? 2 * boxrows : 0);
        uint64_t *full = role == 1 ? full_v : full_k, *empty = role == 1 ? empty_v : empty_k;
        unsigned char *ring = role < 2 ? smem + (role == 0 ? 0 : G::TILE) : smem + L::sc + (role - 2) * KT;
        const int pitch = role < 2 ? 2 * G::TILE : 2 * KT;
        const uint8_t *scales = role == 2 ? p.c.ks : p.c.vs;
        const uint64_t policy = read_once();
        uint32_t used = 0;
        // page numbers, asked for two tiles ahead, those of a unit's first two during the unit before
        auto boxes = [&](const Seg &u) { return (int)((u.len.keys + boxrows - 1) >> p.box_log2); };
        auto ask = [&](const Seg &u, int i) {
            const int box = (u.ta + i) * bpt + lane;
            return lane < bpt && i < u.n && box < boxes(u) ? p.c.table[(long long)u.b * p.c.width + (box >> page_sh)] : -1;
        };
        Seg ahead;
        bool have = walk.next(p, ahead);
        int next0 = have ? ask(ahead, 0) : -1, next1 = have ? ask(ahead, 1) : -1;
        while (have) {
            seg = ahead;
            const int n = seg.n, h = seg.h, nbox = boxes(seg);
            if (seg.len.short_table && role == 0 && lane == 0) atomicOr(p.err, kErrBadPage);
            int box = seg.ta * bpt + lane, id = next0, id1 = next1;
            have = walk.next(p, ahead);
            if (have) {
                next0 = ask(ahead, 0);
                next1 = ask(ahead, 1);
            }
            for (int i = 0; i < n; ++i) {
                const int id2 = ask(seg, i + 2);
                const bool want = lane < bpt && box < nbox, ok = want && id >= 0 && id < p.c.n_pages;
                if (want && !ok && role == 0) atomicOr(p.err, kErrBadPage);
                const uint32_t good = __ballot_sync(0xffffffffu, ok);
                if (!dead && !mbar_wait(&empty[st], ph ^ 1, p.err)) dead = true;
                dead = __any_sync(0xffffffffu, dead);
                if (!dead) {
                    if (lane == 0) {
                        if (role == 0) bad_boxes[st] = ~good & (bpt == 32 ? 0xffffffffu : (1u << bpt) - 1);
                        if (good != 0)
                            mbar_expect_tx(&full[st], __popc(good) * box_bytes);
                        else
                            mbar_arrive(&full[st]);
                    }
                    __syncwarp();
                    if (ok) {
                        const int row = ((id * p.Hkv + h) << p.c.shift) + ((box << p.box_log2) & (p.c.page - 1));
                        unsigned char *dst = ring + st * pitch + lane * bytes;
                        if (role < 2)
                            load_box(dst, role == 0 ? &tm_k : &tm_v, row, &full[st], policy);
                        else
                            bulk_load(dst, scales + row, bytes, &full[st]);
                        if (all_scales && role == 0) {
                            unsigned char *sc = smem + L::sc + st * 2 * KT + lane * boxrows;
                            bulk_load(sc, p.c.ks + row, boxrows, &full[st]);
                            bulk_load(sc + KT, p.c.vs + row, boxrows, &full[st]);
                        }
                    }
                    used |= 1u << st;
                    if (++st == NST) {
                        st = 0;
                        ph ^= 1;
                    }
                }
                box += bpt;
                id = id1;
                id1 = id2;
            }
        }
        // let the copies in flight land before the CTA ends (they have, but after a wait that gave up)
        for (int i = 0; i < NST; ++i) {
            if ((used >> i & 1) == 0) continue;
            const uint32_t phase = i < st ? ph : ph ^ 1;   // the parity of stage i's last fill
            for (uint32_t k = 0; k < kSpinLimit && !mbar_try_wait(&full[i], phase); ++k) {
            }
        }
        return;
    }

    // ---- consumers -----------------------------------------------------------
    const int g = lane >> 2, j = lane & 3;
    uint2 *qf = reinterpret_cast<uint2 *>(smem + L::q);            // [D/16][NT][32]
    float *sS = reinterpret_cast<float *>(smem + L::s);            // [SPLIT][rows][SSTR]
    uint16_t *sP = reinterpret_cast<uint16_t *>(smem + L::p);      // [rows][PSTR]
    float *corr = reinterpret_cast<float *>(smem + L::row), *qscale = corr + L::rows;
    float2 *fin = reinterpret_cast<float2 *>(qscale + L::rows);
    const uint32_t ring = smem_u32(smem);
    // ldmatrix rows and 16-byte chunks of this lane: matrix mi holds rows (mi & 1) * 8 .. and chunk + (mi >> 1)
    // (keys; e4m3 values), or rows (mi >> 1) * 8 .. and chunk + (mi & 1) (bf16 values)
    const int mi = lane >> 3, mr = lane & 7;
    const uint32_t swz = G::SUBB == 128 ? mr : mr >> 1;
    const uint32_t k_row = ((mi & 1) * 8 + mr) * G::SUBB, k_x = ((mi >> 1) ^ swz) << 4;
    const uint32_t v_row = FP8 ? k_row : (uint32_t)((mi >> 1) * 8 + mr) * G::SUBB;
    const uint32_t v_x = FP8 ? k_x : (uint32_t)((mi & 1) ^ swz) << 4;
    const uint32_t substride = boxrows * G::SUBB;
    // the byte offset of 16-byte chunk `c` (even: a pair of chunks) of the rows at `row`, of this lane
    auto at = [&](uint32_t row, uint32_t x, int c) {
        return (uint32_t)(c / (G::SUBB / 16)) * substride + row + (x ^ ((c * 16) & (G::SUBB - 16)));
    };
    // ... and of key k0 (a multiple of 16) of a tile: a box's sub-tiles follow each other
    const uint32_t box_gap = (uint32_t)boxrows * (G::ROWB - G::SUBB);
    auto key_base = [&](int k0) {
        return (uint32_t)k0 * G::SUBB + (G::NSUB > 1 ? (uint32_t)(k0 >> p.box_log2) * box_gap : 0u);
    };
    // this warp's part of S: keys and channels
    const int s_key = G::SPLIT > 1 ? warp / G::SPLIT * 16 : warp * 16 * G::MPW;
    const int s_part = G::SPLIT > 1 ? warp % G::SPLIT : 0;
    // ... of O: its channel block and key blocks
    constexpr int OW = G::DB / G::DPW;
    const int o_blk = warp % OW * G::DPW, o_part = warp / OW;
    // ldmatrix offsets: of the key operands, one per load; of the value operands
    constexpr int KL = G::KS / (FP8 ? 2 : 1), VL = G::DPW / (FP8 ? 2 : 1);
    uint32_t koff[KL], voff[VL], kkey[G::MPW];
#pragma unroll
    for (int i = 0; i < KL; ++i) koff[i] = at(k_row, k_x, 2 * (s_part * KL + i));
#pragma unroll
    for (int i = 0; i < VL; ++i) voff[i] = at(v_row, v_x, 2 * (o_blk / (FP8 ? 2 : 1) + i));
#pragma unroll
    for (int i = 0; i < G::MPW; ++i) kkey[i] = key_base(s_key + i * 16);
    // ... and of the softmax: rows warp, warp + W, ...; keys 2 lane, 2 lane + 1 of every 64
    constexpr int RPW = (L::rows + W - 1) / W;

    int stv = 0;                      // the stage of the tile's values (st: of the next tile's keys), and their parity
    uint32_t phv = 0;
    bool first = true;
    uint32_t tile_no = 0;
    // 8 channels of a query row per thread, asked for a unit ahead (where the registers allow it)
    constexpr bool EARLY = NT <= 2;
    constexpr int QV = (L::rows * (D / 8) + G::THREADS - 1) / G::THREADS;
    uint4 qraw[QV];
    auto ask_queries = [&](const Seg &u) {
        const int nrows = min(p.rows, p.R - u.r0);
#pragma unroll
        for (int x = 0; x < QV; ++x) {
            const int i = x * G::THREADS + tid, r = i / (D / 8), d0 = (i % (D / 8)) * 8;
            qraw[x] = make_uint4(0, 0, 0, 0);
            if (r < nrows) {
                const int rr = u.r0 + r, t = rr * p.g_mul >> 16, hq = u.h * p.G + rr - t * p.G;
                qraw[x] = *reinterpret_cast<const uint4 *>(p.q + (((long long)u.b * p.T + t) * p.Hq + hq) * D + d0);
            }
        }
    };
    Seg ahead;
    bool have = walk.next(p, ahead);
    if (EARLY && have) ask_queries(ahead);
    while (have) {
        seg = ahead;
        if (!EARLY) ask_queries(seg);
        const int b = seg.b, h = seg.h, r0 = seg.r0, ta = seg.ta, n = seg.n;
        const RowLen &len = seg.len;
        const int nrows = min(p.rows, p.R - r0);

        // queries to operand order
#pragma unroll
        for (int x8 = 0; x8 < QV; ++x8) {
            const int i = x8 * G::THREADS + tid, r = i / (D / 8), d0 = (i % (D / 8)) * 8;
            if (QV * G::THREADS != L::rows * (D / 8) && r >= L::rows) continue;
            const uint4 raw = qraw[x8];
            uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
            if (FP8) {
                // a power of two per row brings the largest query to [1, 4): f16 then holds every bit but those
                // below 2^-24 of it
                float x[8];
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
            const int ks = d0 >> 4, hi = (d0 >> 3) & 1;
            uint32_t *base = reinterpret_cast<uint32_t *>(qf + (ks * NT + (r >> 3)) * 32 + (r & 7) * 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                // bf16: k = 2e (+8 hi) of the 16; e4m3: channels 4j .. 4j+3 are k = 2j, 2j+1, 2j+8, 2j+9
                const int ln = FP8 ? hi * 2 + (e >> 1) : e, reg = FP8 ? e & 1 : hi;
                base[ln * 2 + reg] = w[e];
            }
        }
        have = walk.next(p, ahead);
        if (EARLY && have) ask_queries(ahead);
        consumer_sync<G::THREADS>();
        uint2 qr[QREG ? G::KS : 1][QREG ? NT : 1];
        if (QREG) {
#pragma unroll
            for (int ks = 0; ks < G::KS; ++ks)
#pragma unroll
                for (int c = 0; c < NT; ++c) qr[ks][c] = qf[((s_part * G::KS + ks) * NT + c) * 32 + lane];
        }
        // softmax state of this warp's rows
        float m[RPW], l[RPW], dv[RPW], rs[RPW];   // dv: largest (score + value exponent), less m
        int lim[RPW];                 // visible keys, 0 for a row that is not there
        uint32_t seen = 0;            // bit c: this lane saw a key of row c
#pragma unroll
        for (int c = 0; c < RPW; ++c) {
            m[c] = dv[c] = -INFINITY;
            l[c] = 0.0f;
            const int r = c * W + warp, t = (r0 + r) * p.g_mul >> 16;
            lim[c] = r < nrows && t < len.n ? (int)min(max(len.pos + t + 1, 0LL), len.keys) : 0;
            rs[c] = p.scale2 * (FP8 && r < nrows ? qscale[r] : 1.0f);
        }
        float acc[G::DPW][NT][4];
#pragma unroll
        for (int i = 0; i < G::DPW; ++i)
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][c][e] = 0.0f;
        // the gates of this thread's outputs, asked for before they are needed
        const bool gated = p.gate.p != nullptr && seg.whole() && o_part == 0;
        uint32_t gates[EARLY ? G::DPW : 1][EARLY ? NT : 1][2];
        auto gate_pair = [&](int r, int d) {
            // channels as the outputs below; two bf16 in one word
            const int rr = r0 + r, t = rr * p.g_mul >> 16, hq = h * p.G + rr - t * p.G, dt = (o_blk + d) * 16;
            const uint16_t *z = p.gate.p + ((long long)b * p.T + t) * p.gate.ts + hq * p.gate.hs + dt;
            if (FP8) return *reinterpret_cast<const uint32_t *>(z + 2 * g);
            return (uint32_t)z[g] | (uint32_t)z[g + 8] << 16;
        };
        if (EARLY && gated) {
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
#pragma unroll
                    for (int d = 0; d < G::DPW; ++d) {
                        const int r = c * 8 + 2 * j + x;
                        gates[EARLY ? d : 0][EARLY ? c : 0][x] = r < nrows ? gate_pair(r, d) : 0u;
                    }
        }
        const int all_see = (int)min(max(len.pos + 1, 0LL), len.keys);   // keys that every live row sees

        // S^T = K Q^T of the tile in stage st, into registers ...
        float s[G::MPW][NT][4];
        uint32_t bad_next = 0;
        auto wait_keys = [&] {
            if (!dead && !mbar_wait(&full_k[st], ph, p.err)) dead = true;
            dead = __any_sync(0xffffffffu, dead);
        };
        auto see_keys = [&] {
            bad_next = *static_cast<volatile uint32_t *>(&bad_boxes[st]);
        };
        auto scores = [&] {
            constexpr int CH = NT <= 2 && KL > 1 ? 2 : 1;   // chains of products that do not wait for each other
            const uint32_t kbase = ring + st * 2 * G::TILE;
#pragma unroll
            for (int a = 0; a < G::MPW; ++a) {
                const uint32_t base = kbase + kkey[a];
                float t[CH][NT][4];
#pragma unroll
                for (int x = 0; x < CH; ++x)
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) t[x][c][e] = 0.0f;
#pragma unroll
                for (int ks = 0; ks < G::KS; ks += FP8 ? 2 : 1) {
                    uint32_t k[4];
                    ldsm4(base + koff[ks / (FP8 ? 2 : 1)], k);
#pragma unroll
                    for (int e = 0; e < (FP8 ? 2 : 1); ++e) {
                        uint32_t a0 = k[0], a1 = k[1], a2 = k[2], a3 = k[3];
                        if (FP8) {
                            codes_f16(k[2 * e], a0, a2);
                            codes_f16(k[2 * e + 1], a1, a3);
                        }
#pragma unroll
                        for (int c = 0; c < NT; ++c) {
                            const uint2 q = QREG ? qr[QREG ? ks + e : 0][QREG ? c : 0]
                                                 : qf[((s_part * G::KS + ks + e) * NT + c) * 32 + lane];
                            mma<FP8>(t[(ks + e) % CH][c], a0, a1, a2, a3, q.x, q.y);
                        }
                    }
                }
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s[a][c][e] = CH == 2 ? t[0][c][e] + t[CH - 1][c][e] : t[0][c][e];
            }
        };
        // ... and from there to shared memory, the keys' stage given back (with e4m3, after the softmax: its scales)
        auto put_scores = [&] {
            if (dead) return;
#pragma unroll
            for (int a = 0; a < G::MPW; ++a)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sS[(s_part * L::rows + c * 8 + 2 * j + (e & 1)) * G::SSTR + s_key + a * 16 + g + 8 * (e >> 1)] =
                            s[a][c][e];
            if (!FP8) {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty_k[st]);
            }
        };
        wait_keys();
        see_keys();
        if (!dead) scores();
        put_scores();

        for (int i = 0; i < n; ++i) {
            const int key0 = (ta + i) * KT;
            const uint32_t bad = bad_next;
            const bool tail = bad != 0 || key0 + KT > all_see;
            if (!tail) seen = ~0u;
            ++tile_no;
            consumer_sync<G::THREADS>();

            // softmax: weights of this warp's rows
#pragma unroll
            for (int c = 0; c < RPW; ++c) {
                const int r = c * W + warp;
                if (r >= nrows) continue;
                float z[KT / 64][2], ve[KT / 64][2];
                float top = -INFINITY;
#pragma unroll
                for (int x = 0; x < KT / 64; ++x) {
                    const int key = x * 64 + 2 * lane;
                    float2 v = *reinterpret_cast<const float2 *>(sS + r * G::SSTR + key);
#pragma unroll
                    for (int y = 1; y < G::SPLIT; ++y) {
                        const float2 u = *reinterpret_cast<const float2 *>(sS + (y * L::rows + r) * G::SSTR + key);
                        v.x += u.x;
                        v.y += u.y;
                    }
                    z[x][0] = v.x * rs[c];
                    z[x][1] = v.y * rs[c];
                    if (FP8) {
                        const unsigned char *sc = smem + L::sc + st * 2 * KT + key;
                        const float2 ks = e8m0_pair(*reinterpret_cast<const uint16_t *>(sc));
                        const uint32_t vb = *reinterpret_cast<const uint16_t *>(sc + KT);
                        z[x][0] *= ks.x;
                        z[x][1] *= ks.y;
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            // the exponent as a float, by way of 2^23 + byte; byte 255 is NaN
                            const uint32_t y = vb >> (8 * e) & 255u;
                            ve[x][e] = y == 255u ? __uint_as_float(0x7fffffffu)
                                                 : __uint_as_float(0x4b000000u | y) - 8388735.0f;
                        }
                    }
                    if (tail) {
                        const bool there = (bad >> (key >> p.box_log2) & 1) == 0;   // (a box holds both keys)
#pragma unroll
                        for (int e = 0; e < 2; ++e)
                            if (!there || key0 + key + e >= lim[c]) {
                                z[x][e] = -INFINITY;
                                ve[x][e] = 0.0f;
                            } else {
                                seen |= 1u << c;
                            }
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) top = fmaxf(top, z[x][e]);
                }
                const float mn = fmaxf(m[c], warp_max(top));
                // (an infinite maximum only where nothing, an infinity or nothing but NaN was seen: the maxima pass
                // over NaN, which the sum and the weights take up)
                const float base = mn == -INFINITY ? 0.0f : mn;
                l[c] *= ex2(m[c] - base);
                float f, based = 0.0f;
                if (FP8) {
                    // the same of score + exponent, which start from the scores less their maximum: on a score of
                    // 2^24 and more the exponent would be rounded away
                    float topd = -INFINITY;
#pragma unroll
                    for (int x = 0; x < KT / 64; ++x)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            z[x][e] -= base;
                            ve[x][e] += z[x][e];
                            topd = fmaxf(topd, ve[x][e]);
                        }
                    const float d = dv[c] + (m[c] - base), dn = fmaxf(d, warp_max(topd));
                    based = dn == -INFINITY ? 0.0f : dn;
                    f = ex2(d - based);
                    dv[c] = dn;
                } else {
                    f = ex2(m[c] - base);
                }
                if (lane == 0) corr[r] = f;   // (0 where nothing was seen yet: the sums are 0)
                m[c] = mn;
                float sum = 0.0f;   // of the tile: added to the running sum at once, or small weights drift beside a large one
#pragma unroll
                for (int x = 0; x < KT / 64; ++x) {
                    float w[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        w[e] = ex2(FP8 ? z[x][e] : z[x][e] - base);
                        sum += w[e];
                        if (FP8) w[e] = ex2(ve[x][e] - based + kWeightBits);
                    }
                    *reinterpret_cast<uint32_t *>(sP + r * G::PSTR + x * 64 + 2 * lane) = pack16<FP8>(w[0], w[1]);
                }
                l[c] += sum;
            }
            const int scales = st;
            if (++st == NST) {
                st = 0;
                ph ^= 1;
            }
            if (tail) {
                // the values of slots that hold no key: zeros (a weight of 0 times whatever lies there is not 0), so that
                // the products need no masks.  (They are read after the next barrier.)
                if (!dead && !mbar_wait(&full_v[stv], phv, p.err)) dead = true;
                dead = __any_sync(0xffffffffu, dead);
                unsigned char *const values = smem + stv * 2 * G::TILE + G::TILE;
                auto chunk = [&](int key, int c) {   // 16 bytes of a key's value row, in any order
                    return values + (key >> p.box_log2) * (boxrows * G::ROWB) + (c / (G::SUBB / 16)) * substride +
                           (key & (boxrows - 1)) * G::SUBB + c % (G::SUBB / 16) * 16;
                };
                constexpr int CPR = G::ROWB / 16;
                if (!dead && (bad != 0 || key0 + KT > len.keys)) {
                    const int end = min(KT, ((int)len.keys - key0 + 31) & ~31);   // (the products stop there)
#pragma unroll 1
                    for (int x = tid; x < (i + 1 < n ? KT : end) * CPR; x += G::THREADS) {
                        const int key = x / CPR;
                        if (key0 + key >= len.keys || (bad >> (key >> p.box_log2) & 1) != 0)
                            *reinterpret_cast<uint4 *>(chunk(key, x % CPR)) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();   // (before the next fill of the stage)
                }
                // a NaN or infinity among the values that only later tokens see
                if (!dead && p.T > 1) {
                    bool nan = false;
                    for (int key = max(all_see - key0, 0) + warp; key < KT && key0 + key < len.keys; key += W) {
                        if (bad >> (key >> p.box_log2) & 1) continue;
                        for (int x = lane; x < G::ROWB / 4; x += 32) {
                            const uint32_t v = *reinterpret_cast<const uint32_t *>(chunk(key, x / 4) + x % 4 * 4);
                            if (FP8) {
                                const uint32_t y = v & 0x7f7f7f7fu;
                                nan |= (y & 0xff) == 0x7f || (y & 0xff00) == 0x7f00 || (y & 0xff0000) == 0x7f0000 ||
                                       (y >> 24) == 0x7f;
                            } else {
                                nan |= (v & 0x7f80u) == 0x7f80u || (v & 0x7f800000u) == 0x7f800000u;
                            }
                        }
                    }
                    if (nan) nan_tile = tile_no;
                }
            }
            // usually both are there already: one look on the way to the barrier instead of two waits after it
            const bool more = i + 1 < n;
            const bool v_there = mbar_test(&full_v[stv], phv), k_there = mbar_test(&full_k[st], ph);
            consumer_sync<G::THREADS>();
            if (FP8 && !dead && lane == 0) mbar_arrive(&empty_k[scales]);

            // the next tile's scores and this one's O^T += V^T P^T, which do not wait for each other
            if (!__all_sync(0xffffffffu, v_there && (k_there || !more))) {
                if (!dead && !mbar_wait(&full_v[stv], phv, p.err)) dead = true;
                dead = __any_sync(0xffffffffu, dead);
                if (more) wait_keys();
            }
            if (more) see_keys();
            if (!dead) {
                const uint32_t vbase = ring + stv * 2 * G::TILE + G::TILE;
#pragma unroll
                for (int c = 0; c < NT; ++c) {
                    const float2 f = *reinterpret_cast<const float2 *>(corr + c * 8 + 2 * j);
#pragma unroll
                    for (int d = 0; d < G::DPW; ++d) {
                        acc[d][c][0] *= f.x;
                        acc[d][c][1] *= f.y;
                        acc[d][c][2] *= f.x;
                        acc[d][c][3] *= f.y;
                    }
                }
                // two key blocks (32 keys)
                auto step = [&](int kk, bool masked, int see, float (&sum)[G::DPW][NT][4]) {
                    uint32_t pf[NT][4];
#pragma unroll
                    for (int c = 0; c < NT; ++c)
                        ldsm4(smem_u32(sP) + ((c * 8 + mr) * G::PSTR + kk * 16 + mi * 8) * 2, pf[c]);
#pragma unroll
                    for (int k2 = 0; k2 < 2; ++k2) {
                        const int kb = kk + k2;
                        // masked: zeros for values that the token does not see
                        uint32_t keep[2] = {0xffffffffu, 0xffffffffu};
                        if (masked) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const int key = kb * 16 + e * 8 + 2 * j;
                                const bool there = (bad >> (key >> p.box_log2) & 1) == 0;
                                keep[e] = there ? (key0 + key < see ? 0xffffu : 0u) |
                                                      (key0 + key + 1 < see ? 0xffff0000u : 0u)
                                                : 0u;
                            }
                        }
                        const uint32_t base = vbase + key_base(kb * 16);
                        uint32_t vraw[4];
#pragma unroll
                        for (int d = 0; d < G::DPW; ++d) {
                            uint32_t v[4];
                            if (!FP8) {
                                ldsm4t(base + voff[FP8 ? 0 : d], v);
                                if (masked) {
                                    v[0] &= keep[0];
                                    v[1] &= keep[0];
                                    v[2] &= keep[1];
                                    v[3] &= keep[1];
                                }
                            } else {
                                if (d % 2 == 0) ldsm4t(base + voff[d / 2], vraw);
                                uint32_t lo = vraw[2 * (d % 2)], hi = vraw[2 * (d % 2) + 1];
                                if (masked) {
                                    lo &= keep[0];
                                    hi &= keep[1];
                                }
                                lo = __byte_perm(lo, 0, 0x3120);   // (key, key + 1) of channel 2g, then of 2g + 1
                                hi = __byte_perm(hi, 0, 0x3120);
                                codes_f16(lo, v[0], v[1]);
                                codes_f16(hi, v[2], v[3]);
                            }
#pragma unroll
                            for (int c = 0; c < NT; ++c)
                                mma<FP8>(sum[d][c], v[0], v[1], v[2], v[3], pf[c][2 * k2], pf[c][2 * k2 + 1]);
                        }
                    }
                };
                const int kk0 = o_part * G::KK;
                // (a NaN that some tokens do not see: 0 times it is not 0)
                const bool window = tail && p.T > 1 && *static_cast<volatile uint32_t *>(&nan_tile) == tile_no;
                if (!window && more) {
                    scores();
#pragma unroll
                    for (int kk = 0; kk < G::KK; kk += 2) step(kk0 + kk, false, 0, acc);
                } else if (!window) {
                    // (the last tile: blocks of 32 keys that hold none are left out)
                    const int held = ((int)len.keys - key0 + 31) / 32 * 2;
#pragma unroll
                    for (int kk = 0; kk < G::KK; kk += 2) {
                        if (kk0 + kk >= held) break;
                        step(kk0 + kk, false, 0, acc);
                    }
                } else {
                    if (more) scores();
                    // one pass per token over the values it sees, the other rows' sums dropped
                    for (int t = 0; t < len.n; ++t) {
                        float one[G::DPW][NT][4] = {};
                        const int see = (int)min(max(len.pos + t + 1, 0LL), len.keys);
#pragma unroll 1
                        for (int kk = 0; kk < G::KK; kk += 2) step(kk0 + kk, true, see, one);
#pragma unroll
                        for (int c = 0; c < NT; ++c)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (((r0 + c * 8 + 2 * j + (e & 1)) * p.g_mul >> 16) == t) {
#pragma unroll
                                    for (int d = 0; d < G::DPW; ++d) acc[d][c][e] += one[d][c][e];
                                }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty_v[stv]);
            }
            if (++stv == NST) {
                stv = 0;
                phv ^= 1;
            }
            if (more) put_scores();
        }

        // the unit's output, or this share's part of it.  Lane c finishes row c of the warp: its factors (of a row that
        // saw nothing: -1), log-sum-exp or part.  What a row saw is counted and not read off its maximum, which is
        // -inf after scores of NaN too: there the sum is NaN (after scores of -inf: 0, and the output 0 / 0).
        const bool whole = seg.whole();
        const int slot = 2 * blockIdx.x + (first ? 0 : 1);
        {
            float top = -INFINITY, sum = 0.0f, topd = 0.0f;
            bool none = true;
            seen = __reduce_or_sync(0xffffffffu, seen);
#pragma unroll
            for (int c = 0; c < RPW; ++c) {
                float x = l[c];
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                if (lane == c) {
                    top = m[c];
                    topd = dv[c];
                    sum = x;
                    none = lim[c] == 0 || (seen >> c & 1) == 0;   // (also a token that is not there)
                }
            }
            const int r = lane * W + warp;
            if (lane < RPW && r < nrows) {
                // (2^dv: the weighted sum in units of 2^m; without a maximum it is 0 or NaN in any units.  The second
                // factor comes first: it takes the sum to the values' codes, the other one these to the values)
                fin[r] = make_float2(none ? -1.0f : FP8 && top != -INFINITY ? ex2(topd) : 1.0f,
                                     (whole ? rcp_fast(sum) : 1.0f) * (FP8 ? kWeightUnit : 1.0f));
                if (none) {
                    top = -INFINITY;
                    sum = 0.0f;
                }
                if (!whole) {
                    p.part_ml[(size_t)slot * p.rows + r] = make_float2(top, none ? -1.0f : sum);
                } else if (p.lse != nullptr) {
                    const int rr = r0 + r, t = rr * p.g_mul >> 16, hq = h * p.G + rr - t * p.G;
                    p.lse[((long long)b * p.T + t) * p.Hq + hq] = (top + log2f(sum)) * kLn2;
                }
            }
        }
        // the parts of O that went over other keys, joined in their order in S's place
        auto part = [&](int y, int d, int c, int e) -> float & {
            return sS[(((y * NT + c) * G::DB + o_blk + d) * 4 + e) * 32 + lane];
        };
        if (G::KSPL > 1 && o_part > 0) {
#pragma unroll
            for (int d = 0; d < G::DPW; ++d)
#pragma unroll
                for (int c = 0; c < NT; ++c)
#pragma unroll
                    for (int e = 0; e < 4; ++e) part(o_part - 1, d, c, e) = acc[d][c][e];
        }
        consumer_sync<G::THREADS>();
        if (G::KSPL > 1 && o_part == 0) {
#pragma unroll 1
            for (int y = 0; y < G::KSPL - 1; ++y)
#pragma unroll
                for (int d = 0; d < G::DPW; ++d)
#pragma unroll
                    for (int c = 0; c < NT; ++c)
#pragma unroll
                        for (int e = 0; e < 4; ++e) acc[d][c][e] += part(y, d, c, e);
        }
        if (o_part == 0) {
#pragma unroll
            for (int c = 0; c < NT; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const int r = c * 8 + 2 * j + x;
                    if (r >= nrows) continue;
                    const float2 f = fin[r];
                    const int rr = r0 + r, t = rr * p.g_mul >> 16, hq = h * p.G + rr - t * p.G;
                    const long long bt = (long long)b * p.T + t;
#pragma unroll
                    for (int d = 0; d < G::DPW; ++d) {
                        // channels d0, d1 of this thread's two values
                        const int dt = (o_blk + d) * 16, d0 = FP8 ? dt + 2 * g : dt + g, d1 = FP8 ? d0 + 1 : d0 + 8;
                        float o0 = acc[d][c][x], o1 = acc[d][c][2 + x];
                        o0 = f.x < 0.0f ? 0.0f : o0 * f.y * f.x;   // (the reciprocal of no sum is an infinity)
                        o1 = f.x < 0.0f ? 0.0f : o1 * f.y * f.x;
                        if (!whole) {
                            float *dst = p.part_o + ((size_t)slot * p.rows + r) * D;
                            dst[d0] = o0;
                            dst[d1] = o1;
                            continue;
                        }
                        if (gated && !(f.x < 0.0f)) {   // (the gate of a token that is not there may be NaN)
                            const uint32_t z = EARLY ? gates[EARLY ? d : 0][EARLY ? c : 0][x] : gate_pair(r, d);
                            o0 *= gate_value(__uint_as_float(z << 16));
                            o1 *= gate_value(__uint_as_float(z & 0xffff0000u));
                        }
                        uint16_t *dst = p.out + (bt * p.Hq + hq) * D;
                        if (FP8) {
                            *reinterpret_cast<uint32_t *>(dst + d0) = pack2(o0, o1);
                        } else {
                            dst[d0] = f32_to_bf16(o0);
                            dst[d1] = f32_to_bf16(o1);
                        }
                    }
                }
        }
        if (ta == 0 && !whole && tid == 0) {
            // the unit goes on: its last tile lies in the share that holds that tile's slot
            p.meta[3 * blockIdx.x] = (b * p.Hkv + h) * p.RB + (p.RB == 1 ? 0 : r0 / p.rows);
            p.meta[3 * blockIdx.x + 1] = (int)sh.of(seg.first_slot + len.tiles - 1);
            p.meta[3 * blockIdx.x + 2] = slot;
        }
        first = false;
    }
}

// Joins the partial results of the unit that starts in share blockIdx.x and
// goes on, if there is one: rows blockIdx.y, + gridDim.y ...  D/4 threads take
// four channels each of a group of parts; a chain of few loads: what the
// parts hold is asked for before their weights are known.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS) attn_join_kernel(const Params p) {
    constexpr int COLS = D / 4, GROUPS = THREADS / COLS, UNROLL = 4;
    __shared__ float4 sums[GROUPS][COLS];
    __shared__ float red_m[GROUPS], red_l[GROUPS];
    grid_dep_enter();
    const int c0 = blockIdx.x, unit = p.meta[3 * c0];
    if (unit < 0) return;
    // its first part lies in that share's slot, the others in the first slots of the shares that follow
    const int n = p.meta[3 * c0 + 1] - c0 + 1, first_slot = p.meta[3 * c0 + 2];
    const int heads = p.Hkv * p.RB, b = unit / heads, h = unit % heads / p.RB, r0 = (unit % heads % p.RB) * p.rows;
    const int nrows = min(p.rows, p.R - r0);
    const int tid = threadIdx.x, col = tid % COLS, grp = tid / COLS;
    for (int r = blockIdx.y; r < nrows; r += gridDim.y) {
        const int rr = r0 + r, t = rr / p.G, hq = h * p.G + rr % p.G;
        const long long bt = (long long)b * p.T + t;
        constexpr int OUTS = (D + THREADS - 1) / THREADS;
        uint16_t gate[OUTS];   // (asked for before it is needed)
#pragma unroll
        for (int i = 0; i < OUTS; ++i) {
            const int d = tid + i * THREADS;
            gate[i] = p.gate.p != nullptr && d < D ? p.gate.p[bt * p.gate.ts + hq * p.gate.hs + d] : 0;
        }
        // this group's parts, with a running maximum.  A part without a maximum has the weight 0: it saw nothing (its
        // sums are -1 and 0), only scores of -inf (0 and 0) or only NaN (both NaN, and 0 times them is NaN).
        float m = -INFINITY, l = 0.0f;
        bool seen = false;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        for (int i0 = grp; i0 < n; i0 += GROUPS * UNROLL) {
            float2 v[UNROLL];
            float4 x[UNROLL];
#pragma unroll
            for (int k = 0; k < UNROLL; ++k) {
                const int i = i0 + k * GROUPS;
                const size_t slot = i == 0 ? first_slot : 2 * (c0 + i);
                v[k] = make_float2(-INFINITY, -1.0f);
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
                seen |= !(v[k].y < 0.0f);
                const float w = v[k].x == -INFINITY ? 0.0f : ex2(v[k].x - top);
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
            red_l[grp] = seen ? l : -1.0f;
        }
        __syncthreads();
#pragma unroll
        for (int x = 0; x < OUTS; ++x) {
            const int d = tid + x * THREADS;
            if (d >= D) break;
            float top = -INFINITY, acc = 0.0f, total = 0.0f;
            bool any = false;
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) top = fmaxf(top, red_m[i]);
#pragma unroll
            for (int i = 0; i < GROUPS; ++i) {
                any |= !(red_l[i] < 0.0f);
                const float w = red_m[i] == -INFINITY ? 0.0f : ex2(red_m[i] - top);
                acc = fmaf(w, reinterpret_cast<const float *>(sums[i])[d], acc);
                total = fmaf(w, red_l[i], total);
            }
            float y = any ? acc / total : 0.0f;
            if (any && p.gate.p != nullptr) y *= gate_value(bf16_to_f32(gate[x]));
            p.out[(bt * p.Hq + hq) * D + d] = f32_to_bf16(y);
            if (d == 0 && p.lse != nullptr) p.lse[bt * p.Hq + hq] = (top + log2f(total)) * kLn2;
        }
    }
}

// Row blocks of a (b, h) and the query rows of one.  (Blocks of 64 read the keys
// once where two of 32 read them twice, but spill registers: B = 32, 64 rows, 4
// key heads of 256 channels, e4m3, 2300 keys: 213 against 114 us.)
void row_blocks(const AttnSizes &s, int *blocks, int *rows) {
    constexpr int kMost = 32;
    const int R = s.T * (s.Hq / s.Hkv);
    *blocks = (R + kMost - 1) / kMost;
    *rows = (R + *blocks - 1) / *blocks;
}

size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Workspace {
    size_t o, ml, meta, total;
};

Workspace workspace(const AttnSizes &s) {
    int blocks, rows;
    row_blocks(s, &blocks, &rows);
    const size_t ctas = (size_t)num_sms() * kMaxCtas, slots = 2 * ctas;
    Workspace w;
    w.o = 0;
    w.ml = up256(slots * rows * s.D * sizeof(float));
    w.meta = w.ml + up256(slots * rows * sizeof(float2));
    w.total = w.meta + up256(ctas * 3 * sizeof(int));
    return w;
}

template <class G, int NT>
cudaError_t launch_t(const Params &p0, cudaStream_t st) {
    Params p = p0;
    int lg = 0;
    while ((1 << lg) < G::KT) ++lg;
    p.box_log2 = p.c.shift < lg ? p.c.shift : lg;
    constexpr int smem = Smem<G, NT>::total;
    static unsigned long long done = 0;
    cudaError_t e = set_max_smem(done, attn_decode_kernel<G, NT>, smem);
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
    const unsigned long long units = (unsigned long long)p.B * p.Hkv * p.RB;
    if (units * (((unsigned long long)p.c.width << p.c.shift) / G::KT + 1 + kBlank) > 0x7fffffffULL) return cudaErrorNotSupported;
    const int ctas = num_sms() * G::CTAS;
    e = DependentLaunch(dim3(ctas), dim3((G::W + G::PRODUCERS) * 32), smem, st)(attn_decode_kernel<G, NT>, maps[0],
                                                                               maps[1], p);
    if (e != cudaSuccess) return e;
    // (a table with no room for a second tile: no unit has parts; 1 key: 4.7 us, with a join that finds none 7.3)
    if (((long long)p.c.width << p.c.shift) <= G::KT) return cudaSuccess;
    const dim3 grid(ctas, p.rows < 8 ? p.rows : 8);
    // few units: many parts each, more threads to read them; many units: mostly two parts, small CTAs (2 key heads of
    // 256 channels, 8000 keys, one row: 11.6 us for the whole call with 256 threads, 17.0 with 128; 4000 keys, 64
    // rows: 87.0 and 86.0; 512 threads gain 0.5 us on the first and lose 0.8 at 1000 keys)
    if (units * 8 < (unsigned)ctas) return DependentLaunch(grid, dim3(256), 0, st)(attn_join_kernel<G::D, 256>, p);
    return DependentLaunch(grid, dim3(128), 0, st)(attn_join_kernel<G::D, 128>, p);
}

// Eight consumer warps (B = 128, 8 query heads per key head, 2048 keys of 256
// channels in e4m3: 53.5 us; four 56.9, sixteen 58.6).
template <int D, bool FP8>
cudaError_t launch_g(Params &p, const AttnSizes &s, cudaStream_t st) {
    using G = Geo<D, FP8, false>;
    row_blocks(s, &p.RB, &p.rows);
    if constexpr (FP8 || D < 256) {
        // Short tables: a unit's start and end cost more than its keys, and two CTAs go through them side by side (B =
        // 128, 32 and 8 heads of 128 channels, e4m3: one tile of up to 128 keys 15.7 us, with 32 KB tiles 26.4; 300
        // keys 27.1 against 38.3).  With few units and more keys the larger tile is ahead (B = 1, 2 heads, 600 keys:
        // 9.0 against 10.2 us), and so it is with more than 8 query rows (16, 100 keys: 8.6 against 9.2 us).
        using GS = Geo<D, FP8, true>;
        const long long cap = (long long)p.c.width << p.c.shift, units = (long long)p.B * p.Hkv;
        if (p.rows <= 8 && cap <= (units >= 4 * num_sms() ? 4 : 1) * GS::KT) return launch_t<GS, 1>(p, st);
    }
    if (p.rows <= 8) return launch_t<G, 1>(p, st);
    if (p.rows <= 16) return launch_t<G, 2>(p, st);
    return launch_t<G, 4>(p, st);
}

template <int D>
cudaError_t launch_d(Params &p, const AttnSizes &s, cudaStream_t st) {
    return p.c.fp8 ? launch_g<D, true>(p, s, st) : launch_g<D, false>(p, s, st);
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
    p.g_mul = 65536 / p.G + 1;
    p.R = s.T * p.G;
    p.scale2 = scale * kLog2e;
    const Workspace w = workspace(s);
    char *base = static_cast<char *>(ws);
    p.part_o = reinterpret_cast<float *>(base + w.o);
    p.part_ml = reinterpret_cast<float2 *>(base + w.ml);
    p.meta = reinterpret_cast<int *>(base + w.meta);
    if (s.D == 64) return launch_d<64>(p, s, st);
    if (s.D == 128) return launch_d<128>(p, s, st);
    return launch_d<256>(p, s, st);
}

}  // namespace gdn
