// Gradients of a prompt's attention (prompt_fwd.cu).  With P = exp(scale S -
// lse), dO the output's gradient (times the gate), delta = rowsum(dO O):
//   dV = P^T dO,  dP = dO V^T,  dS = P (dP - delta),
//   dQ = scale dS K,  dK = scale dS^T Q,  dgate = dout out (1 - sigmoid(gate)).
// P and dS are rounded to bf16 for their products, as the other operands are.
//
// 10 D operations per seen (query head, key) are needed: bound by the tensor
// cores.  Here a tile of 128 rows (queries of a key head's group, or keys) stays
// in a CTA and the others pass by in steps of 64 rows: one kernel accumulates
// dQ, others dK and dV, so that every sum is in a fixed order in one
// accumulator, without atomics; S and dP are computed twice (14 D; with 256
// channels, where dK and dV do not fit the tensor memory together, S three
// times: 16 D).
//   - The resident rows are A operands in tensor memory (with 256 channels the
//     second one lies in shared memory): a product of 128 x 64 with both
//     operands in shared memory takes 48 clocks for 32 clocks' work (measured),
//     with A in tensor memory 32.  They come by TMA through the stages of the
//     rows that pass by (read row by row by the warps they took 7000 cycles a
//     tile, a quarter of a tile of 20 steps).
//   - A step: S and dP into tensor memory; two warpgroups take half of its columns
//     each (dQ with up to 128 channels: every other step each) into registers,
//     which frees them for the next step at once, and leave P and dS as bf16 in
//     shared memory, the A operands of the accumulating products.
//   - The lists, shares and joins are those of the forward pass (prompt.cuh).
//
// Measured on a GB300, per 10 D operations of a seen pair, calls on fresh inputs
// (in brackets on the same again and again): 8192 tokens, 16 query heads on 2, 256
// channels, gate: 1540-1600 us, 860-895 TFLOP/s (1480-1550; dQ 501, dK 504, dV 361,
// gate and delta 49, join 23, tensor cores 71 to 78 % busy); 8 sequences of 100 to
// 2045 tokens packed, 32 on 8, 128 channels: 370 us, 646 TFLOP/s (369; dQ 146, dK and
// dV 178).  Steps are bound by the shared memory's bandwidth: dQ
// with 128 channels reads 64 KB and writes 48 for 768 cycles of products, some
// 900 cycles at 128 bytes a clock (a second buffer of S and dP changed nothing:
// 382 us for 383).  Pairs of CTAs that share the rows that pass by would halve
// that.
#include "prompt.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace prompt;

enum { kDQ, kDKV, kDK, kDV };

constexpr int kRows = 64;   // of a step

template <int D_, int KIND_>
struct Geo {
    static constexpr int D = D_, KIND = KIND_;
    static constexpr bool KEYS = KIND != kDQ;                       // the resident rows are keys
    static constexpr bool HAS_DP = KIND != kDV, HAS_P = KIND == kDKV || KIND == kDV;   // dP needed; P accumulated
    static constexpr int ACCS = (HAS_DP ? 1 : 0) + (HAS_P ? 1 : 0);
    static constexpr bool A2_SMEM = D == 256 && HAS_DP, A2_RING = D <= 128 && HAS_DP;   // how the second tile comes and stays
    static constexpr int A1_COL = ACCS * D, A2_COL = A1_COL + D / 2, S_COL = HAS_DP && !A2_SMEM ? A2_COL + D / 2 : A2_COL;
    static_assert(S_COL + 128 <= 512, "");
    static constexpr int SUB = kRows * 128;                         // bytes of 64 rows of 64 channels
    static constexpr int STAGE = D / 64 * SUB;
    // the second ring: whole steps, or with 256 channels, where no second one has room, 64 channels at a time
    static constexpr int N1 = D == 256 ? (KIND == kDV ? 2 : 3) : 4;
    static constexpr int STAGE2 = A2_SMEM ? SUB : STAGE, N2 = A2_SMEM ? 5 : D == 256 ? 3 : 4, PER_STEP2 = STAGE / STAGE2;
    static constexpr int XTILE = 128 * 128, XT = ACCS, XB = A2_SMEM ? 1 : 2;   // 128 rows of 64 bf16; tiles; buffers
    static constexpr int A2_BYTES = A2_SMEM ? 128 * D * 2 : 0;
    static constexpr int WARPS = 8, TURN = 32 * 32;
    // two warpgroups: every other step each, the products of a step two steps later; or half of every step's columns each
    static constexpr bool TURNS = D <= 128 && KIND == kDQ;
    static constexpr int LATER = TURNS ? 2 : 1, COLS = TURNS ? 64 : 32, ROWS_WARPS = TURNS ? 4 : 8;
    static constexpr int THREADS = 32 * (WARPS + 2 + (KEYS ? 1 : 0));
    static constexpr int X_AT = A2_BYTES, RING1 = X_AT + XB * XT * XTILE, RING2 = RING1 + N1 * STAGE,
                         SMEM = RING2 + N2 * STAGE2 + 1024;
    static_assert(WARPS * TURN <= XTILE, "");   // (results are turned into rows where P and dS lay)
    static_assert(SMEM + 4608 <= 227 * 1024, "");
};

constexpr int kStats = 4;   // steps of row statistics in shared memory

struct Params {
    List list;
    HeadsIn a1, a2;          // the resident rows
    const uint16_t *out, *dout;
    HeadsIn q, k, v, d_o;    // for rows that are done once more
    float scale, scale2;
    const float *lse;
    float *delta;
    uint16_t *acc_out[2];
    float *part;             // [slot][acc][D / 4][128][4]
    int *again;              // [CTA]: rows of its whole tiles are not finite, and are left to the joins; null: no joins follow
    unsigned *err;
    int Hq, Hkv, G, box, tps;   // tokens: of 64 query rows, of a step
};

struct Bars {
    uint64_t full1[4], empty1[4], full2[5], empty2[5], a_full, a2_full, a2_free, s_full[2], s_free, x_full[2], x_free[2], acc_done, acc_free, end;
    uint64_t stats_full[kStats], stats_free[kStats];
    Loaded loaded1, loaded2;
    int units;   // whose second resident tile was loaded
};

// (s_full and x_free: of even and odd steps.  A wait for a phase is sound if the one before it is over, and each warpgroup
// waits for every other step only.)
struct Stats {
    float nlse[kRows], delta[kRows];   // -lse in powers of two (-infinity: no such row); -delta
    int token[kRows];
};

struct RowOut {
    long long at;       // (token, head) of the outputs
    long long token;
    int head;
    bool mine, valid;
};

template <class G>
__device__ __forceinline__ RowOut row_out(const Params &p, const Unit &u, int head, int r) {
    RowOut o;
    // (queries: two boxes of 64 rows, G heads of a token after the other)
    const int x = (r & (kRows - 1)) / p.G, t = G::KEYS ? r : r / kRows * p.box + x;
    o.head = G::KEYS ? head : head * p.G + (r & (kRows - 1)) - x * p.G;
    const bool row = G::KEYS || x < p.box;
    o.mine = row && t < u.slot_a;
    o.valid = row && t < u.n_a;
    o.token = (long long)u.a0 + t;
    o.at = o.token * (G::KEYS ? p.Hkv : p.Hq) + o.head;
    return o;
}

// ---------------------------------------------------------------------------
// rows by the definition (results that are not finite: what lies in unseen
// slots must not have entered)
// ---------------------------------------------------------------------------
template <int D>
__device__ __forceinline__ void lane_row(const HeadsIn &h, long long n, int head, float (&x)[D / 32]) {
    prompt::lane_row<D>(h.p + n * h.ts + head * h.hs, x);
}

// One row's dQ (KEYS false: query (token, head), over `n` keys from `first`) or
// dK / dV (key (token, head), over the queries of `n` tokens from `first`, of
// which the token i sees it if row <= lim0 + i); channels d0 .. d1 - 1.
template <int D, bool KEYS>
__device__ __noinline__ void exact_row(const Params &p, long long token, int head, int first, int n, int row, int lim0,
                                       bool of_p, uint16_t *out, int d0, int d1) {
    constexpr int N = D / 32;
    const int lane = threadIdx.x & 31;
    float a1[N], a2[N], acc[N];
    lane_row<D>(p.a1, token, head, a1);
    if (!KEYS || !of_p) lane_row<D>(p.a2, token, head, a2);
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
    const int heads = KEYS ? p.G : 1;
    for (int i = 0; i < n; ++i) {
        if (KEYS && row > lim0 + i) continue;
        for (int g = 0; g < heads; ++g) {
            const long long q_token = KEYS ? (long long)first + i : token, k_token = KEYS ? token : (long long)first + i;
            const int qh = KEYS ? head * p.G + g : head, kh = KEYS ? head : head / p.G;
            float x[N], y[N];
            lane_row<D>(KEYS ? p.q : p.k, KEYS ? q_token : k_token, KEYS ? qh : kh, x);
            const float w = expf(row_dot<D>(a1, x) * p.scale - p.lse[q_token * p.Hq + qh]);
            lane_row<D>(KEYS ? p.d_o : p.v, KEYS ? q_token : k_token, KEYS ? qh : kh, y);
            if (KEYS && of_p) {
#pragma unroll
                for (int c = 0; c < N; ++c) acc[c] = fmaf(w, y[c], acc[c]);
            } else {
                const float ds = w * (row_dot<D>(a2, y) - p.delta[q_token * p.Hq + qh]);
#pragma unroll
                for (int c = 0; c < N; ++c) acc[c] = fmaf(ds, x[c], acc[c]);
            }
        }
        if (all_nan(acc)) break;
    }
    const float f = KEYS && of_p ? 1.0f : p.scale;
#pragma unroll
    for (int c = 0; c < N; ++c) {
        const int d = lane * N + c;
        if (d >= d0 && d < d1) out[d] = f32_to_bf16(acc[c] * f);
    }
}

template <class G>
__device__ __forceinline__ void mend_rows(const Params &p, const RowOut &o, const Unit &u, int row, bool of_p, bool bad,
                                          uint16_t *out, int d0, int d1) {
    unsigned todo = __ballot_sync(0xffffffffu, bad && o.mine && o.valid);
    while (todo != 0) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const long long token = __shfl_sync(0xffffffffu, o.token, src), at = __shfl_sync(0xffffffffu, o.at, src);
        const int head = __shfl_sync(0xffffffffu, o.head, src), r = __shfl_sync(0xffffffffu, row, src);
        const int n = G::KEYS ? u.n_b : max(u.lim0 + (int)(token - u.a0), 0);
        exact_row<G::D, G::KEYS>(p, token, head, u.b0, n, r, u.lim0, of_p, out + at * G::D, d0, d1);
    }
}

// 32 channels from d of the warp's rows, rounded (0 for rows that are padding).
template <int D>
__device__ __forceinline__ void write_group(uint8_t *turn, uint16_t *const (&rows)[2], bool valid, int d, const float *x) {
    const int lane = threadIdx.x & 31;
    const bool some = __any_sync(0xffffffffu, !valid);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float *y = x + 16 * h + 8 * i;
            uint4 w = make_uint4(attn::pack2(y[0], y[1]), attn::pack2(y[2], y[3]), attn::pack2(y[4], y[5]), attn::pack2(y[6], y[7]));
            if (some && !valid) w = make_uint4(0, 0, 0, 0);
            *reinterpret_cast<uint4 *>(turn + turn_at(lane, i)) = w;
        }
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (rows[k] != nullptr)
                *reinterpret_cast<uint4 *>(rows[k] + d + 16 * h) =
                    *reinterpret_cast<const uint4 *>(turn + turn_at(16 * k + (lane >> 1), lane & 1));
        __syncwarp();
    }
}

template <int D>
__device__ __forceinline__ void rows_out(const RowOut &o, uint16_t *out, uint16_t *(&rows)[2]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int src = 16 * k + (lane >> 1);
        const long long at = __shfl_sync(0xffffffffu, o.at, src);
        const bool mine = __shfl_sync(0xffffffffu, (int)o.mine, src);
        rows[k] = mine ? out + at * D + (lane & 1) * 8 : nullptr;
    }
}

// ---------------------------------------------------------------------------
// the pass
// ---------------------------------------------------------------------------
// The warps that hold rows meet.
__device__ __forceinline__ void meet() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <class G>
__global__ void __launch_bounds__(G::THREADS, 1)
prompt_backward_kernel(const __grid_constant__ CUtensorMap map1, const __grid_constant__ CUtensorMap map2,
                       const __grid_constant__ CUtensorMap res1, const __grid_constant__ CUtensorMap res2,
                       const __grid_constant__ Params p) {
    constexpr int D = G::D;
    extern __shared__ uint8_t raw[];
    __shared__ Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead, again;   // again: rows are not finite
    __shared__ __align__(16) Stats stats[G::KEYS ? kStats : 1];
    __shared__ float swap[G::KEYS || G::TURNS ? 1 : 256];   // deltas of rows of few keys: [half][row]
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (warp == 0) {
        umma::tmem_alloc(&tmem_slot, 512);
        umma::tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        dead = again = 0;
        bars.loaded1 = bars.loaded2 = {0, 0};
        bars.units = 0;
        for (int i = 0; i < 5; ++i) {
            if (i < 4) {
                mbar_init(&bars.full1[i], 1);
                mbar_init(&bars.empty1[i], 1);
            }
            mbar_init(&bars.full2[i], 1);
            mbar_init(&bars.empty2[i], 1);
        }
        mbar_init(&bars.a_full, G::WARPS);
        mbar_init(&bars.a2_full, 1);
        mbar_init(&bars.a2_free, 1);
        mbar_init(&bars.s_free, G::ROWS_WARPS);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.x_full[i], G::ROWS_WARPS);
            mbar_init(&bars.x_free[i], 1);
        }
        mbar_init(&bars.acc_done, 1);
        mbar_init(&bars.end, 1);
        mbar_init(&bars.acc_free, G::WARPS);
        for (int i = 0; i < kStats; ++i) {
            mbar_init(&bars.stats_full[i], 1);
            mbar_init(&bars.stats_free[i], G::ROWS_WARPS);
        }
        fence_mbar_init();
    }
    if (G::KEYS) {   // rows of a step that no token has: zeros, never written again
        const int used = p.tps * p.G, rows = kRows - used;
        for (int i = threadIdx.x; i < (G::N1 * G::STAGE + G::N2 * G::STAGE2) / G::SUB * rows * 8; i += G::THREADS) {
            const int c = i & 7, r = i >> 3;
            *reinterpret_cast<uint4 *>(smem + G::RING1 + r / rows * G::SUB + (used + r % rows) * 128 + c * 16) =
                make_uint4(0, 0, 0, 0);
        }
    }
    fence_proxy_async_smem();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    attn::grid_dep_enter();

    const Waits wait{p.err, &dead};
    Walk w;
    const bool any = w.begin(p.list, blockIdx.x);
    if (any && warp == G::WARPS) {
        // ---- loads
        if (umma::elect_one()) {
            prefetch_tmap(&map1);
            prefetch_tmap(&map2);
            prefetch_tmap(&res1);
            prefetch_tmap(&res2);
        }
        int s1 = 0, s2 = 0, units = 0;
        uint32_t ph1 = 0, ph2 = 0;
        auto pass1 = [&] {
            if (++s1 == G::N1) {
                s1 = 0;
                ph1 ^= 1;
            }
        };
        auto pass2 = [&] {
            if (++s2 == G::N2) {
                s2 = 0;
                ph2 ^= 1;
            }
        };
        // 64 rows of queries or keys, `subs` groups of 64 channels from group `sub`
        auto load = [&](bool queries, const CUtensorMap *map, uint8_t *dst, uint64_t *bar, int head, int token, int sub, int subs) {
            if (queries) {
                mbar_expect_tx(bar, (uint32_t)(subs * 128 * p.box * p.G));
                for (int i = 0; i < subs; ++i) tma_load_3d(dst + i * G::SUB, map, (sub + i) * 64, head * p.G, token, bar);
            } else {
                mbar_expect_tx(bar, (uint32_t)(subs * G::SUB));
                tma_load_4d(dst, map, 0, token, sub, head, bar);
            }
        };
        do {
            w.uniform();
            // the resident rows, 64 in a stage, come through the rings before the steps
            const int half = G::KEYS ? kRows : p.box;   // tokens of 64 rows
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
                if (!wait.together(&bars.empty1[s1], ph1 ^ 1)) goto loaded;
                if (umma::elect_one())
                    load(!G::KEYS, &res1, smem + G::RING1 + s1 * G::STAGE, &bars.full1[s1], w.head, w.u.a0 + h * half, 0, D / 64);
                pass1();
                if (G::A2_RING) {
                    if (!wait.together(&bars.empty2[s2], ph2 ^ 1)) goto loaded;
                    if (umma::elect_one())
                        load(!G::KEYS, &res2, smem + G::RING2 + s2 * G::STAGE2, &bars.full2[s2], w.head, w.u.a0 + h * half, 0, D / 64);
                    pass2();
                }
            }
            for (int i = w.first; i < w.last; ++i) {
                const int token = w.u.b0 + i * p.tps;
                if (!wait.together(&bars.empty1[s1], ph1 ^ 1)) goto loaded;
                if (umma::elect_one())
                    load(G::KEYS, &map1, smem + G::RING1 + s1 * G::STAGE, &bars.full1[s1], w.head, token, 0, D / 64);
                pass1();
                if (G::A2_SMEM && i == w.first) {   // the second resident tile, to where it stays
                    if (units > 0 && !wait.together(&bars.a2_free, (units - 1) & 1)) goto loaded;
                    if (umma::elect_one()) {
                        mbar_expect_tx(&bars.a2_full, G::KEYS ? 128 * D * 2 : 2 * p.box * p.G * D * 2);
#pragma unroll 1
                        for (int c = 0; c < 2 * (D / 64); ++c) {
                            uint8_t *dst = smem + c * G::SUB;
                            if (G::KEYS)
                                tma_load_4d(dst, &res2, 0, w.u.a0 + (c & 1) * half, c >> 1, w.head, &bars.a2_full);
                            else
                                tma_load_3d(dst, &res2, (c >> 1) * 64, w.head * p.G, w.u.a0 + (c & 1) * half, &bars.a2_full);
                        }
                    }
                    ++units;
                }
#pragma unroll 1
                for (int c = 0; c < G::PER_STEP2; ++c) {
                    if (!wait.together(&bars.empty2[s2], ph2 ^ 1)) goto loaded;
                    if (umma::elect_one())
                        load(G::KEYS, &map2, smem + G::RING2 + s2 * G::STAGE2, &bars.full2[s2], w.head, token, c,
                             G::STAGE2 / G::SUB);
                    pass2();
                }
            }
        } while (__any_sync(0xffffffffu, w.next()));
    loaded:
        bars.loaded1 = {s1, ph1};
        bars.loaded2 = {s2, ph2};
        bars.units = units;
    } else if (any && warp == G::WARPS + 1) {
        // ---- products
        const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0), at = smem_u32(smem);
        constexpr uint32_t id_s = umma::idesc(128, kRows, umma::kFmtBF16);
        constexpr uint32_t id_a = umma::idesc(128, D, umma::kFmtBF16) | umma::kBTransposed;
        const uint64_t d_b1 = umma::desc_sw128(at + G::RING1), d_b2 = umma::desc_sw128(at + G::RING2);
        const uint64_t d_t1 = umma::desc_sw128_mn(at + G::RING1, G::SUB), d_t2 = umma::desc_sw128_mn(at + G::RING2, G::SUB);
        const uint64_t d_x = umma::desc_sw128(at + G::X_AT), d_a2 = umma::desc_sw128(at);
        int s1 = 0, s2 = 0, t1 = 0, t2 = 0, step = 0, units = 0, done = 0;   // s: of the scores, t: of the accumulating products
        uint32_t ph1 = 0, ph2 = 0;
        bool acc = false;
        int waiting = 0;   // steps whose accumulating products are still to come
        // the products of step x into the accumulators
        auto accumulate = [&](int x, bool last) {
            const int xb = x % G::XB;
            wait(&bars.x_full[xb], (x / G::XB) & 1);
            if (!acc && done > 0) wait(&bars.acc_free, (done - 1) & 1);
            umma::fence_after_sync();
            const uint64_t a = d_x + (uint32_t)(xb * G::XT * (G::XTILE >> 4));
            if (!acc) {   // (a new tile: its resident rows have had two stages)
                t1 = (t1 + 2) % G::N1;
                if (G::A2_RING) t2 = (t2 + 2) % G::N2;
            }
            if (G::HAS_DP) {
                umma::warp_mma_bf16_k64_bt(base, a, d_t1 + (uint32_t)(t1 * (G::STAGE >> 4)), id_a, acc);
                umma::warp_mma_commit(&bars.empty1[t1]);
                if (++t1 == G::N1) t1 = 0;
            }
            if (G::HAS_P) {
                umma::warp_mma_bf16_k64_bt(base + (G::HAS_DP ? D : 0), a + (G::HAS_DP ? G::XTILE >> 4 : 0),
                                           d_t2 + (uint32_t)(t2 * (G::STAGE2 >> 4)), id_a, acc);
                umma::warp_mma_commit(&bars.empty2[t2]);
                if (++t2 == G::N2) t2 = 0;
            }
            umma::warp_mma_commit(&bars.x_free[x & 1]);
            acc = true;
            if (last) {
                umma::warp_mma_commit(&bars.acc_done);
                ++done;
                acc = false;
            }
        };
        bool more = true;
        while (more) {
            w.uniform();
            wait(&bars.a_full, units & 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {   // the stages of the resident rows, which are in the tensor memory now
                if (umma::elect_one()) {
                    mbar_arrive(&bars.empty1[s1]);
                    if (G::A2_RING) mbar_arrive(&bars.empty2[s2]);
                }
                if (++s1 == G::N1) {
                    s1 = 0;
                    ph1 ^= 1;
                }
                if (G::A2_RING && ++s2 == G::N2) {
                    s2 = 0;
                    ph2 ^= 1;
                }
            }
            for (int i = w.first; i < w.last; ++i, ++step) {
                if (step > 0) wait(&bars.s_free, (step - 1) & 1);
                wait(&bars.full1[s1], ph1);
                umma::fence_after_sync();
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    umma::warp_mma_bf16_tmem_a_k64(base + G::S_COL, base + G::A1_COL + c * 32,
                                                   d_b1 + (uint32_t)((s1 * G::STAGE + c * G::SUB) >> 4), id_s, c > 0);
                if (!G::HAS_DP) umma::warp_mma_commit(&bars.empty1[s1]);
                if (++s1 == G::N1) {
                    s1 = 0;
                    ph1 ^= 1;
                }
                if (G::A2_SMEM && i == w.first) wait(&bars.a2_full, units & 1);
#pragma unroll 1
                for (int h = 0; h < G::PER_STEP2; ++h) {
                    wait(&bars.full2[s2], ph2);
                    umma::fence_after_sync();
                    if (G::HAS_DP) {
#pragma unroll
                        for (int c = 0; c < G::STAGE2 / G::SUB; ++c) {
                            const uint64_t b = d_b2 + (uint32_t)((s2 * G::STAGE2 + c * G::SUB) >> 4);
                            if (G::A2_SMEM)
                                umma::warp_mma_bf16_k64(base + G::S_COL + 64, d_a2 + (uint32_t)(h * ((128 * 128) >> 4)), b, id_s,
                                                        h > 0);
                            else
                                umma::warp_mma_bf16_tmem_a_k64(base + G::S_COL + 64, base + G::A2_COL + c * 32, b, id_s, c > 0);
                        }
                        if (!G::HAS_P) umma::warp_mma_commit(&bars.empty2[s2]);
                    }
                    if (++s2 == G::N2) {
                        s2 = 0;
                        ph2 ^= 1;
                    }
                }
                umma::warp_mma_commit(&bars.s_full[step & 1]);
                if (G::A2_SMEM && i + 1 == w.last) umma::warp_mma_commit(&bars.a2_free);
                ++waiting;
                // (of this tile: with products two steps later those of the last tile are through, see below)
                if (waiting > G::LATER) {
                    accumulate(step - G::LATER, G::LATER == 1 && i == w.first);
                    --waiting;
                }
            }
            ++units;
            more = __any_sync(0xffffffffu, w.next());
            // One step later: the next tile's first scores come before this one's last products, if the ring has room for
            // the last step, two stages of resident rows and the first step.  Two: not, as their rows' warps would wait for
            // these before they take the scores.
            if (G::LATER > 1 || (G::HAS_DP && G::N1 < 4) || !more)
                for (; waiting > 0; --waiting) accumulate(step - waiting, waiting == 1);
        }
        // every product is through before the tensor memory goes back
        umma::warp_mma_commit(&bars.end);
        wait_end(&bars.end, 0, p.err);
    } else if (G::KEYS && any && warp == G::WARPS + 2) {
        // ---- the statistics of the rows that pass by
        int st = 0;
        uint32_t ph = 0;
        int t[2], g[2];
        for (int k = 0; k < 2; ++k) {
            t[k] = (lane + 32 * k) / p.G;
            g[k] = lane + 32 * k - t[k] * p.G;
        }
        do {
            for (int i = w.first; i < w.last; ++i) {
                float nlse[2], delta[2];
                int token[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int x = i * p.tps + t[k];
                    const bool there = t[k] < p.tps && x < w.u.n_b;
                    const long long at = ((long long)w.u.b0 + x) * p.Hq + w.head * p.G + g[k];
                    nlse[k] = there ? -kLog2e * p.lse[at] : -INFINITY;
                    delta[k] = there && G::HAS_DP ? -p.delta[at] : 0.0f;
                    token[k] = there ? x : -0x40000000;
                }
                wait(&bars.stats_free[st], ph ^ 1);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    stats[st].nlse[lane + 32 * k] = nlse[k];
                    stats[st].delta[lane + 32 * k] = delta[k];
                    stats[st].token[lane + 32 * k] = token[k];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.stats_full[st]);
                if (++st == kStats) {
                    st = 0;
                    ph ^= 1;
                }
            }
        } while (w.next());
    } else if (any && warp < G::WARPS) {
        // ---- P and dS, and the results
        const int half = warp >> 2, r = (warp & 3) * 32 + lane, col0 = G::TURNS ? 0 : half * 32;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21);
        uint8_t *turn = smem + G::X_AT + warp * G::TURN;
        // The resident rows from the stages that they came in (the `at1`th and next of the first ring, the `at2`th and next of
        // the second) to the tensor memory: half of the warps takes A1, half A2, or each half of A1's channels.
        int at1 = 0, at2 = 0;
        auto load_resident = [&](const RowOut &o) {
            const int h = r / kRows, rr = r & (kRows - 1);
            const bool second = G::A2_RING && half == 1;
            const int n = second ? (at2 + h) % G::N2 : (at1 + h) % G::N1;
            wait(second ? &bars.full2[n] : &bars.full1[n], ((second ? (at2 + h) / G::N2 : (at1 + h) / G::N1)) & 1);
            uint8_t *src = smem + (second ? G::RING2 + n * G::STAGE2 : G::RING1 + n * G::STAGE);
#pragma unroll(D <= 128 ? 2 : 1)
            for (int c = G::A2_RING ? 0 : half; c < D / 64; c += G::A2_RING ? 1 : 2) {
                float y[32];
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    uint4 *at = reinterpret_cast<uint4 *>(src + c * G::SUB + umma::sw128(rr, k * 16));
                    const uint4 x = o.valid ? *at : make_uint4(0, 0, 0, 0);
                    y[4 * k] = __uint_as_float(x.x);
                    y[4 * k + 1] = __uint_as_float(x.y);
                    y[4 * k + 2] = __uint_as_float(x.z);
                    y[4 * k + 3] = __uint_as_float(x.w);
                    if (G::KEYS && rr >= p.tps * p.G) *at = make_uint4(0, 0, 0, 0);   // (no token's in the steps, see above)
                }
                umma::tmem_st32(lanes + (second ? G::A2_COL : G::A1_COL) + c * 32, y);
            }
            umma::tmem_st_wait();
            fence_proxy_async_smem();
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.a_full);
            at1 += 2;
            at2 += 2;
        };
        RowOut o = row_out<G>(p, w.u, w.head, r);
        load_resident(o);
        int step = 0, st = 0, units = 0;
        uint32_t ph = 0;
        bool more = true;
        float nlse = -INFINITY, delta = 0.0f;
        int keys = 0;
        auto row_stats = [&](const RowOut &o, const Unit &u) {
            nlse = -INFINITY;
            delta = 0.0f;
            keys = 0;
            if (!G::KEYS && o.valid) {
                keys = max(u.lim0 + (int)(o.token - u.a0), 0);
                if (keys > 0) nlse = -kLog2e * p.lse[o.at];
                if (keys > kRows) delta = p.delta[o.at];   // (else known at step 0; later steps have nothing for the row)
            }
        };
        row_stats(o, w.u);
        while (more) {
            for (int i = w.first; i < w.last; ++i, ++step) {
                const int xb = step % G::XB, stat = st;
                const uint32_t stat_phase = ph;
                if (G::KEYS && ++st == kStats) {
                    st = 0;
                    ph ^= 1;
                }
                if (G::TURNS && (step & 1) != half) continue;   // (the other warpgroup's)
                constexpr int PARTS = G::COLS / 32;
                float s[PARTS][32], dp[PARTS][32];
                wait(&bars.s_full[step & 1], (step >> 1) & 1);
                umma::fence_after_sync();
#pragma unroll
                for (int c = 0; c < PARTS; ++c) umma::tmem_ld32(lanes + G::S_COL + col0 + c * 32, s[c]);
                if (G::HAS_DP)
#pragma unroll
                    for (int c = 0; c < PARTS; ++c) umma::tmem_ld32(lanes + G::S_COL + 64 + col0 + c * 32, dp[c]);
                umma::tmem_ld_wait();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.s_free);
                const Stats *x = &stats[G::KEYS ? stat : 0];
                // P of two scores; dS of two weights, by -delta
                auto weigh = [&](float *v, F2 n) {
                    const float2 e = parts(fma2(f2_of(v[0], v[1]), f2_of(p.scale2, p.scale2), n));
                    v[0] = ex2(e.x);
                    v[1] = ex2(e.y);
                };
                auto slope = [&](float *v, const float *d, F2 n) {
                    const float2 e = parts(mul2(f2_of(v[0], v[1]), add2(f2_of(d[0], d[1]), n)));
                    v[0] = e.x;
                    v[1] = e.y;
                };
                if (G::KEYS) {
                    wait(&bars.stats_full[stat], stat_phase);
#pragma unroll
                    for (int k = 0; k < G::COLS; k += 4) {
                        const float4 n = *reinterpret_cast<const float4 *>(&x->nlse[col0 + k]);
                        weigh(&s[k / 32][k % 32], f2_of(n.x, n.y));
                        weigh(&s[k / 32][k % 32 + 2], f2_of(n.z, n.w));
                    }
                    // (not all keys seen by the step's first token, or rows behind the last token)
                    if (w.u.lim0 + i * p.tps < 127 || (i + 1) * p.tps > w.u.n_b) {
#pragma unroll
                        for (int k = 0; k < G::COLS; k += 4) {
                            const int4 n = *reinterpret_cast<const int4 *>(&x->token[col0 + k]);
                            const int tok[4] = {n.x, n.y, n.z, n.w};
#pragma unroll
                            for (int z = 0; z < 4; ++z)
                                if (r > w.u.lim0 + tok[z]) {
                                    s[k / 32][k % 32 + z] = 0.0f;
                                    if (G::HAS_DP) dp[k / 32][k % 32 + z] = 0.0f;
                                }
                        }
                    }
                } else {
                    const int lim = keys - i * kRows - col0;
#pragma unroll
                    for (int k = 0; k < G::COLS; k += 2) weigh(&s[k / 32][k % 32], f2_of(nlse, nlse));
                    if (__any_sync(0xffffffffu, lim < G::COLS)) {
#pragma unroll
                        for (int k = 0; k < G::COLS; ++k)
                            if (k >= lim) s[k / 32][k % 32] = dp[k / 32][k % 32] = 0.0f;
                    }
                    if (i == 0 && w.u.lim0 <= kRows) {
                        // rows that see no key behind this step: their delta from P and dP themselves (the output's rounding
                        // to bf16 is too coarse for rows of few keys), also for the kernels that come after
                        float t[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int k = 0; k < G::COLS; ++k) t[k & 3] = fmaf(s[k / 32][k % 32], dp[k / 32][k % 32], t[k & 3]);
                        float sum = (t[0] + t[1]) + (t[2] + t[3]);
                        if (!G::TURNS) {
                            swap[half * 128 + r] = sum;
                            meet();
                            sum = swap[r] + swap[128 + r];
                            meet();
                        }
                        if (keys <= kRows) {
                            delta = sum;
                            if (o.valid && (G::TURNS || half == 0)) p.delta[o.at] = delta;
                        }
                    }
                }
                if (step >= G::XB) wait(&bars.x_free[(step - G::XB) & 1], ((step - G::XB) >> 1) & 1);
                uint8_t *xs = smem + G::X_AT + xb * G::XT * G::XTILE;
                auto put = [&](uint8_t *tile) {
#pragma unroll
                    for (int c = 0; c < G::COLS / 8; ++c) {
                        const float *v = &s[c / 4][c % 4 * 8];
                        const float y[8] = {v[0], v[1], v[2], v[3], v[4], v[5], v[6], v[7]};
                        *reinterpret_cast<uint4 *>(tile + umma::sw128(r, col0 * 2 + c * 16)) = attn::pack8(y);
                    }
                };
                if (G::HAS_P) put(xs + (G::HAS_DP ? G::XTILE : 0));
                if (G::HAS_DP) {
                    if (G::KEYS) {
#pragma unroll
                        for (int k = 0; k < G::COLS; k += 4) {
                            const float4 n = *reinterpret_cast<const float4 *>(&x->delta[col0 + k]);
                            slope(&s[k / 32][k % 32], &dp[k / 32][k % 32], f2_of(n.x, n.y));
                            slope(&s[k / 32][k % 32 + 2], &dp[k / 32][k % 32 + 2], f2_of(n.z, n.w));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < G::COLS; k += 2)
                            slope(&s[k / 32][k % 32], &dp[k / 32][k % 32], f2_of(-delta, -delta));
                    }
                    put(xs);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars.x_full[xb]);
                    if (G::KEYS) mbar_arrive(&bars.stats_free[stat]);
                }
            }
            if (G::TURNS) meet();   // (the next rows go where the other warpgroup's last step has its own)
            // the next tile's resident rows, then this one's results
            Walk y = w;
            more = y.next();
            const bool whole = w.whole();
            const int slot = w.slot(blockIdx.x);
            const bool valid = o.valid && (!G::KEYS || w.u.n_b > 0) && (G::KEYS || keys > 0);
            RowOut next = o;
            if (more) {
                next = row_out<G>(p, y.u, y.head, r);
                at1 += w.last - w.first;
                at2 += w.last - w.first;
                load_resident(next);
                row_stats(next, y.u);
            }
            wait(&bars.acc_done, units & 1);
            umma::fence_after_sync();
#pragma unroll 1
            for (int a = 0; a < G::ACCS; ++a) {
                const bool of_p = a == 1 || !G::HAS_DP;
                const float f = of_p ? 1.0f : p.scale;
                uint16_t *rows[2];
                rows_out<D>(o, p.acc_out[a], rows);
#pragma unroll 1
                for (int d = half * 32; d < D; d += 64) {
                    float v[32];
                    umma::tmem_ld32(lanes + a * D + d, v);
                    umma::tmem_ld_wait();
                    if (whole) {
                        const bool bad = scaled(v, f);
                        write_group<D>(turn, rows, valid, d, v);
                        // (where no joins follow a row meets six steps' others at most; what meets more would take longer
                        // than the bounded waits of the other warps allow)
                        if (p.again == nullptr)
                            mend_rows<G>(p, o, w.u, r, of_p, valid && bad, p.acc_out[a], d, d + 32);
                        else if (valid && bad)
                            again = 1;
                    } else {
                        float4 *dst = reinterpret_cast<float4 *>(p.part) +
                                      (((size_t)slot * G::ACCS + a) * (D / 4) + d / 4) * 128 + r;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            dst[(size_t)k * 128] = make_float4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
                    }
                }
            }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars.acc_free);
            meet();   // (the next P and dS go where rows were turned)
            ++units;
            w = y;
            o = next;
        }
        umma::fence_before_sync();
    }
    __syncthreads();
    umma::fence_after_sync();
    if (dead && threadIdx.x == 0) {
        for (int i = 0; i < G::N1; ++i) wait_end(&bars.full1[i], bars.loaded1.parity(i), p.err);
        for (int i = 0; i < G::N2; ++i) wait_end(&bars.full2[i], bars.loaded2.parity(i), p.err);
        if (G::A2_SMEM) wait_end(&bars.a2_full, (bars.units & 1) ^ 1, p.err);
    }
    if (warp == 0) umma::tmem_dealloc(tmem, 512);
    if (threadIdx.x == 0 && p.again != nullptr) p.again[blockIdx.x] = again && !dead;
}

// The rows of a CTA's whole tiles that are not finite once more, a row a warp (the `at`th of `warps`).
template <class G>
__device__ __noinline__ void rows_again(const Params &p, int cta, int at, int warps) {
    Walk w;
    if (!w.begin(p.list, cta)) return;
    do {
        if (!w.whole()) continue;
        for (int x = at; x < 128 * G::ACCS; x += warps) {
            const int r = x % 128, a = x / 128;
            const RowOut o = row_out<G>(p, w.u, w.head, r);
            const int n = G::KEYS ? w.u.n_b : w.u.lim0 + (int)(o.token - w.u.a0);
            uint16_t *out = p.acc_out[a] + o.at * G::D;
            if (!o.valid || n <= 0 || finite_row<G::D>(out)) continue;
            exact_row<G::D, G::KEYS>(p, o.token, o.head, w.u.b0, n, r, w.u.lim0, a == 1 || !G::HAS_DP, out, 0, G::D);
        }
    } while (w.next());
}

// Split tiles' parts added up: 32 channels of 128 rows a block.
template <class G>
__device__ __forceinline__ void join_parts(const Params &p, int slice, uint8_t (&turn)[4][G::TURN]) {
    constexpr int D = G::D;
    if (p.again[blockIdx.x] != 0) rows_again<G>(p, blockIdx.x, slice * 4 + (threadIdx.x >> 5), G::ACCS * (D / 32) * 4);
    if (blockIdx.x + 1 == gridDim.x) return;   // (no tile goes on behind the last share)
    const Parts part = parts_from(p.list, blockIdx.x);
    if (part.n == 0) return;
    const int a = slice / (D / 32), c = slice % (D / 32), r = threadIdx.x;
    const RowOut o = row_out<G>(p, part.u, part.head, r);
    uint16_t *rows[2];
    rows_out<D>(o, p.acc_out[a], rows);
    float x[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = 0.0f;
    // (two parts' loads at a time)
    for (int i = 0; i < part.n; i += 2) {
        float4 v[2][8];
#pragma unroll
        for (int z = 0; z < 2; ++z) {
            const size_t slot = 2 * (size_t)(blockIdx.x + i + z) + (i + z == 0 ? 1 : 0);
            const float4 *src = reinterpret_cast<const float4 *>(p.part) + ((slot * G::ACCS + a) * (D / 4) + c * 8) * 128 + r;
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[z][k] = i + z < part.n ? src[(size_t)k * 128] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        }
#pragma unroll
        for (int z = 0; z < 2; ++z)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                x[4 * k] += v[z][k].x;
                x[4 * k + 1] += v[z][k].y;
                x[4 * k + 2] += v[z][k].z;
                x[4 * k + 3] += v[z][k].w;
            }
    }
    const bool of_p = a == 1 || !G::HAS_DP;
    const bool bad = scaled(x, of_p ? 1.0f : p.scale);
    const bool valid = o.valid && (G::KEYS || part.u.lim0 + (int)(o.token - part.u.a0) > 0);
    write_group<D>(turn[threadIdx.x >> 5], rows, valid, c * 32, x);
    mend_rows<G>(p, o, part.u, r, of_p, valid && bad, p.acc_out[a], c * 32, c * 32 + 32);
}

// All three (dQ, dK, dV): blockIdx.y is the accumulator and its channels.
template <int D>
__global__ void __launch_bounds__(128) prompt_backward_join_kernel(const __grid_constant__ Params q, const __grid_constant__ Params k, const __grid_constant__ Params v) {
    __shared__ __align__(16) uint8_t turn[4][Geo<D, kDQ>::TURN];
    attn::grid_dep_enter();
    const int slice = blockIdx.y;
    if (slice < D / 32) {
        join_parts<Geo<D, kDQ>>(q, slice, turn);
    } else if constexpr (D <= 128) {
        join_parts<Geo<D, kDKV>>(k, slice - D / 32, turn);
    } else if (slice < 2 * (D / 32)) {
        join_parts<Geo<D, kDK>>(k, slice - D / 32, turn);
    } else {
        join_parts<Geo<D, kDV>>(v, slice - 2 * (D / 32), turn);
    }
}

// ---------------------------------------------------------------------------
// before the passes: delta = rowsum(dout out), and with a gate dO = dout
// sigmoid(gate), rounded to bf16 for the products, and the gate's own gradient.
// Memory-bound: 47 us for the 335 MB of 8192 tokens (16 heads of 256 channels,
// gate), 7.1 TB/s with what stays in L2; a tile's rows in one block, one
// after another, took 56.
// ---------------------------------------------------------------------------
struct PrepareParams {
    List list;
    const uint16_t *out, *dout;
    HeadsIn gate;
    uint16_t *d_o, *dgate;
    float *delta;
    const int32_t *cu_q;
    int Hq, Hkv, G, tile, B;
    long long Nq;
};

template <int D>
__global__ void __launch_bounds__(256) prompt_prepare_kernel(const PrepareParams p) {
    // a group of LPR lanes takes two rows of an item of 2 RPB rows: all loads of both, then the rest
    constexpr int LPR = D / 8, RPB = 256 / LPR, ROWS = 2 * RPB;   // (4096 / D)
    const int sub = threadIdx.x / LPR, d = threadIdx.x % LPR * 8;
    attn::grid_dep_enter();
    const Header h = *p.list.header;
    const int rows = p.tile * p.G, parts = (rows + ROWS - 1) / ROWS;
    const long long per_head = (long long)h.units * parts, items = per_head * p.Hkv;
    const bool gated = p.gate.p != nullptr;
    for (long long x = blockIdx.x; x < items; x += gridDim.x) {
        const int head = (int)(x / per_head), y = (int)(x - head * per_head), unit = y / parts;
        const Unit u = p.list.unit[unit];
        long long at[2];
        bool mine[2];
        uint4 dout[2], out[2], gate[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int r = (y - unit * parts) * ROWS + i * RPB + sub, t = r / p.G, hq = head * p.G + r - t * p.G;
            const long long n = (long long)u.a0 + t;
            at[i] = n * p.Hq + hq;
            mine[i] = r < rows && t < u.slot_a;
            const bool there = mine[i] && t < u.n_a;
            const uint4 none = make_uint4(0, 0, 0, 0);
            dout[i] = there ? *reinterpret_cast<const uint4 *>(p.dout + at[i] * D + d) : none;
            out[i] = there ? *reinterpret_cast<const uint4 *>(p.out + at[i] * D + d) : none;
            gate[i] = there && gated ? *reinterpret_cast<const uint4 *>(p.gate.p + n * p.gate.ts + hq * p.gate.hs + d) : none;
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            float a[8], b[8], sum = 0.0f;
            attn::unpack8(dout[i], a);
            attn::unpack8(out[i], b);
#pragma unroll
            for (int k = 0; k < 8; ++k) sum = fmaf(a[k], b[k], sum);
            if (gated) {   // (padding: zeros)
                float g[8], z[8];
                attn::unpack8(gate[i], g);
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const float e = exp_fast(-g[k]), sg = rcp_fast(1.0f + e);
                    z[k] = a[k] * sg;
                    a[k] *= b[k] * (e < INFINITY ? e * sg : 1.0f);   // 1 - sigmoid
                }
                if (mine[i]) {
                    *reinterpret_cast<uint4 *>(p.d_o + at[i] * D + d) = attn::pack8(z);
                    *reinterpret_cast<uint4 *>(p.dgate + at[i] * D + d) = attn::pack8(a);
                }
            }
#pragma unroll
            for (int o = LPR / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o, LPR);
            if (d == 0 && mine[i]) p.delta[at[i]] = sum;
        }
    }
    // rows behind the last sequence, which its last steps may bring along: finite
    if (gated && p.cu_q != nullptr && h.units > 0 && blockIdx.x == 0) {
        const long long end = p.cu_q[p.B], most = end + kRows < p.Nq ? end + kRows : p.Nq;
        for (long long i = threadIdx.x; i < (most - end) * p.Hq * (D / 8); i += 256)
            reinterpret_cast<uint4 *>(p.d_o + end * p.Hq * D)[i] = make_uint4(0, 0, 0, 0);
    }
}

// A tile's start and end in steps (T = 8192: 2 1483 us, 3 1439, 4 1440, 6 1446, 9 1492; packed, 128 channels: 391, 381, 368,
// 369, 383).
constexpr int kBlank = 4;

PromptList q_list(const PromptSizes &s) {
    return PromptList{false, 2 * (kRows / (s.Hq / s.Hkv)), kRows, num_sms(), 4, kBlank, 6};
}

PromptList k_list(const PromptSizes &s) {
    return PromptList{true, 128, kRows / (s.Hq / s.Hkv), num_sms(), 4, kBlank, 6};
}

struct Workspace {
    size_t k, d_o, delta, part[3], again, total;
};

Workspace workspace(const PromptSizes &s, bool gated) {
    Workspace w;
    const size_t part = up256(2 * (size_t)num_sms() * 128 * s.D * sizeof(float));
    w.k = prompt_list_bytes(s, q_list(s));
    w.delta = w.k + prompt_list_bytes(s, k_list(s));
    w.d_o = w.delta + up256((size_t)s.Nq * s.Hq * sizeof(float));
    w.part[0] = w.d_o + (gated ? up256((size_t)s.Nq * s.Hq * s.D * 2) : 0);
    w.part[1] = w.part[0] + part;
    w.part[2] = w.part[1] + part;      // (up to 128 channels: the second half of dK and dV's)
    w.again = w.part[2] + part;
    w.total = w.again + up256(3 * (size_t)num_sms() * sizeof(int));
    return w;
}

template <class G>
cudaError_t launch_pass(const CUtensorMap &m1, const CUtensorMap &m2, const CUtensorMap &r1, const CUtensorMap &r2,
                        const Params &p, cudaStream_t st) {
    static unsigned long long done = 0;
    cudaError_t e = set_max_smem(done, prompt_backward_kernel<G>, G::SMEM);
    if (e != cudaSuccess) return e;
    return DependentLaunch(dim3(num_sms()), dim3(G::THREADS), G::SMEM, st)(prompt_backward_kernel<G>, m1, m2, r1, r2, p);
}

template <int D>
cudaError_t launch_d(const PromptSizes &s, const PromptSeqs &seqs, const HeadsIn &q, const HeadsIn &k, const HeadsIn &v,
                     const HeadsIn &gate, const uint16_t *out, const float *lse, const uint16_t *dout, float scale, uint16_t *dq,
                     uint16_t *dk, uint16_t *dv, uint16_t *dgate, char *ws, unsigned *err, cudaStream_t st) {
    const bool gated = gate.p != nullptr;
    const Workspace w = workspace(s, gated);
    const PromptList lists[2] = {q_list(s), k_list(s)};
    void *const at[2] = {ws, ws + w.k};
    cudaError_t e = launch_prompt_plan(s, seqs, lists, 2, at, err, st);
    if (e != cudaSuccess) return e;
    const int G = s.Hq / s.Hkv;
    uint16_t *d_o = gated ? reinterpret_cast<uint16_t *>(ws + w.d_o) : nullptr;
    PrepareParams r = {};
    r.list = prompt_list_at(s, lists[0], at[0]);
    r.out = out;
    r.dout = dout;
    r.gate = gate;
    r.d_o = d_o;
    r.dgate = dgate;
    r.delta = reinterpret_cast<float *>(ws + w.delta);
    r.cu_q = seqs.cu_q;
    r.Hq = s.Hq;
    r.Hkv = s.Hkv;
    r.G = G;
    r.tile = lists[0].tile;
    r.B = s.B;
    r.Nq = s.Nq;
    const int parts = (r.tile * G + 4096 / D - 1) / (4096 / D);   // items of a tile
    const long long most = ((s.Nq + r.tile - 1) / r.tile + s.B) * s.Hkv * parts, fill = 16LL * num_sms();
    if (s.Nq > 0) e = DependentLaunch(dim3((unsigned)(most < fill ? most : fill)), dim3(256), 0, st)(prompt_prepare_kernel<D>, r);
    if (e != cudaSuccess) return e;

    const HeadsIn g{gated ? d_o : dout, (long long)s.Hq * D, D};
    const bool none = s.Nk == 0;   // (no keys, or no queries: nothing of what is loaded counts, but a map needs a tensor)
    const bool no_q = s.Nq == 0;
    const HeadsIn dummy{no_q ? k.p : q.p, 0, 0};
    CUtensorMap mq, mg, mk, mv;
    const int tps = lists[1].step;
    if (!queries_map(&mq, no_q ? dummy : q, no_q ? 1 : s.Nq, no_q ? 1 : s.Hq, D, G, tps) ||
        !queries_map(&mg, no_q ? dummy : g, no_q ? 1 : s.Nq, no_q ? 1 : s.Hq, D, G, tps) ||
        !keys_map(&mk, none ? dummy : k, none ? 1 : s.Nk, none ? 1 : s.Hkv, D, kRows, D / 64) ||
        !keys_map(&mv, none ? dummy : v, none ? 1 : s.Nk, none ? 1 : s.Hkv, D, kRows, Geo<D, kDQ>::STAGE2 / Geo<D, kDQ>::SUB))
        return cudaErrorInvalidValue;
    Params p = {};
    p.q = q;
    p.k = k;
    p.v = v;
    p.d_o = g;
    p.scale = scale;
    p.scale2 = scale * kLog2e;
    p.lse = lse;
    p.delta = r.delta;
    p.err = err;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.G = G;
    p.box = tps;
    auto part = [&](int i) { return reinterpret_cast<float *>(ws + w.part[i]); };

    Params pq = p;
    pq.list = r.list;
    pq.a1 = q;
    pq.a2 = g;
    pq.acc_out[0] = dq;
    pq.part = part(0);
    pq.tps = kRows;
    Params pk = p;
    pk.list = prompt_list_at(s, lists[1], at[1]);
    pk.a1 = k;
    pk.a2 = v;
    pk.part = part(1);
    pk.tps = tps;
    // (no keys, or no queries: no tile has more than a step)
    const bool joined = !none && !no_q && (prompt_splits(s, seqs, lists[0]) || prompt_splits(s, seqs, lists[1]));
    int *again = joined ? reinterpret_cast<int *>(ws + w.again) : nullptr;
    pq.again = again;
    pk.again = joined ? again + num_sms() : nullptr;
    Params pv = pk;
    pv.again = joined ? again + 2 * num_sms() : nullptr;
    pk.acc_out[0] = dk;
    pk.acc_out[1] = dv;
    pv.acc_out[0] = dv;
    pv.part = part(2);
    if (!no_q) e = launch_pass<Geo<D, kDQ>>(mk, mv, mq, mg, pq, st);
    if constexpr (D == 256) {
        if (e == cudaSuccess && !none) e = launch_pass<Geo<D, kDK>>(mq, mg, mk, mv, pk, st);
        if (e == cudaSuccess && !none) e = launch_pass<Geo<D, kDV>>(mq, mg, mk, mv, pv, st);
    } else {
        if (e == cudaSuccess && !none) e = launch_pass<Geo<D, kDKV>>(mq, mg, mk, mv, pk, st);
    }
    if (e != cudaSuccess) return e;
    if (!joined) return cudaSuccess;
    return DependentLaunch(dim3(num_sms(), 3 * (D / 32)), dim3(128), 0, st)(prompt_backward_join_kernel<D>, pq, pk, pv);
}

}  // namespace

size_t attn_prefill_backward_workspace(const PromptSizes &s, bool gated) { return workspace(s, gated).total; }

cudaError_t launch_attn_prefill_backward(const PromptSizes &s, const HeadsIn &q, const HeadsIn &k, const HeadsIn &v,
                                         const PromptSeqs &seqs, const HeadsIn &gate, float scale, const uint16_t *out,
                                         const float *lse, const uint16_t *dout, uint16_t *dq, uint16_t *dk, uint16_t *dv,
                                         uint16_t *dgate, void *ws, unsigned *err, cudaStream_t st) {
    char *base = static_cast<char *>(ws);
    if (s.D == 64) return launch_d<64>(s, seqs, q, k, v, gate, out, lse, dout, scale, dq, dk, dv, dgate, base, err, st);
    if (s.D == 128) return launch_d<128>(s, seqs, q, k, v, gate, out, lse, dout, scale, dq, dk, dv, dgate, base, err, st);
    return launch_d<256>(s, seqs, q, k, v, gate, out, lse, dout, scale, dq, dk, dv, dgate, base, err, st);
}

}  // namespace gdn
