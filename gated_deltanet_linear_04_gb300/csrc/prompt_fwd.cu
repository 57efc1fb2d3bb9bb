// Causal attention of whole prompts: out = softmax(scale Q K^T) V, query heads
// in groups on one key head, sequences of different lengths, each aligned at
// its end (the last query sees the last key), with the layer's sigmoid gate
// and the log-sum-exp.
//
// One pass over the keys of a tile with the running maximum m and sum l of the
// softmax: P = 2^(scale' S - m), O += P V.  m is taken up only when a row's
// maximum has grown by more than 8 (in powers of two; P stays below 2^8, exact
// in f32 sums and as precise in bf16 as below 1), so that the accumulators are
// hardly ever rescaled.  P is rounded to bf16 for its product (as the values
// are bf16; the sum l takes the unrounded P).
//
// 4 D operations per seen (query head, key): bound by the tensor cores.
//   - Rows of a tile are G query heads of one key head and 128 / G tokens.  Keys
//     and values come by TMA in tiles of 128 into a ring of 128-byte-swizzled
//     stages; S = Q K^T and O are accumulated in tensor memory, P goes back
//     there as the A operand of its product.
//   - One warp loads, one issues the products (as a whole warp: umma.cuh), the
//     others do the softmax, half of a step's keys each warpgroup.  Up to 128
//     channels: two tiles of 128 rows at a time share the keys, two warpgroups
//     each, so that one's softmax runs beside the other's products.  256
//     channels: O alone takes half of the tensor memory; one tile, two buffers of
//     S, the next step's scores beside this one's softmax.
//   - All tiles of all sequences and key heads are one list of steps, cut into
//     equal shares for one CTA per SM (prompt.cuh): no SM waits for the longest
//     tile, and a few rows with many keys use all of them.
//
// Measured on a GB300 (operations of seen pairs; a large bf16 product of the
// library reaches 1882 TFLOP/s; calls on fresh inputs, in brackets on the same
// again and again): 8192 tokens, 16 query heads on 2, 256 channels, gate: 383 us,
// 1435 TFLOP/s (352, 1560); 8 sequences of 100 to 4093 tokens packed, 32 on 8, 128
// channels: 310 us, 1206 (301, 1243); 512 tokens behind long prefixes: 123 us, 1325
// (119, 1370); one prompt of 77 tokens: 11 to 13 us, two launches.  With 256 channels
// a step takes some 2300 cycles for 2048 cycles of products, and a tile's end 13000
// (its results, of all warps) beside which only the next tile's first scores run.
// With 128 channels keys, values and P's reads fill the shared memory's
// bandwidth next to the tensor cores, 2600 cycles for 2048.
#include "prompt_row.cuh"
#include "umma.cuh"

namespace gdn {
namespace {

using namespace prompt;

constexpr int kKeys = 128;             // of a step
constexpr float kRaise = 8.0f;         // powers of two that a row's maximum may grow by before m follows

template <int D_>
struct Geo {
    static constexpr int D = D_;
    static constexpr int TILES = D <= 128 ? 2 : 1;
    static constexpr int SUB = 128 * 128;                  // bytes of 128 rows of 64 channels
    static constexpr int QTILE = D / 64 * SUB;
    // a stage of the ring: 64 channels of 128 keys, or all channels of VK values
    static constexpr int STAGE = SUB, STAGES = D == 256 ? 9 : 8, PER_STEP = D / 64, VK = 128 * 64 / D;
    static constexpr int HALVES = 2;                       // warpgroups that share a tile's softmax: 64 keys of a step each
    static constexpr int WARPS = 4 * HALVES * TILES;
    static constexpr int THREADS = 32 * (WARPS + 2);
    static constexpr int TURN = 32 * 32;                   // bytes in which a warp turns 16 channels of its rows into rows
    // Results go through stages of the ring, into which their gates come by TMA, and out by TMA (packed, 128 channels, the
    // same inputs again: 300 us; turned into rows by each warp 343).  With 256 channels they would take four of nine stages
    // while the next tile's keys and values need them: there they are turned (T = 8192: 353 us; through the ring 367).
    static constexpr bool STAGED = TILES == 2;
    static constexpr int RESULTS = STAGED ? TILES * (D / 64) : 0;   // stages of a unit's results
    static constexpr int SMEM = TILES * QTILE + STAGES * STAGE + (STAGED ? 0 : WARPS * TURN) + 1024;
    static constexpr int S_COL = TILES * D;                // two buffers of 128 columns
    static_assert(SMEM + 6144 <= 227 * 1024, "");
};

struct Params {
    List list;
    HeadsIn q, k, v, gate;
    uint16_t *out;
    float *lse;
    float *part_o;     // [slot][D / 4][rows][4]
    float2 *part_ml;   // [slot][rows]
    unsigned *err;
    int Hq, Hkv, G, tpt;   // tpt: tokens of a tile
    float scale, scale2;   // scale2: in powers of two
};

struct Bars {
    uint64_t full[9], empty[9], q_full, q_free, s_full[2], p_full[2], o_done[2], o_free[2], end;
    Loaded loaded;
    int units, passed;   // units whose queries were loaded; the first stage of those that were passed over, or -1
    float most[2][2][2][128];   // [tile][step parity][half][row]: what the halves of a row tell each other
    float sum[2][2][128];       // [tile][half][row], at a tile's end
};

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The two warpgroups of a tile meet.
__device__ __forceinline__ void pair_sync(int tile) {
    if (tile == 0)
        asm volatile("bar.sync 1, 256;" ::: "memory");
    else
        asm volatile("bar.sync 2, 256;" ::: "memory");
}

// `threads` threads meet (barrier `id`).
__device__ __forceinline__ void team_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// Scores that are not to be seen (from `lim` on) are -infinity.
__device__ __forceinline__ void hide(float (&s)[32], int lim) {
#pragma unroll
    for (int k = 0; k < 32; ++k) s[k] = k < lim ? s[k] : -INFINITY;
}

__device__ __forceinline__ float largest(const float (&x)[32]) {
    float a = max3(x[0], x[1], x[2]), b = max3(x[16], x[17], x[18]);
#pragma unroll
    for (int k = 3; k < 15; k += 2) {
        a = max3(a, x[k], x[k + 1]);
        b = max3(b, x[16 + k], x[17 + k]);
    }
    return max3(a, b, fmaxf(x[15], x[31]));
}

// e = 2^(s mul + add) of 32 scores, their sum added to `sum`, as bf16 pairs.
__device__ __forceinline__ void weights(const float (&s)[32], F2 mul, F2 add, F2 &sum, float *pk) {
#pragma unroll
    for (int k = 0; k < 16; ++k) {
        const float2 x = parts(fma2(f2_of(s[2 * k], s[2 * k + 1]), mul, add));
        const float2 e = make_float2(ex2(x.x), ex2(x.y));
        sum = add2(sum, f2_of(e.x, e.y));
        pk[k] = __uint_as_float(attn::pack2(e.x, e.y));
    }
}

// Writes a row's results, or what is known of it if others hold the rest.
struct RowOut {
    long long at;        // (token, head) in out and lse
    bool mine, valid;    // a row of the sequence's slot; one that holds a token
    int keys;            // that it sees
    const uint16_t *gate;
};

template <int D>
__device__ __forceinline__ RowOut row_out(const Params &p, const Unit &u, int head, int tile, int r) {
    const int t = r / p.G, g = r - t * p.G, tok = tile * p.tpt + t;
    RowOut o;
    o.mine = t < p.tpt && tok < u.slot_a;
    o.valid = t < p.tpt && tok < u.n_a;
    o.keys = o.valid ? max(u.lim0 + tok, 0) : 0;
    const long long n = (long long)u.a0 + tok;
    const int h = head * p.G + g;
    o.at = n * p.Hq + h;
    o.gate = p.gate.p == nullptr || !o.valid ? nullptr : p.gate.p + n * p.gate.ts + h * p.gate.hs;
    return o;
}

// Where a lane stands when a warp writes (or reads) its 32 rows as rows: two
// lanes to 32 bytes of a row, rows 16 k + lane / 2.
struct RowsOut {
    uint16_t *out[2];
    const uint16_t *gate[2];
};

template <int D>
__device__ __forceinline__ RowsOut rows_out(const Params &p, const RowOut &o) {
    const int lane = threadIdx.x & 31;
    RowsOut r;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int src = 16 * k + (lane >> 1);
        const long long at = __shfl_sync(0xffffffffu, o.at, src);
        const bool mine = __shfl_sync(0xffffffffu, (int)o.mine, src);
        const unsigned long long g = __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o.gate), src);
        r.out[k] = mine ? p.out + at * D + (lane & 1) * 8 : nullptr;
        r.gate[k] = g != 0 ? reinterpret_cast<const uint16_t *>(g) + (lane & 1) * 8 : nullptr;
    }
    return r;
}

// The gates of 32 channels of the warp's rows, as they are read.
struct Gates {
    uint4 v[2][2];
};

__device__ __forceinline__ Gates ask_gates(const RowsOut &r, int d) {
    Gates g;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 2; ++k)
            g.v[i][k] = r.gate[k] != nullptr ? *reinterpret_cast<const uint4 *>(r.gate[k] + d + 16 * i) : make_uint4(0, 0, 0, 0);
    return g;
}

// 32 channels from d of the warp's rows: lane i's x of row i, gated, rounded,
// written.  `zero`: the row sees nothing.
__device__ __forceinline__ void write_group(uint8_t *turn, const RowsOut &r, bool zero, bool gated, const Gates &gates, int d,
                                            const float *x) {
    const int lane = threadIdx.x & 31;
    const bool some = __any_sync(0xffffffffu, zero);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint4 w[2];
        if (gated) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<uint4 *>(turn + turn_at(16 * k + (lane >> 1), lane & 1)) = gates.v[h][k];
            __syncwarp();
            float y[2][8];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                attn::unpack8(*reinterpret_cast<const uint4 *>(turn + turn_at(lane, i)), y[i]);
#pragma unroll
                for (int k = 0; k < 8; ++k) y[i][k] = x[16 * h + 8 * i + k] * rcp_fast(1.0f + exp_fast(-y[i][k]));
                w[i] = attn::pack8(y[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float *y = x + 16 * h + 8 * i;
                w[i] = make_uint4(attn::pack2(y[0], y[1]), attn::pack2(y[2], y[3]), attn::pack2(y[4], y[5]), attn::pack2(y[6], y[7]));
            }
        }
        if (some && zero) w[0] = w[1] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<uint4 *>(turn + turn_at(lane, i)) = w[i];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (r.out[k] != nullptr)
                *reinterpret_cast<uint4 *>(r.out[k] + d + 16 * h) =
                    *reinterpret_cast<const uint4 *>(turn + turn_at(16 * k + (lane >> 1), lane & 1));
        __syncwarp();
    }
}

// 32 channels of a row into its place in a stage (from byte b of the row on),
// over its gate if there is one.
__device__ __forceinline__ void put_group(uint8_t *stage, int r, int b, bool zero, bool gated, const float *x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint4 *at = reinterpret_cast<uint4 *>(stage + umma::sw128(r, b + i * 16));
        float y[8];
        if (gated) {
            attn::unpack8(*at, y);
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = x[8 * i + k] * rcp_fast(1.0f + exp_fast(-y[k]));
        } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) y[k] = x[8 * i + k];
        }
        *at = zero ? make_uint4(0, 0, 0, 0) : attn::pack8(y);
    }
}

// The warp's rows that are not finite once more, by the definition.
template <int D>
__device__ __forceinline__ void mend_rows(const Params &p, const RowOut &o, const Unit &u, int head, bool bad, int d0,
                                          int d1) {
    unsigned todo = __ballot_sync(0xffffffffu, bad && o.mine && o.keys > 0);
    while (todo != 0) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const long long at = __shfl_sync(0xffffffffu, o.at, src);
        const int keys = __shfl_sync(0xffffffffu, o.keys, src);
        const long long n = at / p.Hq;
        const int h = (int)(at - n * p.Hq);
        exact_row<D>(p.q.p + n * p.q.ts + h * p.q.hs, p.k.p + u.b0 * p.k.ts + head * p.k.hs, p.k.ts,
                     p.v.p + u.b0 * p.v.ts + head * p.v.hs, p.v.ts, keys, p.scale,
                     p.gate.p == nullptr ? nullptr : p.gate.p + n * p.gate.ts + h * p.gate.hs, p.out + at * D, d0, d1,
                     false);
    }
}

// Behind the CTA's roles: the rows of its whole tiles that are not finite once more, by the definition, a row a warp.  (Not
// before: a row of many keys takes longer than the bounded waits of the roles allow.)
template <int D>
__device__ __forceinline__ void rows_again(const Params &p) {
    Walk w;
    if (!w.begin(p.list, blockIdx.x)) return;
    do {
        if (!w.whole()) continue;   // (joined later, in prompt_join_kernel)
        for (int r = threadIdx.x >> 5; r < Geo<D>::TILES * 128; r += Geo<D>::THREADS / 32) {
            const RowOut o = row_out<D>(p, w.u, w.head, r / 128, r % 128);
            if (!o.mine || o.keys == 0 || finite_row<D>(p.out + o.at * D)) continue;
            const long long n = o.at / p.Hq;
            const int h = (int)(o.at - n * p.Hq);
            exact_row<D>(p.q.p + n * p.q.ts + h * p.q.hs, p.k.p + w.u.b0 * p.k.ts + w.head * p.k.hs, p.k.ts,
                         p.v.p + w.u.b0 * p.v.ts + w.head * p.v.hs, p.v.ts, o.keys, p.scale, o.gate, p.out + o.at * D, 0, D, false);
        }
    } while (w.next());
}

template <int D_>
__global__ void __launch_bounds__(Geo<D_>::THREADS, 1)
prompt_forward_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap k_map,
                      const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap gate_map,
                      const __grid_constant__ CUtensorMap out_map, const __grid_constant__ Params p) {
    using G = Geo<D_>;
    constexpr int D = D_;
    extern __shared__ uint8_t raw[];
    __shared__ Bars bars;
    __shared__ uint32_t tmem_slot;
    __shared__ int dead, again;   // again: rows are not finite
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    uint8_t *ring = smem + G::TILES * G::QTILE;
    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

    if (warp == 0) {
        umma::tmem_alloc(&tmem_slot, 512);
        umma::tmem_relinquish();
    }
    if (threadIdx.x == 32) {
        dead = again = 0;
        bars.loaded = {0, 0};
        bars.units = 0;
        bars.passed = -1;
        for (int i = 0; i < G::STAGES; ++i) {
            mbar_init(&bars.full[i], 1);
            mbar_init(&bars.empty[i], 1);
        }
        mbar_init(&bars.q_full, 1);
        mbar_init(&bars.q_free, 1);
        mbar_init(&bars.end, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars.s_full[i], 1);
            mbar_init(&bars.p_full[i], 4 * G::HALVES);
            mbar_init(&bars.o_done[i], 1);
            mbar_init(&bars.o_free[i], 4 * G::HALVES);
        }
        fence_mbar_init();
    }
    // rows of a tile that no token has (128 is no multiple of G): zeros, never written again
    for (int i = threadIdx.x; i < G::TILES * (D / 64) * (128 - p.tpt * p.G) * 8; i += G::THREADS) {
        const int c = i & 7, r = i >> 3, rows = 128 - p.tpt * p.G;
        *reinterpret_cast<uint4 *>(smem + r / rows * G::SUB + (p.tpt * p.G + r % rows) * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_smem();
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = tmem_slot;
    attn::grid_dep_enter();

    // The barrier and its phase for a step's product with the values.  A wait for a phase is sound if the one before it is
    // over: one tile has two in turn, as its next scores come before its values; a step's scores, once they are there,
    // say that the values two steps back (with two tiles: one step back) are through.
    auto o_done = [&](int tile, int step) { return &bars.o_done[G::TILES == 2 ? tile : step & 1]; };
    auto o_phase = [&](int step) { return (uint32_t)(G::TILES == 2 ? step & 1 : (step >> 1) & 1); };

    const Waits wait{p.err, &dead};
    Walk w;
    const bool any = w.begin(p.list, blockIdx.x);
    if (any && warp == G::WARPS) {
        // ---- loads.  The whole warp goes through the loop, as for the products.
        if (umma::elect_one()) {
            prefetch_tmap(&q_map);
            prefetch_tmap(&k_map);
            prefetch_tmap(&v_map);
        }
        int stage = 0, units = 0;
        uint32_t phase = 0;
        auto stage_done = [&] {
            if (++stage == G::STAGES) {
                stage = 0;
                phase ^= 1;
            }
        };
        // one loop: the keys of step n and the values of step n - 1, in the order of their products
        w.uniform();
        Walk x = w;   // the keys' walk
        int j = x.first, i = w.first;
        bool more = true;
        auto load_values = [&] {
#pragma unroll 1
            for (int c = 0; c < G::PER_STEP; ++c) {
                if (!wait.together(&bars.empty[stage], phase ^ 1)) return false;
                if (umma::elect_one()) {
                    mbar_expect_tx(&bars.full[stage], G::STAGE);
                    tma_load_4d(ring + stage * G::STAGE, &v_map, 0, w.u.b0 + i * kKeys + c * G::VK, 0, w.head, &bars.full[stage]);
                }
                stage_done();
            }
            ++i;
            return true;
        };
        for (int n = 0;; ++n) {
            if (G::TILES == 2 && n > 0 && !load_values()) goto loaded;
            if (more && j == x.last) {
                more = __any_sync(0xffffffffu, x.next());
                x.uniform();
                j = x.first;
            }
            if (more) {
                if (j == x.first) {
                    if (!wait.together(&bars.q_free, (units & 1) ^ 1)) goto loaded;
                    if (umma::elect_one()) {
                        mbar_expect_tx(&bars.q_full, G::TILES * D * 2 * p.tpt * p.G);
#pragma unroll 1
                        for (int c = 0; c < G::TILES * (D / 64); ++c)
                            tma_load_3d(smem + c * G::SUB, &q_map, c % (D / 64) * 64, x.head * p.G,
                                        x.u.a0 + c / (D / 64) * p.tpt, &bars.q_full);
                    }
                    ++units;
                }
#pragma unroll 1
                for (int c = 0; c < G::PER_STEP; ++c) {
                    if (!wait.together(&bars.empty[stage], phase ^ 1)) goto loaded;
                    if (umma::elect_one()) {
                        mbar_expect_tx(&bars.full[stage], G::STAGE);
                        tma_load_4d(ring + stage * G::STAGE, &k_map, 0, x.u.b0 + j * kKeys, c, x.head, &bars.full[stage]);
                    }
                    stage_done();
                }
                ++j;
            }
            if (G::TILES == 1 && n > 0 && !load_values()) goto loaded;
            if (n > 0 && i == w.last) {
                if (G::STAGED && w.whole()) {   // stages for the results, with the gates in them
                    if (!more) {   // (where the next unit's keys would be: the place of these is known without it)
                        bars.passed = stage;
                        for (int c = 0; c < G::PER_STEP; ++c) stage_done();
                    }
#pragma unroll 1
                    for (int c = 0; c < G::RESULTS; ++c) {
                        if (!wait.together(&bars.empty[stage], phase ^ 1)) goto loaded;
                        if (umma::elect_one()) {
                            if (p.gate.p != nullptr) {
                                mbar_expect_tx(&bars.full[stage], 128 * p.tpt * p.G);
                                tma_load_3d(ring + stage * G::STAGE, &gate_map, c % (D / 64) * 64, w.head * p.G,
                                            w.u.a0 + c / (D / 64) * p.tpt, &bars.full[stage]);
                            } else {
                                mbar_arrive(&bars.full[stage]);
                            }
                        }
                        stage_done();
                    }
                }
                if (!__any_sync(0xffffffffu, w.next())) break;
                w.uniform();
                i = w.first;
            }
        }
    loaded:
        bars.loaded = {stage, phase};
        bars.units = units;
    } else if (any && warp == G::WARPS + 1) {
        // ---- products.  The whole warp goes through the loop, so that operands stay uniform; one lane issues.
        const uint32_t base = __shfl_sync(0xffffffffu, tmem, 0);
        int stage = 0, units = 0, step = 0;
        uint32_t phase = 0;
        constexpr uint32_t id_s = umma::idesc(128, 128, umma::kFmtBF16);
        constexpr uint32_t id_o = umma::idesc(128, D, umma::kFmtBF16) | umma::kBTransposed;
        const uint64_t d_ring = umma::desc_sw128(smem_u32(ring)), d_q = umma::desc_sw128(smem_u32(smem));
        const uint64_t d_values = umma::desc_sw128_mn(smem_u32(ring), G::VK * 128);
        auto take = [&](int s, uint32_t ph) {
            wait(&bars.full[s], ph);
            umma::fence_after_sync();
        };
        auto commit = [&](uint64_t *bar) { umma::warp_mma_commit(bar); };
        auto pass = [&](int &s, uint32_t &ph) {
            if (++s == G::STAGES) {
                s = 0;
                ph ^= 1;
            }
        };
        // the scores of 64 channels, in stage s, of tile t into buffer buf
        auto scores = [&](int t, int buf, int c, int s) {
            const uint64_t a = d_q + (uint32_t)((t * G::QTILE + c * G::SUB) >> 4), b = d_ring + (uint32_t)(s * (G::STAGE >> 4));
            umma::warp_mma_bf16_k64(base + G::S_COL + buf * 128, a, b, id_s, c > 0);
        };
        // the product of VK of P's keys with their values, in stage s
        auto values = [&](int t, int buf, int c, int s, bool acc) {
            const uint64_t b = d_values + (uint32_t)(s * (G::STAGE >> 4));
#pragma unroll
            for (int k = 0; k < G::VK / 32; ++k)
                // (P of 64 keys lies over the first half of their scores)
                umma::warp_mma_bf16_tmem_a_k32(
                    base + t * D, base + G::S_COL + buf * 128 + (c * G::VK + k * 32) / 64 * 64 + (c * G::VK + k * 32) % 64 / 2,
                    b + k * (4096 >> 4), id_o, acc || c > 0 || k > 0);
        };
        // one loop: the scores of step n and the values of step n - 1.  One tile: the scores first, into the other buffer.
        // Two tiles: each tile's values, then its scores into the buffer that P has left.
        w.uniform();
        Walk x = w;
        int j = x.first, i = w.first, done = 0;   // done: tiles whose values are through
        bool more = true;
        for (int n = 0;; ++n) {
            const int s0 = stage;
            const uint32_t ph0 = phase;
            int sk = stage;             // the stages of the scores: first, or behind those of the values
            uint32_t pk = phase;
            if (G::TILES == 2 && n > 0)
                for (int c = 0; c < G::PER_STEP; ++c) pass(sk, pk);
            if (more && j == x.last) {
                more = __any_sync(0xffffffffu, x.next());
                x.uniform();
                j = x.first;
            }
            int sv = s0;                // ... of the values
            uint32_t pv = ph0;
            if (G::TILES == 1 && more)
                for (int c = 0; c < G::PER_STEP; ++c) pass(sv, pv);
            auto do_scores = [&](int t) {
                if (j == x.first && t == 0) wait(&bars.q_full, units++ & 1);
                const int buf = G::TILES == 1 ? n & 1 : t;
                int s = sk;
                uint32_t ph = pk;
#pragma unroll 1
                for (int c = 0; c < G::PER_STEP; ++c) {
                    if (t == 0) take(s, ph);
                    scores(t, buf, c, s);
                    if (t == G::TILES - 1) commit(&bars.empty[s]);
                    pass(s, ph);
                }
                commit(&bars.s_full[buf]);
                if (t == G::TILES - 1 && j + 1 == x.last) commit(&bars.q_free);
            };
#pragma unroll 1
            for (int t = 0; t < G::TILES; ++t) {
                if (G::TILES == 1 && more) do_scores(0);
                if (n > 0) {
                    const bool acc = i > w.first;
                    const int buf = G::TILES == 1 ? step & 1 : t;
                    wait(&bars.p_full[buf], o_phase(step));
                    if (!acc && done > 0) wait(&bars.o_free[t], (done - 1) & 1);
                    umma::fence_after_sync();
                    int s = sv;
                    uint32_t ph = pv;
#pragma unroll 1
                    for (int c = 0; c < G::PER_STEP; ++c) {
                        if (t == 0) take(s, ph);
                        values(t, buf, c, s, acc);
                        if (t == G::TILES - 1) commit(&bars.empty[s]);
                        pass(s, ph);
                    }
                    commit(o_done(t, step));
                }
                if (G::TILES == 2 && more) do_scores(t);
            }
            if (n > 0)
                for (int c = 0; c < G::PER_STEP; ++c) pass(stage, phase);
            if (more) {
                for (int c = 0; c < G::PER_STEP; ++c) pass(stage, phase);
                ++j;
            }
            if (n == 0) continue;
            ++step;
            if (++i == w.last) {
                ++done;
                if (G::STAGED && w.whole())
                    for (int c = 0; c < G::RESULTS; ++c) pass(stage, phase);
                if (!__any_sync(0xffffffffu, w.next())) break;
                w.uniform();
                i = w.first;
            }
        }
        // every product is through before the tensor memory goes back
        commit(&bars.end);
        wait_end(&bars.end, 0, p.err);
    } else if (any) {
        // ---- softmax and results.  Two warpgroups a tile, each with half of a step's keys and half of the channels.  One
        // tile: the scores stay in registers.  Two tiles, sixteen warps with 96 registers: they are read twice, for their
        // maximum and for the weights.
        constexpr bool TWICE = G::TILES == 2;
        constexpr int COLS = 64, DH = D / 2;
        const int tile = warp >> 3, half = (warp >> 2) & 1, r = (warp & 3) * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(warp & 3) << 21), o_at = lanes + tile * D + half * DH;
        uint8_t *turn = ring + G::STAGES * G::STAGE + warp * G::TURN;   // (if not STAGED)
        // who writes a stage of results: a warpgroup, or with 64 channels both of a tile
        constexpr bool SHARED = DH < 64;
        const bool leader = G::STAGED && (warp & 3) == 0 && lane == 0 && (!SHARED || half == 0);
        const int team = SHARED ? 1 + tile : 3 + tile * 2 + half, team_size = SHARED ? 256 : 128;
        const float f2 = p.scale2;
        int step = 0, wholes = 0;
        do {
            const RowOut o = row_out<D>(p, w.u, w.head, tile, r);
            const bool whole = w.whole(), gated = p.gate.p != nullptr && whole;
            float m = -INFINITY, l = 0.0f;   // m: of the scores in powers of two; l: of this half's keys
            if (!G::STAGED && gated && o.gate != nullptr)   // (on its way to L2 before it is needed)
                for (int d = half * DH; d < (half + 1) * DH; d += 64)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(o.gate + d));
            for (int i = w.first; i < w.last; ++i, ++step) {
                const int buf = G::TILES == 2 ? tile : step & 1;
                const uint32_t s_at = lanes + G::S_COL + buf * 128;
                wait(&bars.s_full[buf], G::TILES == 2 ? step & 1 : (step >> 1) & 1);
                umma::fence_after_sync();
                const int lim = o.keys - i * kKeys - half * 64;
                const bool masked = __any_sync(0xffffffffu, lim < COLS);
                auto scores_of = [&](float (&s)[32], int c) {   // (after the load)
                    if (masked) hide(s, lim - c * 32);
                };
                float s[TWICE ? 1 : 2][32], most;
                if (TWICE) {
                    umma::tmem_ld32(s_at + half * 64, s[0]);
                    umma::tmem_ld_wait();
                    scores_of(s[0], 0);
                    most = largest(s[0]);
                    umma::tmem_ld32(s_at + half * 64 + 32, s[0]);
                    umma::tmem_ld_wait();
                    scores_of(s[0], 1);
                    most = fmaxf(most, largest(s[0]));
                } else {
                    umma::tmem_ld32(s_at + half * 64, s[0]);
                    umma::tmem_ld32(s_at + half * 64 + 32, s[TWICE ? 0 : 1]);
                    umma::tmem_ld_wait();
                    scores_of(s[0], 0);
                    scores_of(s[TWICE ? 0 : 1], 1);
                    most = fmaxf(largest(s[0]), largest(s[TWICE ? 0 : 1]));
                }
                float *ex = bars.most[tile][step & 1][0];
                ex[half * 128 + r] = most;
                pair_sync(tile);
                most = fmaxf(ex[r], ex[128 + r]);
                most *= f2;
                const bool raise = most > m + kRaise;   // (m = -infinity: the first that is seen)
                if (__any_sync(0xffffffffu, raise)) {
                    const float m1 = raise ? most : m, f = raise ? (m == -INFINITY ? 0.0f : ex2(m - m1)) : 1.0f;
                    m = m1;
                    l *= f;
                    if (i > w.first) {
                        if (G::TILES == 1) {
                            wait(o_done(0, step - 1), o_phase(step - 1));   // (two tiles: their scores came after it)
                            umma::fence_after_sync();
                        }
#pragma unroll 1
                        for (int c = 0; c < DH / 32; ++c) {
                            float x[32];
                            umma::tmem_ld32(o_at + c * 32, x);
                            umma::tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k) x[k] *= f;
                            umma::tmem_st32(o_at + c * 32, x);
                        }
                    }
                }
                const float base = m == -INFINITY ? 0.0f : -m;
                const F2 mul = f2_of(f2, f2), add = f2_of(base, base);
                F2 sum[2] = {f2_of(0.0f, 0.0f), f2_of(0.0f, 0.0f)};
                if (TWICE) {
                    float pk[16];
                    // (the second half is still there, first: P of the first lies over its own scores only)
                    weights(s[0], mul, add, sum[1], pk);
                    umma::tmem_ld32(s_at + half * 64, s[0]);
                    umma::tmem_ld_wait();
                    umma::tmem_st16(s_at + half * 64 + 16, pk);
                    scores_of(s[0], 0);
                    weights(s[0], mul, add, sum[0], pk);
                    umma::tmem_st16(s_at + half * 64, pk);
                } else {
                    float pk[32];
                    weights(s[0], mul, add, sum[0], pk);
                    weights(s[TWICE ? 0 : 1], mul, add, sum[1], pk + 16);
                    umma::tmem_st32(s_at + half * 64, pk);
                }
                const float2 t = parts(add2(sum[0], sum[1]));
                l += t.x + t.y;
                umma::tmem_st_wait();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars.p_full[buf]);
            }
            // the unit's results
            const int slot = w.slot(blockIdx.x);
            bool bad = false;
            bars.sum[tile][half][r] = l;
            pair_sync(tile);
            l = bars.sum[tile][0][r] + bars.sum[tile][1][r];
            const float f = 1.0f / l;
            // the first of the tile's result stages, as the loading warp counts: behind all steps' keys and values, the next
            // unit's first keys and the results before
            const int at0 = (2 * step + 1) * G::PER_STEP + wholes * G::RESULTS + tile * (D / 64);
            RowsOut rows;
            Gates gates[2];   // asked for two groups ahead
            if (!G::STAGED) {
                rows = rows_out<D>(p, o);
                if (gated)
#pragma unroll
                    for (int z = 0; z < 2; ++z) gates[z] = ask_gates(rows, half * DH + z * 32);
            }
            wait(o_done(tile, step - 1), o_phase(step - 1));
            umma::fence_after_sync();
            // (not unrolled: the code would be fetched anew for every tile)
#pragma unroll 1
            for (int c = 0; c < DH / 32; ++c) {
                const int d = half * DH + c * 32;
                float x[32];
                umma::tmem_ld32(o_at + c * 32, x);
                umma::tmem_ld_wait();
                if (c == DH / 32 - 1) {
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars.o_free[tile]);
                }
                if (whole && !G::STAGED) {
                    bad |= scaled(x, f);
                    const Gates now = gates[0];
                    gates[0] = gates[1];
                    if (gated && c + 2 < DH / 32) gates[1] = ask_gates(rows, d + 64);
                    write_group(turn, rows, o.keys == 0, gated, now, d, x);
                } else if (whole) {
                    const int at = at0 + d / 64;
                    // (the stage's last use is over: it was two steps' products back, or this tile's results)
                    wait(&bars.full[at % G::STAGES], (at / G::STAGES) & 1);
                    bad |= scaled(x, f);
                    put_group(ring + at % G::STAGES * G::STAGE, r, d % 64 * 2, o.keys == 0, gated, x);
                } else {
                    float4 *dst = reinterpret_cast<float4 *>(p.part_o) +
                                  ((size_t)slot * (D / 4) + d / 4) * (G::TILES * 128) + tile * 128 + r;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        dst[(size_t)k * (G::TILES * 128)] =
                            make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
                }
            }
            if (whole) {
                if (half == 0 && p.lse != nullptr && o.mine) p.lse[o.at] = o.keys > 0 ? (m + lg2(l)) * kLn2 : -INFINITY;
                if (bad && o.keys > 0) again = 1;
                if (G::STAGED) {
                    const bool complete = (tile + 1) * p.tpt <= w.u.slot_a;   // all rows are the sequence's
                    if (!complete) {
                        __syncwarp();
#pragma unroll 1
                        for (int i = lane; i < 32 * DH / 8; i += 32) {
                            const int rr = (warp & 3) * 32 + i / (DH / 8), d = half * DH + i % (DH / 8) * 8;
                            const RowOut to = row_out<D>(p, w.u, w.head, tile, rr);
                            if (to.mine)
                                *reinterpret_cast<uint4 *>(p.out + to.at * D + d) = *reinterpret_cast<const uint4 *>(
                                    ring + (at0 + d / 64) % G::STAGES * G::STAGE + umma::sw128(rr, d % 64 * 2));
                        }
                    }
                    fence_proxy_async_smem();
                    team_sync(team, team_size);
                    if (leader) {
                        constexpr int N = SHARED ? 1 : DH / 64;
                        const int at = at0 + (SHARED ? 0 : half * N);
                        if (complete) {
                            for (int c = 0; c < N; ++c)
                                tma_store_3d(&out_map, (SHARED ? 0 : half * DH) + c * 64, w.head * p.G, w.u.a0 + tile * p.tpt,
                                             ring + (at + c) % G::STAGES * G::STAGE);
                            bulk_commit();
                            bulk_wait_read();
                        }
                        for (int c = 0; c < N; ++c) mbar_arrive(&bars.empty[(at + c) % G::STAGES]);
                    }
                    __syncwarp();
                    ++wholes;
                }
            } else if (half == 0) {
                p.part_ml[(size_t)slot * (G::TILES * 128) + tile * 128 + r] = make_float2(m, l);
            }
            // (the halves start the next tile together: without it chunks over long prefixes take 126 us, with it 118)
            if (G::TILES == 1) pair_sync(tile);
        } while (w.next());
        if (leader) bulk_wait_all();
        umma::fence_before_sync();
    }
    __syncthreads();
    umma::fence_after_sync();
    if (dead && threadIdx.x == 0) {
        for (int i = 0; i < G::STAGES; ++i) {
            const bool passed = bars.passed >= 0 && (i + G::STAGES - bars.passed) % G::STAGES < G::PER_STEP;
            wait_end(&bars.full[i], bars.loaded.parity(i) ^ (uint32_t)passed, p.err);
        }
        wait_end(&bars.q_full, (bars.units & 1) ^ 1, p.err);
    }
    if (warp == 0) umma::tmem_dealloc(tmem, 512);
    if (again && !dead) rows_again<D>(p);
}

// Every row by the definition: for scales that are not positive, whose scores'
// order the passes above would have to turn round.
template <int D>
__global__ void __launch_bounds__(256) prompt_rows_kernel(const Params p) {
    attn::grid_dep_enter();
    const Header h = *p.list.header;
    const int lane = threadIdx.x & 31;
    const long long rows = (long long)Geo<D>::TILES * 128, all = rows * h.units * p.Hkv;
    for (long long x = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); x < all; x += (long long)gridDim.x * 8) {
        const int head = (int)(x / (rows * h.units)), r = (int)(x % rows);
        const Unit u = p.list.unit[x / rows % h.units];
        const RowOut o = row_out<D>(p, u, head, r / 128, r % 128);
        if (!o.mine) continue;
        float lse = -INFINITY;
        if (o.keys > 0) {
            const long long n = o.at / p.Hq;
            const int hq = (int)(o.at - n * p.Hq);
            lse = exact_row<D>(p.q.p + n * p.q.ts + hq * p.q.hs, p.k.p + u.b0 * p.k.ts + head * p.k.hs, p.k.ts,
                               p.v.p + u.b0 * p.v.ts + head * p.v.hs, p.v.ts, o.keys, p.scale, o.gate, p.out + o.at * D, 0, D, true);
        } else {
            for (int d = lane; d < D; d += 32) p.out[o.at * D + d] = 0;
        }
        if (lane == 0 && p.lse != nullptr) p.lse[o.at] = lse;
    }
}

// A split unit's parts joined: 32 channels of 128 rows a block.
template <int D>
__global__ void __launch_bounds__(128) prompt_join_kernel(const Params p) {
    constexpr int ROWS = Geo<D>::TILES * 128;
    __shared__ __align__(16) uint8_t turn[4][Geo<D>::TURN];
    attn::grid_dep_enter();
    const Parts part = parts_from(p.list, blockIdx.x);
    if (part.n == 0) return;
    const int tile = blockIdx.y / (D / 32), c = blockIdx.y % (D / 32), r = threadIdx.x, row = tile * 128 + r;
    const RowOut o = row_out<D>(p, part.u, part.head, tile, r);
    const RowsOut rows = rows_out<D>(p, o);
    const Gates gates = ask_gates(rows, c * 32);
    float m = -INFINITY, l = 0.0f, x[32];
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = 0.0f;
    for (int i = 0; i < part.n; ++i) {
        const size_t slot = 2 * (size_t)(blockIdx.x + i) + (i == 0 ? 1 : 0);
        const float2 ml = p.part_ml[slot * ROWS + row];
        const float4 *src = reinterpret_cast<const float4 *>(p.part_o) + (slot * (D / 4) + c * 8) * ROWS + row;
        const float top = fmaxf(m, ml.x), f = m == top ? 1.0f : ex2(m - top), g = ml.x == top ? 1.0f : ex2(ml.x - top);
        m = top;
        l = l * f + ml.y * g;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const float4 v = src[(size_t)k * ROWS];
            x[4 * k] = x[4 * k] * f + v.x * g;
            x[4 * k + 1] = x[4 * k + 1] * f + v.y * g;
            x[4 * k + 2] = x[4 * k + 2] * f + v.z * g;
            x[4 * k + 3] = x[4 * k + 3] * f + v.w * g;
        }
    }
    const float f = 1.0f / l;
    const bool bad = scaled(x, f);
    write_group(turn[threadIdx.x >> 5], rows, o.keys == 0, p.gate.p != nullptr, gates, c * 32, x);
    if (c == 0 && p.lse != nullptr && o.mine) p.lse[o.at] = o.keys > 0 ? (m + lg2(l)) * kLn2 : -INFINITY;
    mend_rows<D>(p, o, part.u, part.head, bad, c * 32, c * 32 + 32);
}

int tiles_of(int D) { return D <= 128 ? 2 : 1; }

PromptList list_of(const PromptSizes &s) {
    const int tpt = 128 / (s.Hq / s.Hkv);
    // A tile's start and end in steps (T = 8192, 256 channels: 2 481 us, 4 380, 6 351, 8 355; packed, 128 channels: 2 445,
    // 4 460, 6 468: with two tiles one's end runs beside the other's steps).
    return PromptList{false, tpt * tiles_of(s.D), kKeys, num_sms(), 4, s.D == 256 ? 6 : 2, 4};
}

struct Workspace {
    size_t o, ml, total;
};

Workspace workspace(const PromptSizes &s) {
    Workspace w;
    const size_t rows = 2 * (size_t)num_sms() * tiles_of(s.D) * 128;
    w.o = prompt_list_bytes(s, list_of(s));
    w.ml = w.o + up256(rows * s.D * sizeof(float));
    w.total = w.ml + up256(rows * sizeof(float2));
    return w;
}

template <int D>
cudaError_t launch_d(const PromptSizes &s, Params &p, bool splits, cudaStream_t st) {
    using G = Geo<D>;
    if (!(p.scale > 0.0f)) return DependentLaunch(dim3(8 * num_sms()), dim3(256), 0, st)(prompt_rows_kernel<D>, p);
    static unsigned long long done = 0;
    cudaError_t e = set_max_smem(done, prompt_forward_kernel<D>, G::SMEM);
    if (e != cudaSuccess) return e;
    CUtensorMap q, k, v, gate, out;
    // (no keys: nothing of what is loaded counts, but a map needs a tensor)
    const bool none = s.Nk == 0;
    const HeadsIn dummy{p.q.p, 0, 0};
    const HeadsIn results{p.out, (long long)s.Hq * D, D};
    if (!queries_map(&q, p.q, s.Nq, s.Hq, D, p.G, p.tpt) ||
        (G::STAGED && !queries_map(&out, results, s.Nq, s.Hq, D, p.G, p.tpt)) ||
        (G::STAGED && p.gate.p != nullptr && !queries_map(&gate, p.gate, s.Nq, s.Hq, D, p.G, p.tpt)) ||
        !keys_map(&k, none ? dummy : p.k, none ? 1 : s.Nk, none ? 1 : s.Hkv, D, kKeys, 1) ||
        !keys_map(&v, none ? dummy : p.v, none ? 1 : s.Nk, none ? 1 : s.Hkv, D, G::VK, D / 64))
        return cudaErrorInvalidValue;
    if (!G::STAGED) out = q;   // (not used)
    if (!G::STAGED || p.gate.p == nullptr) gate = q;
    const int ctas = num_sms();
    e = DependentLaunch(dim3(ctas), dim3(G::THREADS), G::SMEM, st)(prompt_forward_kernel<D>, q, k, v, gate, out, p);
    if (e != cudaSuccess || !splits) return e;
    return DependentLaunch(dim3(ctas - 1, G::TILES * (D / 32)), dim3(128), 0, st)(prompt_join_kernel<D>, p);
}

}  // namespace

size_t attn_prefill_workspace(const PromptSizes &s) { return workspace(s).total; }

cudaError_t launch_attn_prefill(const PromptSizes &s, const HeadsIn &q, const HeadsIn &k, const HeadsIn &v,
                                const PromptSeqs &seqs, const HeadsIn &gate, float scale, uint16_t *out, float *lse,
                                void *ws, unsigned *err, cudaStream_t st) {
    const PromptList list = list_of(s);
    const Workspace w = workspace(s);
    char *base = static_cast<char *>(ws);
    cudaError_t e = launch_prompt_plan(s, seqs, &list, 1, &ws, err, st);
    if (e != cudaSuccess) return e;
    Params p = {};
    p.list = prompt_list_at(s, list, ws);
    p.q = q;
    p.k = k;
    p.v = v;
    p.gate = gate;
    p.out = out;
    p.lse = lse;
    p.part_o = reinterpret_cast<float *>(base + w.o);
    p.part_ml = reinterpret_cast<float2 *>(base + w.ml);
    p.err = err;
    p.Hq = s.Hq;
    p.Hkv = s.Hkv;
    p.G = s.Hq / s.Hkv;
    p.tpt = 128 / p.G;
    p.scale = scale;
    p.scale2 = scale * kLog2e;
    const bool splits = prompt_splits(s, seqs, list);
    if (s.D == 64) return launch_d<64>(s, p, splits, st);
    if (s.D == 128) return launch_d<128>(s, p, splits, st);
    return launch_d<256>(s, p, splits, st);
}

}  // namespace gdn
