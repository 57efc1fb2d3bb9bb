// The work lists of a prompt's attention (prompt_fwd.cu, prompt_bwd.cu), made
// by one small kernel from the sequences' offsets (prompt_plan.cu), and the
// walk over them.
//
// A unit is a tile of one sequence's tokens (queries: the G heads of a key head
// are rows of one tile, row t * G + g, so that keys are read once for all of
// them; or 128 keys) with the tokens of the other kind that it has to meet, in
// steps of a fixed number.  The units of all sequences, once for each key head,
// are one list of steps, each unit with a few blank ones before its own, which
// stand for the time that its start and end take; every CTA takes an equal
// share of the list.  A unit whose steps cross shares leaves partial results,
// which a second kernel joins in order.
#pragma once

#include "attn.cuh"

namespace gdn {
namespace prompt {

struct __align__(16) Unit {
    int a0, n_a, slot_a;   // first token of the tile (in the buffer); valid ones; with those that are padding
    int b0, n_b;           // first token of the other kind (in the buffer), their number
    int lim0;              // queries: keys that the first token sees.  keys: key j of the tile is seen by token i of
                           // the b's if j <= lim0 + i
    int steps, pad;
    long long pre;         // steps of the units before, blank ones among them
    long long pad2;
};

struct __align__(16) Start {   // a CTA's share
    int head, unit;
    long long offset;      // where it begins: steps into the unit, blank ones first
    long long left;        // its steps
    int units, blank;      // of the list: units of a key head, blank steps of a unit
    Unit u;                // the first unit
};

struct Header {
    long long steps;       // of one key head
    long long share;       // of a CTA (but for lists whose tiles are not split)
    int units, blank;
    long long pad;
};

// One list in the workspace: header, shares (CTAs), units.
struct List {
    Header *header;
    Start *start;
    Unit *unit;
};

struct Sequences {
    int B;
    long long Nq, Nk;            // rows of the buffers
    const int32_t *cu_q, *cu_k;  // [B + 1], or null: equal slots
    const int32_t *n_q, *n_k;    // [B] or null
};

struct Seq {
    int q0, slot_q, nq, k0, slot_k, nk;
    bool ok;
};

__device__ __forceinline__ Seq load_seq(const Sequences &p, int s) {
    Seq r;
    const long long sq = p.Nq / p.B, sk = p.Nk / p.B;
    const long long q0 = p.cu_q ? p.cu_q[s] : s * sq, q1 = p.cu_q ? p.cu_q[s + 1] : q0 + sq;
    const long long k0 = p.cu_k ? p.cu_k[s] : s * sk, k1 = p.cu_k ? p.cu_k[s + 1] : k0 + sk;
    r.ok = q0 >= 0 && q1 >= q0 && q1 <= p.Nq && k0 >= 0 && k1 >= k0 && k1 <= p.Nk;
    r.q0 = (int)q0;
    r.k0 = (int)k0;
    r.slot_q = (int)(q1 - q0);
    r.slot_k = (int)(k1 - k0);
    r.nq = p.n_q ? min(max(p.n_q[s], 0), r.slot_q) : r.slot_q;
    r.nk = p.n_k ? min(max(p.n_k[s], 0), r.slot_k) : r.slot_k;
    return r;
}

// A CTA's way through its share.
struct Walk {
    const Unit *units;
    int n_units, blank;
    long long left;        // steps of the share after the current unit's
    int head, unit, first, last;   // the current unit's steps first .. last - 1
    Unit u;
    int4 ahead[2];         // the next unit, asked for early

    // the unit's steps from `at` (blank ones counted); units of which the share holds only blank steps are passed over
    __device__ __forceinline__ bool open(long long at) {
        while (left > 0) {
            const int4 x = ahead[0], y = ahead[1];
            ask(unit + 1 == n_units ? 0 : unit + 1);
            u.a0 = x.x;
            u.n_a = x.y;
            u.slot_a = x.z;
            u.b0 = x.w;
            u.n_b = y.x;
            u.lim0 = y.y;
            u.steps = y.z;
            const long long whole = (long long)u.steps + blank - at, n = whole < left ? whole : left;
            first = at > blank ? (int)(at - blank) : 0;
            last = at + n > blank ? (int)(at + n - blank) : 0;
            left -= n;
            if (last > first) return true;
            advance();
            at = 0;
        }
        return false;
    }
    __device__ __forceinline__ void ask(int i) {
        const int4 *p = reinterpret_cast<const int4 *>(units + i);
        ahead[0] = p[0];
        ahead[1] = p[1];
    }
    __device__ __forceinline__ void advance() {
        if (++unit == n_units) {
            unit = 0;
            ++head;
        }
    }
    __device__ __forceinline__ bool begin(const List &l, int cta) {
        const Start *s = l.start + cta;
        const int4 *p = reinterpret_cast<const int4 *>(s);
        const int4 a = p[0], b = p[1];
        ahead[0] = p[2];
        ahead[1] = p[3];
        left = ((long long)(uint32_t)b.x) | ((long long)b.y << 32);
        units = l.unit;
        n_units = b.z;
        blank = b.w;
        head = a.x;
        unit = a.y;
        return left > 0 && open(((long long)(uint32_t)a.z) | ((long long)a.w << 32));
    }
    // the same values in every lane, and known to be (for loops of a whole warp)
    __device__ __forceinline__ void uniform() {
        first = __shfl_sync(0xffffffffu, first, 0);
        last = __shfl_sync(0xffffffffu, last, 0);
        head = __shfl_sync(0xffffffffu, head, 0);
        u.a0 = __shfl_sync(0xffffffffu, u.a0, 0);
        u.b0 = __shfl_sync(0xffffffffu, u.b0, 0);
    }
    __device__ __forceinline__ bool next() {
        advance();
        return open(0);
    }
    __device__ __forceinline__ bool whole() const { return first == 0 && last == u.steps; }
    // the partial results' slot of a unit that is not whole: of the two of a CTA, the second for one that begins here
    __device__ __forceinline__ int slot(int cta) const { return 2 * cta + (first == 0 ? 1 : 0); }
};

// The parts of the unit, split over shares, that begins in CTA `cta`'s: how
// many (0: none does), in the slots 2 cta + 1, 2 (cta + 1), 2 (cta + 2), ...
struct Parts {
    int n, head;
    Unit u;
};

__device__ __forceinline__ Parts parts_from(const List &l, int cta) {
    Parts r;
    r.n = 0;
    const Header h = *l.header;
    const Start s = l.start[cta + 1];
    const long long mine = s.offset - h.blank;   // steps of the unit that the next CTA goes on with, before it
    if (s.left <= 0 || mine <= 0) return r;
    const long long x1 = h.share * (cta + 1);
    if (mine > h.share) return r;                // (it began before this share)
    r.u = s.u;
    r.head = s.head;
    const long long end = x1 - s.offset + h.blank + r.u.steps;
    r.n = (int)((end - 1) / h.share) - cta + 1;
    return r;
}

__device__ __forceinline__ float lg2(float x) {   // (off by less than 2^-22)
    float r;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Waits of a CTA's roles: after one that gave up, none waits any more (`dead`,
// in shared memory).  False: not there.  The loop is out of line: it would be
// in the code some twenty times, and a tile's start and end run through code
// that has to be fetched anew.
__device__ __noinline__ inline bool wait_long(uint64_t *bar, uint32_t parity, unsigned *err, volatile int *dead) {
    for (uint32_t i = 0; i < kSpinLimit; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if (*dead) return false;
    }
    atomicOr(err, kErrMbarTimeout);
    *dead = 1;
    return false;
}

struct Waits {
    unsigned *err;
    volatile int *dead;
    __device__ __forceinline__ bool operator()(uint64_t *bar, uint32_t parity) const {
        return mbar_try_wait(bar, parity) || mbar_try_wait(bar, parity) || wait_long(bar, parity, err, dead);
    }
    // The same answer in all lanes of the warp: when waits give up, one lane may still find the phase complete and another
    // not, and an election, which names all lanes, has to be reached by all.
    __device__ __forceinline__ bool together(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xffffffffu, (*this)(bar, parity));
    }
};

// Waits for a copy or products that are under way, whether or not a wait has given up (`dead` says that nobody is to wait
// for what may never be issued; what was issued ends, in microseconds).
__device__ __noinline__ inline void wait_end(uint64_t *bar, uint32_t parity, unsigned *err) {
    for (uint32_t i = 0; i < kSpinLimit / 16; ++i)
        if (mbar_try_wait(bar, parity)) return;
    atomicOr(err, kErrMbarTimeout);
}

// Where the loading warp ended in a ring: the next stage to be filled, and its phase.  It ends where a wait gives up; a CTA
// in which one did waits for the last copy of each stage before it ends.  (No account of single copies: what is added to
// the loop costs.  A prompt of 8192 tokens, 256 channels: 385 us; with a note of each copy 424, a flag beside each wait 478.)
struct Loaded {
    int stage;
    uint32_t phase;
    // (a stage that was not reached in this phase: the copy before; before the first one the phase of parity 1 counts as over)
    __device__ __forceinline__ uint32_t parity(int i) const { return i < stage ? phase : phase ^ 1; }
};

constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Two f32 in one register pair.
struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2_of(float a, float b) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 parts(F2 x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x.v));
    return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
    F2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
    return r;
}
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}

// A row of D bf16 in a warp, D / 32 channels a lane.
template <int D>
__device__ __forceinline__ void lane_row(const uint16_t *p, float (&x)[D / 32]) {
    constexpr int N = D / 32;
    const uint16_t *q = p + (threadIdx.x & 31) * N;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint32_t w = reinterpret_cast<const uint32_t *>(q)[i];
        x[2 * i] = __uint_as_float(w << 16);
        x[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
    }
}

template <int D>
__device__ __forceinline__ float row_dot(const float (&a)[D / 32], const float (&b)[D / 32]) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) t = fmaf(a[i], b[i], t);
    return warp_sum(t);
}

// Every channel of the row is NaN (and stays so: no more keys have to be read).
template <int N>
__device__ __forceinline__ bool all_nan(const float (&x)[N]) {
    bool nan = true;
#pragma unroll
    for (int i = 0; i < N; ++i) nan = nan && x[i] != x[i];
    return __all_sync(0xffffffffu, nan);
}

// Whether a row in memory is finite.
template <int D>
__device__ __forceinline__ bool finite_row(const uint16_t *p) {
    float x[D / 32], check = 0.0f;
    lane_row<D>(p, x);
#pragma unroll
    for (int i = 0; i < D / 32; ++i) check = fmaf(x[i], 0.0f, check);   // (0 times an infinity or NaN)
    return __all_sync(0xffffffffu, check == 0.0f);
}

// x *= f; returns whether one of them is not finite.
__device__ __forceinline__ bool scaled(float (&x)[32], float f) {
    float check = 0.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) {
        x[k] *= f;
        check = fmaf(x[k], 0.0f, check);   // (0 times an infinity or NaN)
    }
    return check != 0.0f;
}

// Byte offset of 16 bytes (chunk 0 or 1) of a row in a warp's 32 x 32 bytes: no
// two of the eight lanes of a phase, by rows or by chunks, meet in a bank.
__device__ __forceinline__ int turn_at(int row, int chunk) { return row * 32 + ((chunk ^ ((row >> 2) & 1)) << 4); }

inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }

inline long long head_stride(const HeadsIn &x, int H, int D) { return H > 1 ? x.hs : D; }
inline long long token_stride(const HeadsIn &x, long long rows, int H, int D) { return rows > 1 ? x.ts : (long long)H * D; }

// [rows, H, D] as (64 channels, heads, tokens): boxes of one tile's rows.
inline bool queries_map(CUtensorMap *map, const HeadsIn &x, long long rows, int H, int D, int box_heads, int box_tokens) {
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)H, (uint64_t)rows};
    const uint64_t strides[2] = {(uint64_t)head_stride(x, H, D) * 2, (uint64_t)token_stride(x, rows, H, D) * 2};
    const uint32_t box[3] = {64, (uint32_t)box_heads, (uint32_t)box_tokens};
    return encode_tmap_strided(map, x.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

// ... as (64 channels, tokens, groups of 64 channels, heads): boxes of one head's tokens, groups one after the other.
inline bool keys_map(CUtensorMap *map, const HeadsIn &x, long long rows, int H, int D, int box_tokens, int box_groups) {
    const uint64_t dims[4] = {64, (uint64_t)rows, (uint64_t)(D / 64), (uint64_t)H};
    const uint64_t strides[3] = {(uint64_t)token_stride(x, rows, H, D) * 2, 128, (uint64_t)head_stride(x, H, D) * 2};
    const uint32_t box[4] = {64, (uint32_t)box_tokens, (uint32_t)box_groups, 1};
    return encode_tmap_strided(map, x.p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

}  // namespace prompt
}  // namespace gdn
