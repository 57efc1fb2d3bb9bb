// The work lists of a prompt's attention (prompt_fwd.cu, prompt_bwd.cu), made
// by one small kernel from the sequences' offsets (prompt_plan.cu), and the
// walk over them.
//
// A unit is a tile of one sequence's tokens (queries: the G heads of a key head
// are rows of one tile, row t * G + g, so that keys are read once for all of
// them; or 128 keys) with the tokens of the other kind that it has to meet, in
// steps of a fixed number.  The units of all sequences, once for each key head,
// are one list of steps; every CTA takes an equal share of it.  A unit that
// crosses shares leaves partial results, which a second kernel joins in order.
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
    long long pre;         // steps of the units before
    long long pad2;
};

struct Start {             // where a CTA's share begins
    int head, unit;
    long long offset;      // steps into the unit
};

struct Header {
    long long steps;       // of one key head
    long long share;       // of a CTA
    int units, pad;
    long long pad2;
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
    int n_units, heads;
    long long left;        // steps of the share after the current unit's
    int head, unit, first, last;   // the current unit's steps first .. last - 1
    Unit u;

    __device__ __forceinline__ bool open(int at) {
        if (left <= 0) return false;
        const int4 *p = reinterpret_cast<const int4 *>(units + unit);
        const int4 x = p[0], y = p[1];
        u.a0 = x.x;
        u.n_a = x.y;
        u.slot_a = x.z;
        u.b0 = x.w;
        u.n_b = y.x;
        u.lim0 = y.y;
        u.steps = y.z;
        first = at;
        last = (long long)(u.steps - at) <= left ? u.steps : at + (int)left;
        left -= last - first;
        return true;
    }
    __device__ __forceinline__ bool begin(const List &l, int cta, int heads_) {
        const Header h = *l.header;
        const long long total = h.steps * heads_, x = h.share * cta;
        left = total - x < h.share ? total - x : h.share;
        if (left <= 0) return false;
        units = l.unit;
        n_units = h.units;
        heads = heads_;
        const Start s = l.start[cta];
        head = s.head;
        unit = s.unit;
        return open((int)s.offset);
    }
    __device__ __forceinline__ bool next() {
        if (++unit == n_units) {
            unit = 0;
            ++head;
        }
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

__device__ __forceinline__ Parts parts_from(const List &l, int cta, int ctas, int heads) {
    Parts r;
    r.n = 0;
    const Header h = *l.header;
    const long long total = h.steps * heads, x1 = h.share * (cta + 1);
    if (cta + 1 >= ctas || x1 >= total) return r;
    const Start s = l.start[cta + 1];
    if (s.offset == 0 || s.offset > h.share) return r;   // (begins there, or before this share)
    r.u = l.unit[s.unit];
    r.head = s.head;
    const long long end = x1 - s.offset + r.u.steps;
    r.n = (int)((end - 1) / h.share) - cta + 1;
    return r;
}

}  // namespace prompt
}  // namespace gdn
