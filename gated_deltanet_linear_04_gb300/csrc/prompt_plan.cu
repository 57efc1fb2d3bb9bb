// The work lists of a prompt's attention: one CTA a list.  Three passes, each
// a scan over the block: sequences to their first unit, units to their first
// step, shares to where they begin.  Latency-bound (one sequence of 8192
// tokens, 512 units: a few us, hidden behind the launch of the kernel that
// reads it as far as that goes).
#include "prompt.cuh"

namespace gdn {
namespace {

using namespace prompt;

constexpr int kThreads = 1024, kCached = 2048, kSeqs = 1024;

struct ListParams {
    Header *header;
    Start *start;
    Unit *unit;
    int *seq_first;    // [B + 1]: a sequence's first unit
    int keys;          // tiles of keys, steps of queries; or the other way round
    int tile, step;    // tokens
    int ctas, heads, least, blank;   // least: steps of a share
    int whole;         // no tile is split
};

struct PlanParams {
    Sequences s;
    ListParams l[2];
    unsigned *err;
};

template <typename T>
__device__ T block_scan(T v, T *sums, T &total) {   // exclusive
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    T x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();   // (the last call's readers)
    if (lane == 31) sums[warp] = x;
    __syncthreads();
    if (warp == 0) {
        T y = sums[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const T z = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) y += z;
        }
        sums[lane] = y;
    }
    __syncthreads();
    total = sums[31];
    return x - v + (warp > 0 ? sums[warp - 1] : (T)0);
}

// The largest i in [0, n) with a[i] <= x; a[0] <= x.
template <typename T>
__device__ int last_not_above(const T *a, int n, T x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

__device__ Unit make_unit(const Seq &q, int i, const ListParams &l) {
    Unit u = {};
    const int off = q.nk - q.nq;   // token t sees off + t + 1 keys
    if (!l.keys) {
        const int t0 = i * l.tile;
        u.a0 = q.q0 + t0;
        u.slot_a = min(l.tile, q.slot_q - t0);
        u.n_a = min(max(q.nq - t0, 0), l.tile);
        u.b0 = q.k0;
        u.lim0 = off + t0 + 1;
        u.n_b = u.n_a > 0 ? max(off + t0 + u.n_a, 0) : 0;
    } else {
        const int j0 = i * l.tile, t0 = max(j0 - off, 0);
        u.a0 = q.k0 + j0;
        u.slot_a = min(l.tile, q.slot_k - j0);
        u.n_a = min(max(q.nk - j0, 0), l.tile);
        u.n_b = u.n_a > 0 ? max(q.nq - t0, 0) : 0;
        u.b0 = q.q0 + (u.n_b > 0 ? t0 : 0);
        u.lim0 = off + t0 - j0;
    }
    u.steps = max(1, (int)(((long long)u.n_b + l.step - 1) / l.step));
    return u;
}

__global__ void __launch_bounds__(kThreads) prompt_plan_kernel(const PlanParams p) {
    __shared__ long long sums[32];
    __shared__ long long cached[kCached];
    __shared__ int first_cached[kCached];
    __shared__ Seq seqs[kSeqs];
    __shared__ int bad;
    const ListParams &l = p.l[blockIdx.x];
    const int tid = threadIdx.x, B = p.s.B;
    if (tid == 0) bad = 0;
    grid_dep_wait();
    grid_dep_launch();
    __syncthreads();
    long long units = 0, total = 0;
    bool ok = true;
    for (int base = 0; base < B; base += kThreads) {
        const int s = base + tid;
        long long n = 0;
        if (s < B) {
            const Seq q = load_seq(p.s, s);
            if (s < kSeqs) seqs[s] = q;
            ok = ok && q.ok;
            if (q.ok) n = ((l.keys ? q.slot_k : q.slot_q) + (long long)l.tile - 1) / l.tile;
        }
        long long sum;
        const long long at = units + block_scan(n, sums, sum);
        if (s < B) {
            l.seq_first[s] = (int)at;
            if (s < kCached) first_cached[s] = (int)at;
        }
        units += sum;
    }
    if (!ok) bad = 1;
    __syncthreads();
    if (bad) {   // (nothing is done, and the error word says why)
        units = 0;
        if (tid == 0) atomicOr(p.err, kErrBadOffsets);
    }
    for (long long base = 0; base < units; base += kThreads) {
        const long long u = base + tid;
        Unit unit = {};
        if (u < units) {
            const int s = B <= kCached ? last_not_above(first_cached, B, (int)u) : last_not_above(l.seq_first, B, (int)u);
            unit = make_unit(s < kSeqs ? seqs[s] : load_seq(p.s, s), (int)u - (B <= kCached ? first_cached[s] : l.seq_first[s]), l);
        }
        long long sum;
        unit.pre = total + block_scan(u < units ? (long long)unit.steps + l.blank : 0, sums, sum);
        if (u < units) {
            l.unit[u] = unit;
            if (u < kCached) cached[u] = unit.pre;
        }
        total += sum;
    }
    __syncthreads();
    const long long all = total * l.heads;
    long long share = (all + l.ctas - 1) / l.ctas;
    if (!l.whole && share < l.least) share = l.least;
    if (tid == 0) *l.header = Header{total, share, (int)units, l.blank, 0};
    // where a share begins; if no tile is to be split, at the tile's end that is nearer
    auto begin = [&](int c, Start &s) -> long long {
        const long long x = share * c;
        s = Start{};
        s.units = (int)units;
        s.blank = l.blank;
        if (x >= all) return all;
        s.head = (int)(x / total);
        const long long r = x - s.head * total;
        if (units <= kCached) {
            s.unit = last_not_above(cached, (int)units, r);
        } else {
            int lo = 0, hi = (int)units;
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (l.unit[mid].pre <= r)
                    lo = mid;
                else
                    hi = mid;
            }
            s.unit = lo;
        }
        s.u = l.unit[s.unit];
        s.offset = r - s.u.pre;
        if (s.offset == 0 || !l.whole) return x;
        const long long rest = s.u.steps + l.blank - s.offset;
        if (s.offset <= rest) {
            const long long back = s.offset;
            s.offset = 0;
            return x - back;
        }
        if (x + rest >= all) return all;
        if (++s.unit == units) {
            s.unit = 0;
            ++s.head;
        }
        s.u = l.unit[s.unit];
        s.offset = 0;
        return x + rest;
    };
    for (int c = tid; c < l.ctas; c += kThreads) {
        Start s, next;
        const long long x = begin(c, s);
        s.left = begin(c + 1, next) - x;
        l.start[c] = s;
    }
}

}  // namespace

using prompt::up256;

size_t prompt_list_bytes(const PromptSizes &s, const PromptList &l) {
    const long long rows = l.keys ? s.Nk : s.Nq;
    const size_t units = (size_t)((rows + l.tile - 1) / l.tile + s.B);
    return up256(sizeof(Header) + sizeof(Start) * (size_t)l.ctas) + up256(sizeof(Unit) * units) +
           up256(sizeof(int) * ((size_t)s.B + 1));
}

bool prompt_splits(const PromptSizes &s, const PromptSeqs &q, const PromptList &l) {
    // (the tokens that a sequence can have at most)
    const long long n = l.keys ? (q.cu_q != nullptr ? s.Nq : s.Nq / s.B) : (q.cu_k != nullptr ? s.Nk : s.Nk / s.B);
    return (n + l.step - 1) / l.step > l.whole;
}

cudaError_t launch_prompt_plan(const PromptSizes &s, const PromptSeqs &q, const PromptList *lists, int n, void *const *ws,
                               unsigned *err, cudaStream_t st) {
    PlanParams p = {};
    p.s = Sequences{s.B, s.Nq, s.Nk, q.cu_q, q.cu_k, q.n_q, q.n_k};
    p.err = err;
    for (int i = 0; i < n; ++i) {
        const PromptList &l = lists[i];
        const List a = prompt_list_at(s, l, ws[i]);
        char *end = static_cast<char *>(ws[i]) + prompt_list_bytes(s, l) - up256(sizeof(int) * ((size_t)s.B + 1));
        p.l[i] = ListParams{a.header, a.start, a.unit, reinterpret_cast<int *>(end), l.keys ? 1 : 0, l.tile, l.step,
                            l.ctas, s.Hkv, l.least, l.blank, prompt_splits(s, q, l) ? 0 : 1};
    }
    return DependentLaunch(dim3(n), dim3(kThreads), 0, st)(prompt_plan_kernel, p);
}

prompt::List prompt_list_at(const PromptSizes &s, const PromptList &l, void *ws) {
    char *b = static_cast<char *>(ws);
    (void)s;
    return List{reinterpret_cast<Header *>(b), reinterpret_cast<Start *>(b + sizeof(Header)),
                reinterpret_cast<Unit *>(b + up256(sizeof(Header) + sizeof(Start) * (size_t)l.ctas))};
}

}  // namespace gdn
