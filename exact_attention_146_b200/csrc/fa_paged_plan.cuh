// fa_paged_plan.cuh -- how the attention over a paged cache is cut into work.
//
// A unit is (request r, group g of `pack` query heads of one KV head, block b of `tpb` new
// tokens); it visits the key tiles js .. je - 1 (KS keys each) that its tokens can see:
//     last  = max(0, the block's last token + L - n)   (causal; L - 1 without a mask)
//     first = max(0, the block's first token + L - n - W + 1)   (window W; else 0)
//     js = first / KS,   je = last / KS + 1            (at least one tile, masked if need be).
// Units in the order (r, g, b) are laid end to end on a line of steps, one a key tile and `overhead`
// before them for what a unit costs besides, and the line is
// cut into one equal range per worker (a CTA or a warp): every worker does the same number of
// steps, whatever the mix of lengths, and a unit that a cut crosses is merged afterwards.
//
// The lengths are on the device, so every worker finds its own range.  The steps of a request are
// a closed form: with A(c) = sum over blocks of floor(max(0, tpb b + c) / KS) (a floor sum, by the
// Euclidean recursion that follows from the reciprocity of such sums: Graham, Knuth and Patashnik, Concrete
// Mathematics, section 3.5), a group of nb blocks takes nb (1 + overhead) + A(tpb - 1 + L - n) -
// A(L - n - W + 1) steps.  A block sums the requests once (each thread a contiguous segment of them), scans the
// segment sums, and a worker finds its place by bisection.
#pragma once

#include <cstdint>

#include "fa_cache.h"

namespace fa {

#define FA_PLAN __host__ __device__ inline   // the arithmetic also runs on the host, in a test

struct PlanParams {
    const int *cu, *lens;          // [R + 1], [R]
    int *status;
    long long max_len;             // max_blocks * page_size
    int R, T, max_new;
    int n_lo, n_hi;                // requests of n_lo .. n_hi new tokens take part
    int causal, window;
    int groups;                    // head groups a request: Hq / pack
    int tpb;                       // new tokens a unit
    int workers;
    int overhead;                  // steps that a unit costs besides its key tiles
};

struct Request {
    int q0, n, L;
};

// Quotient of values >= 0; 32-bit ones (nearly always) take the short division.
FA_PLAN long long div_pos(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (long long)((unsigned)a / (unsigned)b);
    return a / b;
}

// sum_{i < n} floor((a i + b) / m), a, b >= 0, m >= 1.
FA_PLAN long long floor_sum(long long n, long long m, long long a, long long b) {
    long long sum = 0;
    while (n > 0) {
        if (a >= m) {
            const long long q = div_pos(a, m);
            sum += (n - 1) * n / 2 * q;
            a -= q * m;
        }
        if (b >= m) {
            const long long q = div_pos(b, m);
            sum += n * q;
            b -= q * m;
        }
        if (a == 0) break;
        const long long y = a * n + b;
        if (y < m) break;
        n = div_pos(y, m);
        b = y - n * m;
        const long long t = m;
        m = a;
        a = t;
    }
    return sum;
}

// sum_{b < nb} floor(max(0, a b + c) / m).
FA_PLAN long long floor_sum_from(long long nb, long long m, long long a, long long c) {
    if (c < 0) {
        const long long skip = div_pos(-c + a - 1, a);   // blocks whose value is below 0
        if (skip >= nb) return 0;
        nb -= skip;
        c += skip * a;
    }
    return floor_sum(nb, m, a, c);
}

// Request r of rows q0 .. end - 1 and L keys; one that is out of range counts as having no tokens (and
// is reported once).
FA_PLAN Request make_request(const PlanParams &p, int r, int q0, int end, int L, bool say) {
    Request q{q0, end - q0, L};
    if (q.q0 < 0 || q.n < 0 || q.n > p.max_new || (long long)q.q0 + q.n > p.T || q.L < 0 || (long long)q.L > p.max_len) {
#ifdef __CUDA_ARCH__
        if (say) fa_host::report_range(p.status, fa_host::kSiteLengths, r);
#endif
        q.n = 0;
    }
    if (q.n < p.n_lo || q.n > p.n_hi) q.n = 0;
    return q;
}
FA_PLAN Request load_request(const PlanParams &p, int r) { return make_request(p, r, p.cu[r], p.cu[r + 1], p.lens[r], false); }

FA_PLAN int plan_blocks(const PlanParams &p, const Request &q) { return (q.n + p.tpb - 1) / p.tpb; }

// The key tiles [js, je) of token block b.
template <int KS>
FA_PLAN void plan_range(const PlanParams &p, const Request &q, int b, int &js, int &je) {
    const long long diag = (long long)q.L - q.n;
    long long last = (long long)q.L - 1;
    if (p.causal) last = min((long long)q.n, (long long)(b + 1) * p.tpb) - 1 + diag;
    long long first = 0;
    if (p.window > 0) first = (long long)b * p.tpb + diag - p.window + 1;
    je = int(max(last, 0LL) / KS) + 1;
    js = int(max(first, 0LL) / KS);
}

// Steps of the first nb token blocks of one head group.
template <int KS>
FA_PLAN long long plan_steps(const PlanParams &p, const Request &q, int nb) {
    if (nb <= 0) return 0;
    int js, je;
    plan_range<KS>(p, q, nb - 1, js, je);   // the last block apart: it may be short
    long long s = je - js + (long long)nb * p.overhead;
    if (nb > 1) {
        const long long diag = (long long)q.L - q.n;
        s += nb - 1;
        if (p.causal) s += floor_sum_from(nb - 1, KS, p.tpb, p.tpb - 1 + diag);
        else s += (nb - 1) * (max((long long)q.L - 1, 0LL) / KS);
        if (p.window > 0) s -= floor_sum_from(nb - 1, KS, p.tpb, diag - p.window + 1);
    }
    return s;
}

FA_PLAN int plan_units(const PlanParams &p, const Request &q) { return p.groups * plan_blocks(p, q); }

// What a block knows of the whole line: the steps and the units before each thread's segment of
// requests (segment t: requests [t seg, (t + 1) seg), seg = ceil(R / NT)).
template <int NT_>
struct PlanScan {
    static constexpr int NT = NT_;   // threads that take part = segments
    long long seg_start[NT + 1];
    long long warp_sum[NT / 32];
    int warp_units[NT / 32];
    int seg_units[NT + 1];
};

// Sum of the values of the threads before this one, over all NT threads of the block.
template <int NT>
__device__ inline long long block_before(long long mine, long long *warp_sum, int tid, long long &total) {
    const int lane = tid % 32, warp = tid / 32;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    __syncthreads();   // the last use of warp_sum is over
    if (lane == 31) warp_sum[warp] = upto;
    __syncthreads();
    long long before = 0;
    total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long s = warp_sum[w];
        if (w < warp) before += s;
        total += s;
    }
    return before + upto - mine;
}

// By all NT threads of the block.  Returns the total.
template <int KS, int NT>
__device__ inline long long plan_scan(const PlanParams &p, PlanScan<NT> &sh, int tid, bool say) {
    const int seg = (p.R + NT - 1) / NT, lane = tid % 32, warp = tid / 32;
    long long steps = 0;
    int units = 0;
    const int last = min(p.R, (tid + 1) * seg);
    for (int r0 = tid * seg; r0 < last; r0 += 4) {   // the loads of four requests together
        int cu[5], L[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            cu[k] = p.cu[min(r0 + k, last)];
            L[k] = p.lens[min(r0 + k, last - 1)];
        }
        cu[4] = p.cu[min(r0 + 4, last)];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (r0 + k >= last) break;
            const Request q = make_request(p, r0 + k, cu[k], cu[k + 1], L[k], say);
            if (q.n > 0) {
                steps += p.groups * plan_steps<KS>(p, q, plan_blocks(p, q));
                units += plan_units(p, q);
            }
        }
    }
    long long upto = steps;
    int units_upto = units;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        const int z = __shfl_up_sync(0xffffffffu, units_upto, o);
        if (lane >= o) {
            upto += y;
            units_upto += z;
        }
    }
    if (lane == 31) {
        sh.warp_sum[warp] = upto;
        sh.warp_units[warp] = units_upto;
    }
    __syncthreads();
    long long before = 0, total = 0;
    int units_before = 0, total_units = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long y = sh.warp_sum[w];
        const int z = sh.warp_units[w];
        if (w < warp) {
            before += y;
            units_before += z;
        }
        total += y;
        total_units += z;
    }
    sh.seg_start[tid] = before + upto - steps;
    sh.seg_units[tid] = units_before + units_upto - units;
    if (tid == 0) {
        sh.seg_start[NT] = total;
        sh.seg_units[NT] = total_units;
    }
    __syncthreads();
    return total;
}

// First step of worker w's range.
FA_PLAN long long range_start(long long total, int workers, int w) {
    const long long q = div_pos(total, workers), rem = total - q * workers;
    return w * q + min((long long)w, rem);
}

// What the merge is told of one cut: the unit that it crosses first (parts = 0: none), its pieces
// and its rows.  Piece 0 is in slot `first_slot`, piece s > 0 in slot 2 (w - 1 + s) for cut w.
struct MergeJob {
    int parts, first_slot;
    int row0, tokens, g;       // first row of q, tokens, head group
};

// A unit on the line: its place, and where on the line it begins and ends.
struct Unit {
    int r, g, b, js, je;
    Request q;
    long long begin;   // first step on the line
};

FA_PLAN int plan_length(const PlanParams &p, const Unit &u) { return u.je - u.js + p.overhead; }

// The block of a request's head group that step x of the group lies in, and the steps before it.
// On the device a whole warp looks through 32 blocks at a time.
template <int KS>
FA_PLAN int find_block(const PlanParams &p, const Request &q, long long x, long long &before) {
    const int nb = plan_blocks(p, q);
    before = 0;
    if (nb == 1) return 0;
#ifdef __CUDA_ARCH__
    const int lane = int(threadIdx.x) % 32;
    for (int b0 = 0; b0 < nb; b0 += 32) {
        int len = 0;
        if (b0 + lane < nb) {
            int js, je;
            plan_range<KS>(p, q, b0 + lane, js, je);
            len = je - js + p.overhead;
        }
        long long upto = len;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const long long y = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o) upto += y;
        }
        const unsigned past = __ballot_sync(0xffffffffu, b0 + lane < nb && before + upto > x);
        if (past != 0) {
            const int at = __ffs(int(past)) - 1;
            before += __shfl_sync(0xffffffffu, upto - len, at);
            return b0 + at;
        }
        before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return nb - 1;
#else
    for (int b = 0;; ++b) {
        int js, je;
        plan_range<KS>(p, q, b, js, je);
        if (b == nb - 1 || before + je - js + p.overhead > x) return b;
        before += je - js + p.overhead;
    }
#endif
}

// A request on the line: its first step, and the steps of one head group.
struct Place {
    int r;
    Request q;
    long long at, group;
};

// The request that step x lies in, which is one of segment `lo`'s.
template <int KS>
FA_PLAN Place find_request(const PlanParams &p, const long long *steps_before, int lo, int seg, long long x) {
    Place f{};
    f.at = steps_before[lo];
    for (f.r = lo * seg; f.r < p.R; ++f.r) {
        f.q = load_request(p, f.r);
        if (f.q.n == 0) continue;
        f.group = plan_steps<KS>(p, f.q, plan_blocks(p, f.q));
        if (x < f.at + f.group * p.groups) break;
        f.at += f.group * p.groups;
    }
    return f;
}

// The unit of that request that step x lies in; by all threads of a warp.
template <int KS>
FA_PLAN Unit find_unit(const PlanParams &p, const Place &f, long long x) {
    Unit u{};
    u.r = f.r;
    u.q = f.q;
    u.g = int(div_pos(x - f.at, f.group));
    const long long at = f.at + u.g * f.group;
    long long before;
    u.b = find_block<KS>(p, u.q, x - at, before);
    u.begin = at + before;
    plan_range<KS>(p, u.q, u.b, u.js, u.je);
    return u;
}

// The unit that step x (0 <= x < total) lies in; by all threads of a warp.  `steps_before` are the
// steps before each of `segments` segments of `seg` requests.
template <int KS>
FA_PLAN Unit plan_find(const PlanParams &p, const long long *steps_before, int segments, int seg, long long x) {
    int lo = 0, hi = segments;
    while (hi - lo > 1) {   // the last segment that begins at or before x
        const int mid = (lo + hi) / 2;
        if (steps_before[mid] <= x) lo = mid;
        else hi = mid;
    }
    return find_unit<KS>(p, find_request<KS>(p, steps_before, lo, seg, x), x);
}

// Unit number k (0 <= k < units) of the line, without its place on it (begin = 0); `units_before` are
// the units before each of `segments` segments of `seg` requests.
template <int KS>
FA_PLAN Unit plan_unit(const PlanParams &p, const int *units_before, int segments, int seg, int k) {
    int lo = 0, hi = segments;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (units_before[mid] <= k) lo = mid;
        else hi = mid;
    }
    Unit u{};
    int at = units_before[lo];
    for (u.r = lo * seg; u.r < p.R; ++u.r) {
        u.q = load_request(p, u.r);
        const int n = u.q.n > 0 ? plan_units(p, u.q) : 0;
        if (k < at + n) break;
        at += n;
    }
    const int nb = plan_blocks(p, u.q);
    u.g = (k - at) / nb;
    u.b = k - at - u.g * nb;
    plan_range<KS>(p, u.q, u.b, u.js, u.je);
    return u;
}

// The next unit of the line (there is one).
template <int KS>
FA_PLAN void plan_next(const PlanParams &p, Unit &u) {
    u.begin += plan_length(p, u);
    if (++u.b >= plan_blocks(p, u.q)) {
        u.b = 0;
        if (++u.g >= p.groups) {
            u.g = 0;
            do {
                if (++u.r >= p.R) return;
                u.q = load_request(p, u.r);
            } while (u.q.n == 0);
        }
    }
    plan_range<KS>(p, u.q, u.b, u.js, u.je);
}

// CTAs that a call is worth: each with at least kLeastShare steps (its overhead among them).
constexpr int kLeastShare = 6;
FA_PLAN int plan_active(const PlanParams &p, long long total) {
    return int(max(1LL, min((long long)p.workers, total / kLeastShare)));
}

// The schedule of the CTAs of a tile kernel, in two phases.  First whole units, CTA c units c,
// c + G, c + 2 G, ...: CTAs that run at the same time have neighbouring units, the token blocks of one
// head, and go through its keys side by side, so that K and V come from L2.  As many rounds of G units
// as leave every CTA within its equal share of the steps; then the rest of the line is cut, each
// CTA taking what its share still lacks: CTA c the steps cuts[c] .. cuts[c + 1] - 1.
// By all NT >= G threads; `cuts` is shared memory for G + 1 places.  Returns the rounds.
template <int KS, int NT>
__device__ inline int plan_schedule(const PlanParams &p, PlanScan<NT> &sh, long long total, long long *cuts, int tid) {
    const int G = p.workers, active = plan_active(p, total), units = sh.seg_units[NT], seg = (p.R + NT - 1) / NT;
    const long long share = tid < active ? range_start(total, active, tid + 1) - range_start(total, active, tid) : 0;
    long long mine = 0;
    int rounds = 0;
    for (;; ++rounds) {
        int len = 0;
        bool stop = false;
        if (tid < G) {
            const long long k = (long long)rounds * G + tid;
            stop = k >= units;
            if (!stop) {
                const Unit u = plan_unit<KS>(p, sh.seg_units, NT, seg, int(k));
                len = plan_length(p, u);
                stop = mine + len > share;
            }
        }
        if (__syncthreads_or(stop)) break;
        mine += len;
    }
    long long rest;
    const long long before = block_before<NT>(share - mine, sh.warp_sum, tid, rest);
    if (tid < G) cuts[tid] = total - rest + before;
    if (tid == 0) cuts[G] = total;
    __syncthreads();
    return rounds;
}

// A range of the line, from step o of unit u on.  The steps of a unit's overhead have no tiles: a
// cut among them leaves the unit whole to the worker behind it.
struct Walk {
    Unit u;
    long long o, left;
    bool first;        // the next piece is the range's first
};
struct Piece {
    Unit u;
    int js, je;        // key tiles
    bool first;
};

// The next piece that has tiles; false at the end of the range.
template <int KS>
FA_PLAN bool walk_next(const PlanParams &p, Walk &w, Piece &piece) {
    while (w.left > 0) {
        const long long len = plan_length(p, w.u), end = min(len, w.o + w.left);
        piece.u = w.u;
        piece.js = w.u.js + int(max(0LL, w.o - p.overhead));
        piece.je = w.u.js + int(max(0LL, end - p.overhead));
        piece.first = w.first;
        w.first = false;
        w.left -= end - w.o;
        w.o = 0;
        if (w.left > 0) plan_next<KS>(p, w.u);
        if (piece.je > piece.js) return true;
    }
    return false;
}

// The merge job of cut w (w >= 1), which lies at cuts[w] in unit u; cuts[0 .. workers].
template <class Cuts>
FA_PLAN MergeJob merge_job(const PlanParams &p, const Unit &u, int w, int workers, const Cuts &cuts) {
    MergeJob j{};
    const long long cut = cuts(w), before = cuts(w - 1), end = u.begin + plan_length(p, u);
    // tiles on both sides, and none of the unit's cuts before this one has
    if (before == cut || cut - u.begin <= p.overhead || before - u.begin > p.overhead) return j;
    int last = w;
    while (last + 1 < workers && cuts(last + 1) < end) ++last;
    j.parts = last - (w - 1) + 1;
    j.first_slot = 2 * (w - 1) + (before >= u.begin ? 0 : 1);
    j.row0 = u.q.q0 + u.b * p.tpb;
    j.tokens = min(u.q.n - u.b * p.tpb, p.tpb);
    j.g = u.g;
    return j;
}

#undef FA_PLAN

}  // namespace fa
