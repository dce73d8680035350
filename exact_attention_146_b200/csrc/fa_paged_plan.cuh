// fa_paged_plan.cuh -- how the attention over a paged cache is cut into work.
//
// A unit is (request r, group g of `pack` query heads of one KV head, block b of `tpb` new
// tokens); it visits the key tiles js .. je - 1 (KS keys each) that its tokens can see:
//     last  = max(0, the block's last token + L - n)   (causal; L - 1 without a mask)
//     first = max(0, the block's first token + L - n - W + 1)   (window W; else 0)
//     js = first / KS,   je = last / KS + 1            (at least one tile, masked if need be).
// Units in the order (r, g, b) are laid end to end on a line of key-tile steps, and the line is
// cut into one equal range per worker (a CTA or a warp): every worker does the same number of
// steps, whatever the mix of lengths, and a unit that a cut crosses is merged afterwards.
//
// The lengths are on the device, so every worker finds its own range.  The steps of a request are
// a closed form: with A(c) = sum over blocks of floor(max(0, tpb b + c) / KS) (a floor sum, by the
// Euclidean recursion), a group of nb blocks takes nb + A(tpb - 1 + L - n) - A(L - n - W + 1)
// steps.  A block sums the requests once (each thread a contiguous segment of them), scans the
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
    int causal, window;
    int groups;                    // head groups a request: Hq / pack
    int tpb;                       // new tokens a unit
    int workers;
};

struct Request {
    int q0, n, L;
};

// sum_{i < n} floor((a i + b) / m), a, b >= 0, m >= 1.
FA_PLAN long long floor_sum(long long n, long long m, long long a, long long b) {
    long long sum = 0;
    while (n > 0) {
        if (a >= m) {
            sum += (n - 1) * n / 2 * (a / m);
            a %= m;
        }
        if (b >= m) {
            sum += n * (b / m);
            b %= m;
        }
        if (a == 0) break;
        const long long y = a * n + b;
        if (y < m) break;
        n = y / m;
        b = y % m;
        const long long t = m;
        m = a;
        a = t;
    }
    return sum;
}

// sum_{b < nb} floor(max(0, a b + c) / m).
FA_PLAN long long floor_sum_from(long long nb, long long m, long long a, long long c) {
    if (c < 0) {
        const long long skip = (-c + a - 1) / a;   // blocks whose value is below 0
        if (skip >= nb) return 0;
        nb -= skip;
        c += skip * a;
    }
    return floor_sum(nb, m, a, c);
}

// Request r; one that is out of range counts as having no tokens (and is reported once).
FA_PLAN Request load_request(const PlanParams &p, int r, bool say = false) {
    Request q;
    q.q0 = p.cu[r];
    q.n = p.cu[r + 1] - q.q0;
    q.L = p.lens[r];
    if (q.q0 < 0 || q.n < 0 || q.n > p.max_new || (long long)q.q0 + q.n > p.T || q.L < 0 || (long long)q.L > p.max_len) {
#ifdef __CUDA_ARCH__
        if (say) fa_host::report_range(p.status, fa_host::kSiteLengths, r);
#endif
        q.n = 0;
    }
    return q;
}

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
    long long s = je - js;
    if (nb > 1) {
        const long long diag = (long long)q.L - q.n;
        s += nb - 1;
        if (p.causal) s += floor_sum_from(nb - 1, KS, p.tpb, p.tpb - 1 + diag);
        else s += (nb - 1) * (max((long long)q.L - 1, 0LL) / KS);
        if (p.window > 0) s -= floor_sum_from(nb - 1, KS, p.tpb, diag - p.window + 1);
    }
    return s;
}

// What the block knows of the whole line: total steps, and the sums before each thread's segment.
template <int NT_>
struct PlanScan {
    static constexpr int NT = NT_;   // threads that take part = segments
    long long seg_start[NT + 1];
    long long warp_sum[NT / 32];
};

// By all NT threads of the block.  Returns the total.
template <int KS, int NT>
__device__ inline long long plan_scan(const PlanParams &p, PlanScan<NT> &sh, int tid, bool say) {
    const int seg = (p.R + NT - 1) / NT;
    long long mine = 0;
    for (int r = tid * seg; r < min(p.R, (tid + 1) * seg); ++r) {
        const Request q = load_request(p, r, say);
        if (q.n > 0) mine += p.groups * plan_steps<KS>(p, q, plan_blocks(p, q));
    }
    const int lane = tid % 32, warp = tid / 32;
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const long long y = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += y;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const long long s = sh.warp_sum[w];
        if (w < warp) before += s;
        total += s;
    }
    sh.seg_start[tid] = before + upto - mine;
    if (tid == 0) sh.seg_start[NT] = total;
    __syncthreads();
    return total;
}

// First step of worker w's range, and the worker that step x belongs to.
FA_PLAN long long range_start(long long total, int workers, int w) {
    const long long q = total / workers, rem = total % workers;
    return w * q + min((long long)w, rem);
}
FA_PLAN int range_owner(long long total, int workers, long long x) {
    const long long q = total / workers, rem = total % workers;
    if (x < rem * (q + 1)) return int(x / (q + 1));
    return int(rem + (x - rem * (q + 1)) / q);
}

// A unit on the line: its place, and where on the line it begins and ends.
struct Unit {
    int r, g, b, js, je;
    Request q;
    long long begin;   // first step on the line
};

// The unit that step x (0 <= x < total) lies in.
template <int KS, int NT>
FA_PLAN Unit plan_find(const PlanParams &p, const PlanScan<NT> &sh, long long x) {
    int lo = 0, hi = NT;
    while (hi - lo > 1) {   // the last segment that begins at or before x
        const int mid = (lo + hi) / 2;
        if (sh.seg_start[mid] <= x) lo = mid;
        else hi = mid;
    }
    const int seg = (p.R + NT - 1) / NT;
    Unit u{};
    long long at = sh.seg_start[lo], group = 0;
    for (u.r = lo * seg; u.r < p.R; ++u.r) {
        u.q = load_request(p, u.r);
        if (u.q.n == 0) continue;
        group = plan_steps<KS>(p, u.q, plan_blocks(p, u.q));
        if (x < at + group * p.groups) break;
        at += group * p.groups;
    }
    u.g = int((x - at) / group);
    at += u.g * group;
    int b_lo = 0, b_hi = plan_blocks(p, u.q);
    while (b_hi - b_lo > 1) {
        const int mid = (b_lo + b_hi) / 2;
        if (at + plan_steps<KS>(p, u.q, mid) <= x) b_lo = mid;
        else b_hi = mid;
    }
    u.b = b_lo;
    u.begin = at + plan_steps<KS>(p, u.q, b_lo);
    plan_range<KS>(p, u.q, u.b, u.js, u.je);
    return u;
}

// The next unit of the line (there is one).
template <int KS>
FA_PLAN void plan_next(const PlanParams &p, Unit &u) {
    u.begin += u.je - u.js;
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

#undef FA_PLAN

}  // namespace fa
