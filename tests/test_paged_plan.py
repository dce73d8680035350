"""How the paged attention cuts its work, on the CPU: the header's arithmetic compiled for the host.
Closed-form step counts against counting, and the ranges of all workers against the list of units:
every step of every unit is done once, in order, and the cuts name the right workers."""
import shutil
import subprocess
from pathlib import Path

import pytest

ROOT = Path(__file__).resolve().parents[1]
CSRC = ROOT / "exact_attention_146_b200" / "csrc"
NVCC = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"

PROGRAM = r'''
#include "fa_paged_plan.cuh"
#include <algorithm>
#include <array>
#include <cstdio>
#include <random>
#include <vector>
using namespace fa;

struct Listed { int r, g, b, js, je; };

template <int KS, int NT> int check(std::mt19937 &rng, int round) {
    auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(rng); };
    const int R = pick(1, 9);
    std::vector<int> cu{0}, lens;
    for (int r = 0; r < R; ++r) {
        const int n = pick(0, 3) == 0 ? 0 : pick(1, pick(0, 1) ? 3 : 700);
        cu.push_back(cu.back() + n);
        lens.push_back(pick(0, 5) == 0 ? pick(0, 40) : n + pick(0, pick(0, 1) ? 50 : 5000));
    }
    PlanParams p{};
    p.cu = cu.data();
    p.lens = lens.data();
    p.R = R;
    p.T = cu.back();
    p.max_new = 700;
    p.n_lo = 1;
    p.n_hi = 700;
    p.max_len = 1 << 20;
    p.causal = pick(0, 3) > 0;
    p.window = p.causal && pick(0, 1) ? pick(1, 900) : 0;
    p.groups = pick(1, 5);
    p.tpb = pick(0, 1) ? pick(1, 16) : (1 << pick(0, 8));
    p.workers = pick(1, 40);
    p.overhead = pick(0, 4);
    // counting
    std::vector<Listed> units;
    std::vector<long long> begin{0};
    PlanScan<NT> sh{};
    const int seg = (R + NT - 1) / NT;
    std::vector<long long> per_request(R, 0);
    for (int r = 0; r < R; ++r) {
        const Request q = load_request(p, r);
        const int n = cu[r + 1] - cu[r], L = lens[r];
        if (q.n != n) return 1;
        for (int g = 0; g < p.groups; ++g) {
            long long group = 0;
            for (int b = 0; b * p.tpb < n; ++b) {
                long long lo = 1LL << 40, hi = -1;   // keys that some token of the block sees
                for (int i = b * p.tpb; i < n && i < (b + 1) * p.tpb; ++i)
                    for (long long j : {0LL, (long long)L - 1}) {
                        const long long last = p.causal ? std::min<long long>(i + L - n, L - 1) : L - 1;
                        const long long first = p.window ? std::max<long long>(0, (long long)i + L - n - p.window + 1) : 0;
                        (void)j;
                        if (last >= first) lo = std::min(lo, first), hi = std::max(hi, last);
                    }
                int js, je;
                plan_range<KS>(p, q, b, js, je);
                if (hi >= 0 && (lo / KS < js || hi / KS >= je)) return 2;      // a visible key left out
                if (hi >= 0 && je != hi / KS + 1) return 3;                    // more tiles than needed
                if (je <= js || js < 0) return 4;
                group += je - js + p.overhead;
                if (plan_steps<KS>(p, q, b + 1) != group) return 5;
                units.push_back({r, g, b, js, je});
                begin.push_back(begin.back() + je - js + p.overhead);
                per_request[r] += je - js + p.overhead;
            }
        }
    }
    const long long total = begin.back();
    long long at = 0;
    for (int t = 0; t < NT; ++t) {
        sh.seg_start[t] = at;
        sh.seg_units[t] = int(std::lower_bound(begin.begin(), begin.end(), at) - begin.begin());
        for (int r = t * seg; r < std::min(R, (t + 1) * seg); ++r) at += per_request[r];
    }
    sh.seg_start[NT] = at;
    if (at != total) return 6;
    for (size_t i = 0; i < units.size(); ++i) {
        const Unit u = plan_unit<KS>(p, sh.seg_units, NT, seg, int(i));
        const Listed &e = units[i];
        if (u.r != e.r || u.g != e.g || u.b != e.b || u.js != e.js || u.je != e.je) return 11;
    }
    // the workers' walks
    size_t k = 0;
    long long x = 0;
    for (int w = 0; w < p.workers; ++w) {
        const long long x0 = range_start(total, p.workers, w), x1 = range_start(total, p.workers, w + 1);
        if (x0 != x || x1 < x0 || x1 - x0 > total / p.workers + 1) return 7;
        if (x1 == x0) continue;
        Unit u = plan_find<KS>(p, sh.seg_start, NT, seg, x0);
        while (x < x1) {
            while (begin[k + 1] <= x) ++k;
            const Listed &e = units[k];
            if (u.r != e.r || u.g != e.g || u.b != e.b || u.js != e.js || u.je != e.je || u.begin != begin[k]) return 9;
            x = std::min(x1, begin[k + 1]);
            if (x < x1) plan_next<KS>(p, u);
        }
    }
    if (x != total) return 10;
    // pieces and merge jobs, for even cuts and for uneven ones (empty ranges among them)
    for (int kind = 0; kind < 2; ++kind) {
        std::vector<long long> cuts;
        const long long x0 = kind ? begin[pick(0, int(units.size()))] : 0;   // the rest of a line behind whole units
        for (int w = 0; w <= p.workers; ++w)
            cuts.push_back(kind ? x0 + (total - x0 > 0 ? std::uniform_int_distribution<long long>(0, total - x0)(rng) : 0)
                                : range_start(total, p.workers, w));
        std::sort(cuts.begin(), cuts.end());
        cuts.front() = x0;
        cuts.back() = total;
        auto cut_at = [&](int w) { return cuts[w]; };
        std::vector<std::vector<std::array<int, 3>>> done(units.size());   // pieces (js, je, slot) of each unit; slot -1: whole
        for (int w = 0; w < p.workers; ++w) {
            if (cuts[w] >= total) continue;
            Walk walk{};
            walk.u = plan_find<KS>(p, sh.seg_start, NT, seg, cuts[w]);
            walk.o = cuts[w] - walk.u.begin;
            walk.left = cuts[w + 1] - cuts[w];
            walk.first = true;
            Piece piece;
            int slots = 0;
            while (walk_next<KS>(p, walk, piece)) {
                const size_t i = std::lower_bound(begin.begin(), begin.end(), piece.u.begin) - begin.begin();
                const bool whole = piece.js == piece.u.js && piece.je == piece.u.je;
                const int slot = whole ? -1 : 2 * w + (piece.first ? 0 : 1);
                if (!whole && (slots & (piece.first ? 1 : 2))) return 12;   // a slot used twice
                if (!whole) slots |= piece.first ? 1 : 2;
                done[i].push_back({piece.js, piece.je, slot});
            }
        }
        std::vector<int> merged(units.size(), 0);
        for (int w = 1; w < p.workers; ++w) {
            if (cuts[w] >= total) continue;
            const Unit u = plan_find<KS>(p, sh.seg_start, NT, seg, cuts[w]);
            const MergeJob job = merge_job(p, u, w, p.workers, cut_at);
            if (job.parts == 0) continue;
            const size_t i = std::lower_bound(begin.begin(), begin.end(), u.begin) - begin.begin();
            if (merged[i]++) return 13;
            std::vector<int> slots;
            for (int s = 0; s < job.parts; ++s)
                if (cuts[w - 1 + s] < cuts[w + s]) slots.push_back(s == 0 ? job.first_slot : 2 * (w - 1 + s));
            if (slots.size() != done[i].size()) return 14;
            for (size_t s = 0; s < slots.size(); ++s)
                if (slots[s] != done[i][s][2]) return 15;
            if (job.row0 != cu[u.r] + u.b * p.tpb || job.g != u.g) return 16;
        }
        for (size_t i = 0; i < units.size(); ++i) {
            if (begin[i] < x0) continue;
            int js = units[i].js;
            for (auto &d : done[i]) {
                if (d[0] != js || d[1] <= d[0]) return 17;
                js = d[1];
            }
            if (js != units[i].je) return 18;
            if ((done[i].size() > 1) != (merged[i] == 1)) return 19;
        }
    }
    return 0;
}

int main() {
    std::mt19937 rng(7);
    for (int i = 0; i < 4000; ++i) {
        int e = check<16, 4>(rng, i);
        if (e == 0) e = check<128, 32>(rng, i);
        if (e == 0) e = check<64, 2>(rng, i);
        if (e) { printf("round %d: check %d\n", i, e); return 1; }
    }
    // beyond 32 bits: the sums of a long request
    if (floor_sum(3, 7, 1LL << 40, 5) != ((0 + 5) / 7 + ((1LL << 40) + 5) / 7 + ((2LL << 40) + 5) / 7)) return 2;
    printf("ok\n");
    return 0;
}
'''


def test_plan_arithmetic(tmp_path):
    if not Path(NVCC).exists():
        pytest.skip("nvcc not found")
    src, exe = tmp_path / "plan.cu", tmp_path / "plan"
    src.write_text(PROGRAM)
    cc = subprocess.run([NVCC, "-std=c++17", "-O1", "-arch=sm_100a", f"-I{CSRC}", f"-I{ROOT / 'include'}", str(src), "-o", str(exe)],
                        capture_output=True, text=True)
    assert cc.returncode == 0, cc.stderr
    run = subprocess.run([str(exe)], capture_output=True, text=True, timeout=120)
    assert run.returncode == 0 and run.stdout.strip() == "ok", run.stdout + run.stderr
