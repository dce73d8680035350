// fa_paged_rows.cuh -- attention over a paged cache for units of up to 16 rows (a decoding step:
// the query heads of one KV head, times a few new tokens).
//
// Few rows make it a matter of reading K and V once: 4 d flops a key and row against 4 d bytes a
// key, at most 16 flops a byte, where the card's rates cross at about 250.  So every warp is a
// worker of its own: it takes one contiguous range of 16-key steps (fa_paged_plan.cuh), streams
// the keys' rows by cp.async into its own ring in shared memory, and never waits for another
// warp; nothing but the ring's depth limits the bytes in flight.  Rows are gathered one by one
// through the block table, so any page size and any strides do; rows that are not visible are
// filled with zeros by the copy itself (what lies behind a request's last key is never read).
//
// Per step: S (16 x 16) = Q K^T, the running maximum m and sum l of the online softmax, and
// O += P V, all in registers with the warp-level m16n8k16 product (an MMA of 128 rows would be
// 7/8 empty here).  At the end of a unit the warp writes O / l and LSE, or, where a cut of the
// line crosses the unit, its own normalised O and LSE to the workspace (fp32); the merge kernel
// combines those in the order of the workers:  LSE = ln sum_s e^LSE_s,  O = sum_s e^(LSE_s - LSE) O_s.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fa_paged_plan.cuh"
#include "sm100.cuh"

namespace fa {

struct PagedParams {
    PlanParams plan;
    const uint16_t *q, *k, *v;
    uint16_t *out;
    float *lse;                    // [Hq, T] or nullptr
    const int *table;
    long long table_stride, q_stride;
    long long block_stride, slot_stride, head_stride;
    float *o_part, *lse_part;      // workspace: [workers][2][rows][d], [workers][2][rows]
    int Hq, pack, n_rep, page, num_blocks;
    float scale_log2;              // scale * log2(e)
    int say;                       // this kernel reports requests that are out of range
    MergeJob *jobs;                // workspace: [workers], the job of each cut
};

constexpr int kRowKeys = 16;       // keys a step
constexpr int kRowRows = 16;       // rows a unit
constexpr int kMaxPagedCtas = 192;
constexpr float kLn2 = 0.6931471805599453f;

template <int D_, bool F16_>
struct RowCfg {
    static constexpr int D = D_;
    static constexpr bool F16 = F16_;
    static constexpr int WARPS = D >= 192 ? 4 : 8;
    static constexpr int THREADS = 32 * WARPS;
    static constexpr int UNITS = D / 8;                  // 16-byte units a row
    static constexpr int ROW = (UNITS + 1) * 16;         // bytes; an odd number of units, so that the
                                                         // eight rows of an ldmatrix fall in distinct banks
    static constexpr int TILE = kRowKeys * ROW;
    static constexpr int STAGE = 2 * TILE;               // K and V
    static constexpr int FIT = (224 * 1024) / (WARPS * STAGE);
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int SMEM = WARPS * STAGES * STAGE;
    static_assert(STAGES >= 3, "ring depth");
    static_assert(UNITS % 2 == 0, "whole copies of a warp");
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A worker's place on the line: the unit, the next step in it and how many steps are left.
struct Cursor {
    Unit u;
    int j;
    int left;
};

template <int KS>
__device__ __forceinline__ void cursor_step(const PlanParams &p, Cursor &c) {
    if (--c.left > 0 && ++c.j >= c.u.je) {
        plan_next<KS>(p, c.u);
        c.j = c.u.js;
    }
}

// Keys that some row of the unit sees: [lo, hi].
__device__ __forceinline__ void unit_keys(const PlanParams &p, const Unit &u, int &lo, int &hi) {
    const long long diag = (long long)u.q.L - u.q.n;
    hi = u.q.L - 1;
    if (p.causal) hi = int(min((long long)u.q.n, (long long)(u.b + 1) * p.tpb) - 1 + diag);
    lo = p.window > 0 ? int(max(0LL, (long long)u.b * p.tpb + diag - p.window + 1)) : 0;
}

// The keys that token i of a request sees: [lo, hi] (hi < lo: none).
__device__ __forceinline__ void token_keys(const PlanParams &p, const Request &q, int i, int &lo, int &hi) {
    const long long at = (long long)i + q.L - q.n;
    hi = p.causal ? int(max(at, -1LL)) : q.L - 1;
    lo = p.window > 0 ? int(max(0LL, at - p.window + 1)) : 0;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) fa_paged_rows_kernel(const __grid_constant__ PagedParams p) {
    constexpr int D = C::D;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ PlanScan<C::THREADS> scan;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge may be set up meanwhile
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32;
    const long long total = plan_scan<kRowKeys>(p.plan, scan, int(threadIdx.x), blockIdx.x == 0 && p.say != 0);
    // Neighbouring workers are on different SMs, so that few of them spread out.
    const int worker = warp * int(gridDim.x) + int(blockIdx.x);
    // A call too small for all: a unit of U steps in pieces of s costs s steps and then the merge of U / s
    // pieces, eight loads of them at a time; with a step and such a round about equally long, s^2 = U / 8.
    const float mean = float(total) / float(max(1, scan.seg_units[C::THREADS]));
    const long long least = max(2LL, (long long)sqrtf(mean * 0.125f));
    const int workers = int(max(1LL, min((long long)p.plan.workers, total / least)));
    const long long x0 = worker < workers ? range_start(total, workers, worker) : total;
    const long long x1 = worker < workers ? range_start(total, workers, worker + 1) : total;
    if (x0 >= x1) {
        if (lane == 0) p.jobs[worker].parts = 0;
        return;
    }

    Cursor load;
    load.u = plan_find<kRowKeys>(p.plan, scan.seg_start, C::THREADS, (p.plan.R + C::THREADS - 1) / C::THREADS, x0);
    load.j = load.u.js + int(x0 - load.u.begin);
    load.left = int(min(x1 - x0, 0x7fffffffLL));
    Cursor cur = load;
    if (lane == 0) {
        MergeJob job{};
        if (worker > 0) job = merge_job(p.plan, load.u, worker, workers, [&](int w) { return range_start(total, workers, w); });
        p.jobs[worker] = job;
    }

    const uint32_t base = sm100::smem_u32(ring) + uint32_t(warp * C::STAGES * C::STAGE);

    // Where key (lane % 16) of the step under `load` lies (elements from the cache's base; -1: not
    // visible, filled with zeros).
    auto find_key = [&]() -> long long {
        if (load.left <= 0) return -1;
        int lo, hi;
        unit_keys(p.plan, load.u, lo, hi);
        const int key = load.j * kRowKeys + (lane & 15);
        if (key < lo || key > hi) return -1;
        const int page = key / p.page;
        const int id = __ldg(p.table + load.u.r * p.table_stride + page);
        if (id < 0 || id >= p.num_blocks) {
            if (lane < 16) fa_host::report_range(p.plan.status, fa_host::kSiteTableId, load.u.r);
            return -1;
        }
        return id * p.block_stride + (key - page * p.page) * p.slot_stride +
               (long long)(load.u.g * p.pack / p.n_rep) * p.head_stride;
    };
    // Copies the rows at `at` (one key a lane) into ring slot `s` and commits the group.
    auto copy_rows = [&](long long at, bool any, int s) {
        if (any) {
            const uint32_t dst = base + uint32_t(s * C::STAGE);
#pragma unroll
            for (int i = 0; i < C::UNITS / 2; ++i) {
                const int unit = lane + 32 * i, row = unit / C::UNITS, col = unit - row * C::UNITS;
                const long long off = __shfl_sync(0xffffffffu, at, row);
                const uint32_t n = off < 0 ? 0u : 16u;
                const long long e = off < 0 ? 0 : off + col * 8;
                cp_async16(dst + uint32_t(row * C::ROW + col * 16), p.k + e, n);
                cp_async16(dst + uint32_t(C::TILE + row * C::ROW + col * 16), p.v + e, n);
            }
        }
        cp_async_commit();
    };

    long long at = find_key();
    bool any = load.left > 0;
    int put = 0;
#pragma unroll
    for (int s = 0; s < C::STAGES - 1; ++s) {
        cursor_step<kRowKeys>(p.plan, load);
        const long long next = find_key();
        copy_rows(at, any, put);
        put = put + 1 == C::STAGES ? 0 : put + 1;
        at = next;
        any = load.left > 0;
    }

    uint32_t qf[D / 16][4];
    float o[D / 8][4];
    float m[2], l[2];
    int lo[2], hi[2], token[2], head[2];
    bool there[2];
    int j0 = cur.j;             // first step of the piece of this unit
    bool fresh = true;
    int get = 0;
    const int t2 = (lane & 3) * 2;
    // ldmatrix row addresses: K (matrices: keys 0-7 | 0-7 | 8-15 | 8-15, columns 0 | 8 | 0 | 8) and
    // V, transposed (keys 0-7 | 8-15 | 0-7 | 8-15, columns 0 | 0 | 8 | 8)
    const uint32_t k_addr = uint32_t(((lane & 7) + ((lane >> 4) << 3)) * C::ROW + ((lane >> 3) & 1) * 16);
    const uint32_t v_addr = uint32_t(C::TILE + ((lane & 7) + ((lane >> 3) & 1) * 8) * C::ROW + (lane >> 4) * 16);

    while (cur.left > 0) {
        if (fresh) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int row = (lane >> 2) + 8 * h, i = row / p.pack;
                token[h] = cur.u.b * p.plan.tpb + i;
                head[h] = cur.u.g * p.pack + row - i * p.pack;
                there[h] = i < p.plan.tpb && token[h] < cur.u.q.n;
                token_keys(p.plan, cur.u.q, token[h], lo[h], hi[h]);
                if (!there[h]) hi[h] = -1;
                m[h] = -INFINITY;
                l[h] = 0.f;
                const uint16_t *src = p.q + (long long)(cur.u.q.q0 + token[h]) * p.q_stride + (long long)head[h] * D + t2;
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    qf[kk][h] = there[h] ? *reinterpret_cast<const uint32_t *>(src + 16 * kk) : 0u;
                    qf[kk][2 + h] = there[h] ? *reinterpret_cast<const uint32_t *>(src + 16 * kk + 8) : 0u;
                }
            }
#pragma unroll
            for (int n = 0; n < D / 8; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
            fresh = false;
        }
        cp_async_wait<C::STAGES - 2>();
        __syncwarp();
        // the slot that the step before this one used takes the step STAGES - 1 ahead
        {
            cursor_step<kRowKeys>(p.plan, load);
            const long long next = find_key();
            copy_rows(at, any, put);
            put = put + 1 == C::STAGES ? 0 : put + 1;
            at = next;
            any = load.left > 0;
        }
        const uint32_t tile = base + uint32_t(get * C::STAGE);
        get = get + 1 == C::STAGES ? 0 : get + 1;

        float s[2][4] = {};
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            uint32_t b[4];
            ldmatrix4(b, tile + k_addr + uint32_t(32 * kk));
            mma16816<C::F16>(s[0], qf[kk], b[0], b[1]);
            mma16816<C::F16>(s[1], qf[kk], b[2], b[3]);
        }
        const int key0 = cur.j * kRowKeys + t2;
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                const int key = key0 + 8 * n + (c & 1), h = c >> 1;
                s[n][c] = (key < lo[h] || key > hi[h]) ? -INFINITY : s[n][c] * p.scale_log2;
                mx[h] = fmaxf(mx[h], s[n][c]);
            }
        bool grew = false;
        float alpha[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
            mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
            const float now = fmaxf(m[h], mx[h]);
            alpha[h] = now == -INFINITY ? 1.f : sm100::ex2_approx(m[h] - now);
            grew |= now != m[h];
            m[h] = now;
        }
        if (__any_sync(0xffffffffu, grew)) {
            l[0] *= alpha[0];
            l[1] *= alpha[1];
#pragma unroll
            for (int n = 0; n < D / 8; ++n) {
                o[n][0] *= alpha[0];
                o[n][1] *= alpha[0];
                o[n][2] *= alpha[1];
                o[n][3] *= alpha[1];
            }
        }
        const float ref[2] = {m[0] == -INFINITY ? 0.f : m[0], m[1] == -INFINITY ? 0.f : m[1]};
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                s[n][c] = sm100::ex2_approx(s[n][c] - ref[c >> 1]);
                l[c >> 1] += s[n][c];
            }
        const uint32_t pf[4] = {sm100::pack_x2<C::F16>(s[0][0], s[0][1]), sm100::pack_x2<C::F16>(s[0][2], s[0][3]),
                                sm100::pack_x2<C::F16>(s[1][0], s[1][1]), sm100::pack_x2<C::F16>(s[1][2], s[1][3])};
#pragma unroll
        for (int n = 0; n < D / 16; ++n) {
            uint32_t b[4];
            ldmatrix4_trans(b, tile + v_addr + uint32_t(32 * n));
            mma16816<C::F16>(o[2 * n], pf, b[0], b[1]);
            mma16816<C::F16>(o[2 * n + 1], pf, b[2], b[3]);
        }
        __syncwarp();   // the slot may be filled again

        if (cur.left == 1 || cur.j + 1 == cur.u.je) {   // the end of this unit's piece
            const bool whole = j0 == cur.u.js && cur.j + 1 == cur.u.je;
            const int slot = 2 * worker + (j0 - cur.u.js + cur.u.begin == x0 ? 0 : 1);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float sum = l[h];
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                const float inv = sum > 0.f ? 1.f / sum : 0.f;
                const float lse = sum > 0.f ? (m[h] + log2f(sum)) * kLn2 : -INFINITY;
                if (!there[h]) continue;
                if (whole) {
                    const long long row = cur.u.q.q0 + token[h];
                    uint16_t *dst = p.out + (row * p.Hq + head[h]) * D + t2;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<uint32_t *>(dst + 8 * n) =
                            sm100::pack_x2<C::F16>(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                    if (p.lse != nullptr && (lane & 3) == 0) p.lse[(long long)head[h] * p.plan.T + row] = lse;
                } else {
                    const long long row = (long long)slot * kRowRows + (lane >> 2) + 8 * h;
                    float *dst = p.o_part + row * D + t2;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n)
                        *reinterpret_cast<float2 *>(dst + 8 * n) = make_float2(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
                    if ((lane & 3) == 0) p.lse_part[row] = lse;
                }
            }
            fresh = true;
        }
        cursor_step<kRowKeys>(p.plan, cur);
        if (fresh) j0 = cur.j;
    }
    cp_async_wait<0>();
}

// Merges the pieces of the unit that cut w crosses first: rows [row0, row1) of it, a warp each in turn.
// ROWS: rows a unit has in the workspace, in tiles of TILE (each TILE / pack tokens of `pack` heads).
// there(s): whether worker w - 1 + s did any steps.  All pieces' rows are loaded eight at a time.
template <int D, bool F16, int ROWS, int TILE, class There>
__device__ __forceinline__ void merge_unit(const PagedParams &p, int w, int row0, int row1, const There &there) {
    const MergeJob job = p.jobs[w];
    if (job.parts == 0) return;
    constexpr int VEC = D % 128 == 0 ? 4 : (D % 64 == 0 ? 2 : 1), PER = (D + 32 * VEC - 1) / (32 * VEC);
    const int lane = int(threadIdx.x) % 32, warps = int(blockDim.x) / 32;
    auto row_of = [&](int s, int row) { return (long long)(s == 0 ? job.first_slot : 2 * (w - 1 + s)) * ROWS + row; };
    for (int row = row0 + int(threadIdx.x) / 32; row < row1; row += warps) {
        const int tile = row / TILE, in_tile = row - tile * TILE, i = in_tile / p.pack, tq = TILE / p.pack;
        const int token = tile * tq + i, head = job.g * p.pack + in_tile - i * p.pack;
        if (i >= tq || token >= job.tokens) continue;
        float m = -INFINITY, sum = 0.f;
        float acc[PER][VEC] = {};
        for (int base = 0; base < job.parts; base += 32) {   // 32 pieces at a time, as the online softmax
            const int s = base + lane;
            const float ls = s < job.parts && there(s) ? p.lse_part[row_of(s, row)] : -INFINITY;
            float mx = ls;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float now = fmaxf(m, mx);
            if (now == -INFINITY) continue;
            const float wl = __expf(ls - now), keep = __expf(m - now);
            m = now;
            float add = wl;
#pragma unroll
            for (int o = 16; o > 0; o /= 2) add += __shfl_xor_sync(0xffffffffu, add, o);
            sum = sum * keep + add;
#pragma unroll
            for (int e = 0; e < PER; ++e)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[e][v] *= keep;
            const int n = min(32, job.parts - base);
            for (int t0 = 0; t0 < n; t0 += 8) {
                float x[8][PER][VEC];
                float wt[8];
#pragma unroll
                for (int t = 0; t < 8; ++t) {
                    wt[t] = __shfl_sync(0xffffffffu, wl, (t0 + t) % 32);
                    const bool use = t0 + t < n && wt[t] != 0.f;   // a piece of weight 0 may not have been written
#pragma unroll
                    for (int e = 0; e < PER; ++e) {
                        const int col = (e * 32 + lane) * VEC;
                        const float *src = p.o_part + row_of(base + t0 + t, row) * D + col;
#pragma unroll
                        for (int v = 0; v < VEC; ++v) x[t][e][v] = 0.f;
                        if (use && col < D) {
                            if constexpr (VEC == 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(src);
                                x[t][e][0] = f.x, x[t][e][1] = f.y, x[t][e][2] = f.z, x[t][e][3] = f.w;
                            } else if constexpr (VEC == 2) {
                                const float2 f = *reinterpret_cast<const float2 *>(src);
                                x[t][e][0] = f.x, x[t][e][1] = f.y;
                            } else {
                                x[t][e][0] = *src;
                            }
                        }
                    }
                }
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int e = 0; e < PER; ++e)
#pragma unroll
                        for (int v = 0; v < VEC; ++v) acc[e][v] = fmaf(wt[t], x[t][e][v], acc[e][v]);
            }
        }
        const float inv = sum > 0.f ? 1.f / sum : 0.f;
        const long long at = job.row0 + token;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
            const int col = (e * 32 + lane) * VEC;
            if (col >= D) continue;
            uint16_t *dst = p.out + (at * p.Hq + head) * D + col;
            if constexpr (VEC == 1) {
                const float x = acc[e][0] * inv;
                *dst = F16 ? __half_as_ushort(__float2half_rn(x)) : __bfloat16_as_ushort(__float2bfloat16_rn(x));
            } else {
#pragma unroll
                for (int v = 0; v < VEC; v += 2)
                    *reinterpret_cast<uint32_t *>(dst + v) = sm100::pack_x2<F16>(acc[e][v] * inv, acc[e][v + 1] * inv);
            }
        }
        if (p.lse != nullptr && lane == 0) p.lse[(long long)head * p.plan.T + at] = sum > 0.f ? m + logf(sum) : -INFINITY;
    }
}

// The merge of a call that has pieces of few rows only: one block a cut.
template <int D, bool F16>
__global__ void __launch_bounds__(256) fa_paged_merge_rows_kernel(const __grid_constant__ PagedParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the pieces and jobs are written
    merge_unit<D, F16, kRowRows, kRowRows>(p, int(blockIdx.x) + 1, 0, kRowRows, [](int) { return true; });
}

}  // namespace fa
