// fa_paged_rows.cuh -- attention over a paged cache for units of up to 16 rows (a decoding step:
// the query heads of one KV head, times a few new tokens).
//
// Few rows make it a matter of reading K and V once: 4 d flops a key and row against 4 d bytes a
// key, at most 16 flops a byte, where the card's rates cross at about 250.  So every warp is a
// worker of its own: it takes one contiguous range of steps of 16 or 32 keys (fa_paged_plan.cuh), streams
// the keys' rows into its own ring in shared memory, and never waits for another warp; nothing but
// the ring's depth limits the bytes in flight.  Pages of whole swizzle atoms (8 slots) come by TMA, a
// box a page or the largest power-of-two run of slots that divides it; any other page row by row, a bulk
// copy a lane.  A thread spends about 70 cycles on each such instruction (16-byte cp.async held the
// warp for 1300 to 1600 cycles a step in the load unit's queue, 32 bulk copies 2200), so few and large
// ones count.  What lies outside the visible keys never reaches a result: runs without any are not
// read, and V's other rows are overwritten with zeros in shared memory (0 x NaN = NaN).
//
// Per step, 16 keys at a time: S^T (keys x rows) = K Q^T, the running maximum m and sum l of the online
// softmax down each column, and O^T (d x rows) += V^T P^T, all in registers with the warp-level m16n8k16
// product.  The rows are its narrow side (8, or 2 x 8): an MMA of 128 rows would be 15/16 empty here, and
// the other way round (rows as the 16) a decoding step of up to 8 rows took twice the products.  The
// transposed operands cost nothing: V^T comes from ldmatrix.trans, P^T from one movmatrix per 8 keys.
// m, l, S and O are fp32; P is rounded to the inputs' type for the second product (its operands have one
// type; the error is half a step of each weight, and l sums the unrounded values), O once at the end.
//
// At the end of a unit the warp writes O / l and LSE, or, where a cut of the line crosses the unit, its
// own normalised O and LSE to the workspace (fp32); the merge kernel combines those in the order of
// the workers:  LSE = ln sum_s e^LSE_s,  O = sum_s e^(LSE_s - LSE) O_s.  A row whose sum is NaN has LSE = NaN in its
// pieces too, so that it comes out NaN wherever the cuts fall.
//
// Measured (B200, in a CUDA graph): 48 requests of 4k to 16k keys (Hq 32, Hkv 8, d 128) 247 us, 6.56 TB/s (the measured copy
// rate is 6.55); 4 requests of up to 1000 keys 11.6 us: the plan 4, the first copies 2, the merge 3.
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
    int run, slot_first;           // pages by TMA: slots a box; the map's second axis is the slot (else the head)
    MergeJob *jobs;                // workspace: [workers], the job of each cut
};

constexpr int kRowRows = 16;       // rows a unit at most
constexpr int kMaxPagedCtas = 192;
constexpr int kCachedRequests = 512;
constexpr float kLn2 = 0.6931471805599453f;

// Keys a step, warps a CTA, rows a unit (8 or 16), pages by TMA, and the ring's depth.  A step costs a
// warp its chain from K Q^T over the softmax to V^T P^T however few bytes it takes, so small head dims
// take 32 keys at once; the depth is what 222 KB hold.  Measured (48 requests of 4k to 16k keys, Hkv 8):
// see fa_paged.cu.
template <int D_, bool F16_, int KEYS_, int WARPS_, int ROWS_, bool TMA_>
struct RowCfg {
    static constexpr int D = D_;
    static constexpr bool F16 = F16_;
    static constexpr int KEYS = KEYS_;
    static constexpr int WARPS = WARPS_;
    static constexpr int ROWS = ROWS_;
    static constexpr bool TMA = TMA_;
    static constexpr int THREADS = 32 * WARPS;
    // The eight rows of an ldmatrix have to fall in distinct banks.  TMA: chunks of 64 (d = 32: 32)
    // columns, swizzled; else rows padded to an odd number of 16-byte units.
    static constexpr int RB = TMA ? (D >= 64 ? 128 : 64) : (D / 8 + 1) * 16;   // bytes a row (of a chunk)
    static constexpr int CW = TMA ? RB / 2 : D;                                // columns a chunk
    static constexpr int NCH = (D + CW - 1) / CW;
    static constexpr int CHUNK = KEYS * RB;
    static constexpr int TILE = NCH * CHUNK;
    static constexpr int STAGE = 2 * TILE;               // K and V
    static constexpr int FIT = (222 * 1024) / (WARPS * STAGE);
    static constexpr int STAGES = FIT > 8 ? 8 : FIT;
    static constexpr int SMEM = WARPS * STAGES * STAGE + (TMA ? 1024 : 0);   // (alignment of the swizzle)
    static_assert(KEYS == 16 || KEYS == 32, "a key a lane");
    static_assert(ROWS == 8 || ROWS == 16, "one or two n8 tiles");
    static_assert(STAGES >= 3, "ring depth");

    // 16-byte unit c of a row in its chunk, where the swizzle puts it.
    static __device__ __forceinline__ uint32_t unit(int r, int c) {
        return uint32_t((!TMA ? c : RB == 128 ? c ^ (r & 7) : c ^ (r >> 1 & 3)) * 16);
    }
};
constexpr int kSiteRowsFull = 16;   // the wait for a step's rows (bits 8..15 of the status word)

// `bytes` (a multiple of 16) from global to shared memory, counted on `bar` when they have landed.
__device__ __forceinline__ void bulk_copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
}

// Waits for a phase of this warp's barrier, a second at most; false: it ran out (and was recorded).
__device__ __forceinline__ bool wait_rows(uint32_t bar, uint32_t parity, int *status) {
    if (sm100::mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = sm100::global_timer_ns();
    while (!sm100::mbar_try_wait(bar, parity)) {
        if (sm100::global_timer_ns() - t0 > 1000000000ull) {
            atomicCAS(status, 0, int(FA_ERR_DEVICE_TIMEOUT) | (kSiteRowsFull << 8) | (int(blockIdx.x) << 16));
            return false;
        }
    }
    return true;
}

__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}

// Transpose of the 8 x 8 tile of 16-bit values that the warp holds (row lane / 4, columns 2 (lane % 4), + 1).
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// D (16 x 8, fp32) += A (16 x 16) B (16 x 8).
template <bool F16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// A step that has been looked up: block and slot of this lane's key (TMA: of the first key of its
// box), its request and head.
struct Found {
    int id, slot, r, head;
    bool seen, any;   // the key is visible; there is such a step

    // The block is there, or has to be read as zeros (and is reported if the table names none).
    __device__ __forceinline__ bool real(const PagedParams &p) const {
        if (seen && (id < 0 || id >= p.num_blocks)) fa_host::report_range(p.plan.status, fa_host::kSiteTableId, r);
        return seen && id >= 0 && id < p.num_blocks;
    }
};

// The loading side of a worker: a step ahead of the copies, each lane knows where one key lies.
template <class C>
struct KeyStream {
    Walk walk;
    Piece piece;
    int j;                     // the piece's next step
    bool any;                  // there is one
    int key, page, slot;       // this lane's key of step j (or its box's first), its page and slot
    int span;                  // keys of which that is the first
    int lo, hi;                // keys that the unit sees
    const int *table;
    int head;                  // KV head

    __device__ __forceinline__ void enter(const PagedParams &p, const PlanParams &plan) {
        any = walk_next<C::KEYS>(plan, walk, piece);
        if (!any) return;
        j = piece.js;
        unit_keys(plan, piece.u, lo, hi);
        table = p.table + piece.u.r * p.table_stride;
        head = piece.u.g * p.pack / p.n_rep;
        span = C::TMA ? p.run : 1;
        key = j * C::KEYS + int(threadIdx.x) * span % C::KEYS;
        page = key / p.page;
        slot = key - page * p.page;
    }
    // Asks for the block of the key's page.  Nothing may look at the answer before the next step's send:
    // it may have to come from L2.
    __device__ __forceinline__ Found find() const {
        Found f;
        f.seen = any && key <= hi && key + span > lo;
        f.id = f.seen ? __ldg(table + page) : 0;
        f.slot = slot;
        f.r = piece.u.r;
        f.head = head;
        f.any = any;
        return f;
    }
    __device__ __forceinline__ void step(const PagedParams &p, const PlanParams &plan) {
        if (!any) return;
        if (++j < piece.je) {
            key += C::KEYS;
            slot += C::KEYS;
            if (slot >= p.page) {
                slot -= p.page;
                ++page;
                if (slot >= p.page) {   // pages shorter than a step
                    page = key / p.page;
                    slot = key - page * p.page;
                }
            }
        } else {
            enter(p, plan);
        }
    }
};

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
fa_paged_rows_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                     const __grid_constant__ PagedParams p) {
    constexpr int D = C::D;
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ PlanScan<C::THREADS> scan;
    __shared__ uint64_t landed[C::WARPS][C::STAGES];   // a step's rows are in their slot
    __shared__ int segment[C::WARPS];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge may be set up meanwhile
    const int tid = int(threadIdx.x), lane = tid % 32, warp = tid / 32;
    if (C::TMA && tid == 0) {
        sm100::prefetch_tensormap(&tm_k);
        sm100::prefetch_tensormap(&tm_v);
    }
    // Lengths in shared memory, where they fit: a worker that goes from one request to the next asks for
    // them in the middle of its stream.
    __shared__ int lengths[2 * kCachedRequests + 1];
    PlanParams plan = p.plan;
    if (plan.R <= kCachedRequests) {
        for (int i = tid; i <= plan.R; i += C::THREADS) {
            lengths[i] = p.plan.cu[i];
            if (i < plan.R) lengths[kCachedRequests + 1 + i] = p.plan.lens[i];
        }
        plan.cu = lengths;
        plan.lens = lengths + kCachedRequests + 1;
        __syncthreads();
    }
    const long long total = plan_scan<C::KEYS>(plan, scan, tid, blockIdx.x == 0 && p.say != 0);
    // A call too small for all workers: a unit of U steps in pieces of s costs s steps and then the merge of
    // U / s pieces, eight loads of them at a time; with a step and such a round about equally long, s^2 = U / 8.
    const float mean = float(total) / float(max(1, scan.seg_units[C::THREADS]));
    const long long least = max(2LL, (long long)sqrtf(mean * 0.125f));
    const int workers = int(max(1LL, min((long long)p.plan.workers, div_pos(total, least))));
    const long long share = div_pos(total, workers), more = total - share * workers;   // as range_start
    // Neighbouring workers are on different SMs, so that few of them spread out.
    auto worker_of = [&](int w) { return w * int(gridDim.x) + int(blockIdx.x); };
    auto start_of = [&](int i) { return i < workers ? i * share + min((long long)i, more) : total; };
    {   // the thread whose requests hold a worker's first step says so
        const long long from = scan.seg_start[tid], to = scan.seg_start[tid + 1];
#pragma unroll
        for (int w = 0; w < C::WARPS; ++w) {
            const long long x = start_of(worker_of(w));
            if (x >= from && x < to) segment[w] = tid;
        }
    }
    __syncthreads();
    const int worker = worker_of(warp);
    const long long x0 = start_of(worker), x1 = start_of(worker + 1);
    if (x0 >= x1) {
        if (lane == 0) p.jobs[worker].parts = 0;
        asm volatile("griddepcontrol.wait;" ::: "memory");   // (see the end)
        return;
    }

    Walk walk{};                // the computing side's
    walk.u = find_unit<C::KEYS>(plan, find_request<C::KEYS>(plan, scan.seg_start, segment[warp], (plan.R + C::THREADS - 1) / C::THREADS, x0), x0);
    walk.o = x0 - walk.u.begin;
    walk.left = x1 - x0;
    walk.first = true;
    KeyStream<C> load;
    load.walk = walk;
    load.enter(p, plan);

    const uint32_t ring0 = C::TMA ? (sm100::smem_u32(ring) + 1023u) & ~1023u : sm100::smem_u32(ring);
    const uint32_t base = ring0 + uint32_t(warp * C::STAGES * C::STAGE);
    const uint32_t bars = sm100::smem_u32(&landed[warp][0]);
    if (lane == 0) {
#pragma unroll
        for (int s = 0; s < C::STAGES; ++s) sm100::mbar_init(bars + 8u * s, 1);
        sm100::fence_mbar_init();
    }
    __syncwarp();
    // Sends a step's rows to ring slot `s`.
    auto send_rows = [&](const Found &f, int s) {
        if (!f.any) return;
        const bool real = f.real(p);
        const uint32_t bar = bars + 8u * s, slot0 = base + uint32_t(s * C::STAGE);
        if constexpr (C::TMA) {
            // a box at a time; one that is not there takes a block past the cache, which reads as zeros
            const int id = real ? f.id : p.num_blocks;
            if (lane == 0) sm100::mbar_arrive_expect_tx(bar, C::STAGE);
#pragma unroll 1
            for (int i = 0; i * p.run < C::KEYS; ++i) {
                const int b = __shfl_sync(0xffffffffu, id, i), sl = __shfl_sync(0xffffffffu, f.slot, i);
                const int c1 = p.slot_first ? sl : f.head, c2 = p.slot_first ? f.head : sl;
                const uint32_t dst = slot0 + uint32_t(i * p.run * C::RB);
                if (lane == 0)
#pragma unroll
                    for (int c = 0; c < C::NCH; ++c) {
                        sm100::tma_load_4d(dst + uint32_t(c * C::CHUNK), &tm_k, bar, c * C::CW, c1, c2, b);
                        sm100::tma_load_4d(dst + uint32_t(C::TILE + c * C::CHUNK), &tm_v, bar, c * C::CW, c1, c2, b);
                    }
            }
        } else {
            // with 16 keys a step, lanes 0-15 the rows of K and 16-31 those of V; with 32, each lane both
            constexpr uint32_t kBytes = 2 * D;
            const unsigned seen = __ballot_sync(0xffffffffu, real);
            if (lane == 0) sm100::mbar_arrive_expect_tx(bar, uint32_t(__popc(seen)) * (C::KEYS == 32 ? 2 * kBytes : kBytes));
            __syncwarp();
            const uint32_t dst = slot0 + uint32_t((lane % C::KEYS) * C::RB + (C::KEYS == 16 ? lane / 16 * C::TILE : 0));
            if (real) {
                const long long at = f.id * p.block_stride + f.slot * p.slot_stride + f.head * p.head_stride;
                bulk_copy(dst, (C::KEYS == 16 && lane >= 16 ? p.v : p.k) + at, kBytes, bar);
                if constexpr (C::KEYS == 32) bulk_copy(dst + uint32_t(C::TILE), p.v + at, kBytes, bar);
            } else {
#pragma unroll 1
                for (int i = 0; i < D / 8; ++i) {
                    sm100::st_shared_v4(dst + 16 * i, 0u, 0u, 0u, 0u);
                    if constexpr (C::KEYS == 32) sm100::st_shared_v4(dst + uint32_t(C::TILE + 16 * i), 0u, 0u, 0u, 0u);
                }
                sm100::fence_proxy_async_smem();   // before the slot's next copies
            }
        }
    };

    Found found = load.find();
    int put = 0, get = 0;
    uint32_t parity = 0;
    // Sends the step that was looked up last to the next ring slot, and looks up the one after it.
    auto send = [&]() {
        load.step(p, plan);
        const Found next = load.find();
        send_rows(found, put);
        put = put + 1 == C::STAGES ? 0 : put + 1;
        found = next;
    };
#pragma unroll 1
    for (int s = 0; s < C::STAGES - 1; ++s) send();
    if (lane == 0) {
        MergeJob job{};
        if (worker > 0) job = merge_job(plan, walk.u, worker, workers, start_of);
        p.jobs[worker] = job;
    }

    constexpr int NR = C::ROWS / 8;   // n8 tiles of rows
    uint32_t qf[NR][D / 16][2];       // Q^T: columns (rows of q) lane / 4, d 2 (lane % 4) ...
    float o[NR][D / 16][4];           // O^T: d lane / 4 (+ 8), columns 2 (lane % 4), + 1
    float m[NR][2], l[NR][2];         // of those columns
    int lo[NR][2], hi[NR][2];
    const int t2 = (lane & 3) * 2, g = lane >> 2;
    // ldmatrix rows and units: K (matrices: keys 0-7 | 8-15 | 0-7 | 8-15, units 0 | 0 | 1 | 1) and V,
    // transposed (keys 0-7 | 0-7 | 8-15 | 8-15, units 0 | 1 | 0 | 1)
    // Offset of unit c + 2 i of row r + 16 k: a register for each of a chunk's four pairs of units, and
    // constants, however the row is swizzled.
    struct Lines {
        uint32_t at[4];
        __device__ __forceinline__ Lines(int r, int c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) at[i] = uint32_t(r * C::RB) + C::unit(r, c + 2 * i);
        }
        __device__ __forceinline__ uint32_t operator()(int i, int k) const {
            constexpr int PER = C::TMA ? C::CW / 16 : 4;   // pairs of units a chunk (else: four registers, 128 bytes on)
            return at[i % PER] + uint32_t(i / PER * (C::TMA ? C::CHUNK : 128) + 16 * k * C::RB);
        }
    };
    const Lines k_at((lane & 7) + ((lane >> 3) & 1) * 8, lane >> 4), v_at((lane & 7) + (lane >> 4) * 8, (lane >> 3) & 1);

    Piece piece;
#pragma unroll 1
    while (walk_next<C::KEYS>(plan, walk, piece)) {
        const Unit &u = piece.u;
        const int tokens = min(plan.tpb, u.q.n - u.b * plan.tpb);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int i = (8 * r + t2 + c) / p.pack;
                token_keys(plan, u.q, u.b * plan.tpb + i, lo[r][c], hi[r][c]);
                m[r][c] = -INFINITY;
                l[r][c] = 0.f;
            }
            const int row = 8 * r + g, i = row / p.pack;
            const uint16_t *src = p.q + (long long)(u.q.q0 + u.b * plan.tpb + i) * p.q_stride +
                                  (long long)(u.g * p.pack + row - i * p.pack) * D + t2;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qf[r][kk][0] = i < tokens ? *reinterpret_cast<const uint32_t *>(src + 16 * kk) : 0u;
                qf[r][kk][1] = i < tokens ? *reinterpret_cast<const uint32_t *>(src + 16 * kk + 8) : 0u;
            }
#pragma unroll
            for (int n = 0; n < D / 16; ++n) o[r][n][0] = o[r][n][1] = o[r][n][2] = o[r][n][3] = 0.f;
        }
        int unit_lo, unit_hi, clear_lo, clear_hi, any_hi, any_lo;
        unit_keys(plan, u, unit_lo, unit_hi);
        // keys that every row of the unit sees: the first token sees the least, the last one loses the most
        token_keys(plan, u.q, u.b * plan.tpb, any_lo, clear_hi);
        token_keys(plan, u.q, u.b * plan.tpb + tokens - 1, clear_lo, any_hi);

#pragma unroll 1
        for (int j = piece.js; j < piece.je; ++j) {
            if (!__all_sync(0xffffffffu, wait_rows(bars + 8u * get, parity, p.plan.status))) {
                // gives up: the copies still on their way land before the warp ends (the last ones of each slot)
                for (int s = 0; s < C::STAGES; ++s)
                    if (s != get) wait_rows(bars + 8u * s, s > get ? parity : parity ^ 1u, p.plan.status);
                asm volatile("griddepcontrol.wait;" ::: "memory");
                return;
            }
            send();   // into the slot that the step before this one used
            const uint32_t tile = base + uint32_t(get * C::STAGE);
            if (++get == C::STAGES) {
                get = 0;
                parity ^= 1u;
            }
            const int first = j * C::KEYS;
            if (C::TMA && (first < unit_lo || first + C::KEYS - 1 > unit_hi)) {   // V's rows outside the unit's keys
                const int row = lane % C::KEYS, part = lane / C::KEYS, parts = 32 / C::KEYS;
                if (first + row < unit_lo || first + row > unit_hi)
#pragma unroll 1
                    for (int i = part * 16; i < C::NCH * C::RB; i += parts * 16)
                        sm100::st_shared_v4(tile + uint32_t(C::TILE + i / C::RB * C::CHUNK + row * C::RB + i % C::RB), 0u, 0u, 0u, 0u);
                sm100::fence_proxy_async_smem();   // before the slot's next copies
                __syncwarp();
            }
            // Rows that are not there need no mask either: their Q is zero and nothing of theirs is written.
            const bool masked = first < clear_lo || first + C::KEYS - 1 > clear_hi;

            // All of K's fragments are asked for before the first product, and all of V's before the softmax,
            // whose chain then covers their way from shared memory.
            float s[C::KEYS / 16][NR][4] = {};
            uint32_t f[D / 16][C::KEYS / 16][4];
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int k = 0; k < C::KEYS / 16; ++k) ldmatrix4(f[kk][k], tile + k_at(kk, k));
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
                for (int k = 0; k < C::KEYS / 16; ++k)
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma16816<C::F16>(s[k][r], f[kk][k], qf[r][kk][0], qf[r][kk][1]);
#pragma unroll
            for (int n = 0; n < D / 16; ++n)
#pragma unroll
                for (int k = 0; k < C::KEYS / 16; ++k) ldmatrix4_trans(f[n][k], tile + uint32_t(C::TILE) + v_at(n, k));
            if (masked) {
#pragma unroll
                for (int k = 0; k < C::KEYS / 16; ++k)
#pragma unroll
                    for (int r = 0; r < NR; ++r)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int key = first + 16 * k + g + 8 * (e >> 1), c = e & 1;
                            if (key < lo[r][c] || key > hi[r][c]) s[k][r][e] = -INFINITY;
                        }
            }
            bool grew = false;
            float alpha[NR][2], ref[NR][2];
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int k = 0; k < C::KEYS / 16; ++k) mx = fmaxf(mx, fmaxf(s[k][r][c], s[k][r][2 + c]));
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
                    const float now = fmaxf(m[r][c], mx * p.scale_log2);
                    ref[r][c] = now == -INFINITY ? 0.f : now;
                    alpha[r][c] = sm100::ex2_approx(m[r][c] - ref[r][c]);   // (before the first key: 0, times sums of 0)
                    grew |= now != m[r][c];
                    m[r][c] = now;
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    l[r][0] *= alpha[r][0];
                    l[r][1] *= alpha[r][1];
#pragma unroll
                    for (int n = 0; n < D / 16; ++n)
#pragma unroll
                        for (int e = 0; e < 4; ++e) o[r][n][e] *= alpha[r][e & 1];
                }
            }
            uint32_t pf[C::KEYS / 16][NR][2];   // P^T: keys 2 (lane % 4) (+ 8), columns lane / 4
#pragma unroll
            for (int k = 0; k < C::KEYS / 16; ++k)
#pragma unroll
                for (int r = 0; r < NR; ++r) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        s[k][r][e] = sm100::ex2_approx(fmaf(s[k][r][e], p.scale_log2, -ref[r][e & 1]));
                        l[r][e & 1] += s[k][r][e];
                    }
                    pf[k][r][0] = movmatrix(sm100::pack_x2<C::F16>(s[k][r][0], s[k][r][1]));
                    pf[k][r][1] = movmatrix(sm100::pack_x2<C::F16>(s[k][r][2], s[k][r][3]));
                }
#pragma unroll
            for (int k = 0; k < C::KEYS / 16; ++k)
#pragma unroll
                for (int n = 0; n < D / 16; ++n)
#pragma unroll
                    for (int r = 0; r < NR; ++r) mma16816<C::F16>(o[r][n], f[n][k], pf[k][r][0], pf[k][r][1]);
            __syncwarp();   // the slot may be filled again

        }

        // the piece is done
        {
            const bool whole = piece.js == u.js && piece.je == u.je;
            const int slot = 2 * worker + (piece.first ? 0 : 1);
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                float inv[2], lse[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float sum = l[r][c];
#pragma unroll
                    for (int x = 4; x < 32; x *= 2) sum += __shfl_xor_sync(0xffffffffu, sum, x);
                    inv[c] = sum == 0.f ? 0.f : 1.f / sum;   // (a sum that is NaN stays NaN, in both)
                    lse[c] = sum == 0.f ? -INFINITY : (m[r][c] + log2f(sum)) * kLn2;
                }
                if (whole) {   // transposed back: row g, d 2 (lane % 4), + 1
                    const int row = 8 * r + g, i = row / p.pack;
                    const long long at_row = u.q.q0 + u.b * plan.tpb + i;
                    uint16_t *dst = p.out + (at_row * p.Hq + u.g * p.pack + row - i * p.pack) * D + t2;
#pragma unroll
                    for (int n = 0; n < D / 16; ++n)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const uint32_t x = movmatrix(sm100::pack_x2<C::F16>(o[r][n][2 * h] * inv[0], o[r][n][2 * h + 1] * inv[1]));
                            if (i < tokens) *reinterpret_cast<uint32_t *>(dst + 16 * n + 8 * h) = x;
                        }
                }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = 8 * r + t2 + c, i = row / p.pack;
                    if (i >= tokens) continue;
                    if (whole) {
                        if (p.lse != nullptr && g == 0)
                            p.lse[(long long)(u.g * p.pack + row - i * p.pack) * p.plan.T + u.q.q0 + u.b * plan.tpb + i] = lse[c];
                    } else {
                        const long long at_row = (long long)slot * C::ROWS + row;
                        float *dst = p.o_part + at_row * D + g;
#pragma unroll
                        for (int n = 0; n < D / 16; ++n) {
                            dst[16 * n] = o[r][n][c] * inv[c];
                            dst[16 * n + 8] = o[r][n][2 + c] * inv[c];
                        }
                        if (g == 0) p.lse_part[at_row] = lse[c];
                    }
                }
            }
        }
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");   // ends after the tile kernel that it may run beside
}

// Merges the pieces of the unit that cut w crosses first: rows row0 .. row0 + rows - 1 of it, by the
// 8 warps of a block, rows a power of two.  With fewer rows than warps, 8 / rows warps share one, each
// taking every (8 / rows)-th round of eight pieces, and the first of them adds the shares in order.
// ROWS: rows a unit has in the workspace, in tiles of TILE (each TILE / pack tokens of `pack` heads).
// there(s): whether worker w - 1 + s did any steps.
template <int D, bool F16, int ROWS, int TILE, class There>
__device__ __forceinline__ void merge_unit(const PagedParams &p, const MergeJob &job, int w, int row0, int rows, const There &there) {
    constexpr int VEC = D % 128 == 0 ? 4 : (D % 64 == 0 ? 2 : 1), PER = (D + 32 * VEC - 1) / (32 * VEC);
    __shared__ float share[8][PER * VEC * 32 + 2];
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32;
    const int side_by_side = min(rows, 8), helpers = 8 / side_by_side, helper = warp / side_by_side;
    auto row_of = [&](int s, int row) { return (long long)(s == 0 ? job.first_slot : 2 * (w - 1 + s)) * ROWS + row; };
    for (int row = row0 + warp % side_by_side; row < row0 + rows; row += side_by_side) {
        const int tile = row / TILE, in_tile = row - tile * TILE, i = in_tile / p.pack, tq = TILE / p.pack;
        const int token = tile * tq + i, head = job.g * p.pack + in_tile - i * p.pack;
        const bool real = i < tq && token < job.tokens;
        float m = -INFINITY, sum = 0.f;
        float acc[PER][VEC] = {};
        for (int base = 8 * helper; real && base < job.parts; base += 8 * helpers) {
            const int n = min(8, job.parts - base);
            const bool mine = lane < n && there(base + lane);
            const unsigned alive = __ballot_sync(0xffffffffu, mine);
            const float ls = mine ? p.lse_part[row_of(base + lane, row)] : -INFINITY;
            float x[8][PER][VEC];
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int e = 0; e < PER; ++e) {
                    const int col = (e * 32 + lane) * VEC;
                    const float *src = p.o_part + row_of(base + t, row) * D + col;
#pragma unroll
                    for (int v = 0; v < VEC; ++v) x[t][e][v] = 0.f;
                    if ((alive >> t & 1u) && col < D) {
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
            float mx = ls;
#pragma unroll
            for (int o = 4; o > 0; o /= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            const float now = fmaxf(m, __shfl_sync(0xffffffffu, mx, 0));
            if (now == -INFINITY && !__any_sync(0xffffffffu, isnan(ls))) continue;   // (a NaN makes all weights NaN, and the row)
            const float wl = __expf(ls - now), keep = __expf(m - now);
            m = now;
            sum *= keep;
#pragma unroll
            for (int e = 0; e < PER; ++e)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[e][v] *= keep;
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                const float wt = __shfl_sync(0xffffffffu, wl, t);
                sum += wt;
#pragma unroll
                for (int e = 0; e < PER; ++e)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) acc[e][v] = fmaf(wt, x[t][e][v], acc[e][v]);
            }
        }
        if (helpers > 1) {   // (uniform over the block, and then every warp has one row)
#pragma unroll
            for (int e = 0; e < PER; ++e)
#pragma unroll
                for (int v = 0; v < VEC; ++v) share[warp][(e * VEC + v) * 32 + lane] = acc[e][v];
            if (lane == 0) {
                share[warp][PER * VEC * 32] = m;
                share[warp][PER * VEC * 32 + 1] = sum;
            }
            __syncthreads();
            float all = m;
            for (int h = 1; helper == 0 && h < helpers; ++h) all = fmaxf(all, share[warp + h * side_by_side][PER * VEC * 32]);
            const float keep = all == -INFINITY ? 0.f : __expf(m - all);
            sum *= keep;
#pragma unroll
            for (int e = 0; e < PER; ++e)
#pragma unroll
                for (int v = 0; v < VEC; ++v) acc[e][v] *= keep;
            for (int h = 1; helper == 0 && h < helpers; ++h) {
                const float *other = share[warp + h * side_by_side];
                const float wt = all == -INFINITY ? 0.f : __expf(other[PER * VEC * 32] - all);
                sum = fmaf(wt, other[PER * VEC * 32 + 1], sum);
#pragma unroll
                for (int e = 0; e < PER; ++e)
#pragma unroll
                    for (int v = 0; v < VEC; ++v) acc[e][v] = fmaf(wt, other[(e * VEC + v) * 32 + lane], acc[e][v]);
            }
            m = all;
        }
        if (!real || helper != 0) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
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
        if (p.lse != nullptr && lane == 0) p.lse[(long long)head * p.plan.T + at] = sum == 0.f ? -INFINITY : m + logf(sum);
    }
}

// The few-rows kernel's pieces at cut w.
template <int D, bool F16, int ROWS>
__device__ __forceinline__ void merge_rows(const PagedParams &p, int w) {
    const MergeJob job = p.jobs[w];
    if (job.parts == 0) return;
    int rows = 1;
    while (rows < job.tokens * p.pack) rows *= 2;
    merge_unit<D, F16, ROWS, ROWS>(p, job, w, 0, rows, [](int) { return true; });
}

// The merge of a call that has pieces of few rows only: one block a cut.
template <int D, bool F16, int ROWS>
__global__ void __launch_bounds__(256) fa_paged_merge_rows_kernel(const __grid_constant__ PagedParams p) {
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the pieces and jobs are written
    merge_rows<D, F16, ROWS>(p, int(blockIdx.x) + 1);
}

}  // namespace fa
