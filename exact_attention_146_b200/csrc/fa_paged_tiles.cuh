// fa_paged_tiles.cuh -- attention over a paged cache for chunks of new tokens, on the tensor cores
// (tcgen05): the roles and tilings of the dense forward (fa_kernel.cuh) over gathered pages.
//
// Bound by the tensor cores: a unit's 256 rows (NQT = 2) make 256 flops a byte of K and V.  What is
// different from the dense forward:
//   * a row tile stacks `pack` query heads of one KV head over 128 / pack tokens (flat row
//     token * pack + head), so a short chunk still fills it, and the heads share every K/V load;
//   * every CTA gets the same number of key-tile steps (plan_schedule): whole units first, then a range of
//     the rest of the line, so that a single long request keeps every SM busy to the end.  A range
//     ends inside at most two units; their pieces go to the workspace and the merge kernel combines them;
//   * K and V tiles are put together from the largest power-of-two runs of slots that divide a page
//     (8 rows at least: one swizzle atom), one TMA box each; runs that no row of the unit sees take a
//     block index past the cache and are filled with zeros by the copy engine.  Slots of the last run
//     behind the request's last key may hold anything (0 x NaN = NaN in P V), so the MMA warp zeroes
//     those rows of V in shared memory before it multiplies; K needs nothing, its scores are masked.
//   * one warp plans the units for the other roles (a queue in shared memory): the plan's arithmetic in each
//     role had cost 2 us a unit and, by its size, the instruction cache (78 % hits; 89 % now).
// Measured (B200, in a CUDA graph): 4096 new tokens over 28672 keys (Hq 32, Hkv 8, d 128) 1.71 ms, 1206 TFLOP/s; 8 requests
// of up to 512 new tokens over 8k 203 us, of which 2.0 to 2.2 us for each 256 rows x 128 keys.
#pragma once

#include "fa_kernel.cuh"
#include "fa_paged_rows.cuh"

namespace fa {

struct PagedTileParams : PagedParams {
    int tq;            // tokens a row tile: 128 / pack
    long long *cuts;   // workspace: the cuts of the line, each CTA's copy (kMaxPagedCtas + 1 places)
};

// The units and steps before each of 64 segments of the requests: what the planner finds its units by.
constexpr int kCoarse = 64;
constexpr int kQueue = 4;   // units planned ahead

// A unit as one CTA does it, made by the planner warp for the other roles.
struct PagedUnit {
    int js[2], je[2];          // key tiles each row tile visits here (empty: js == je)
    int j_lo, j_hi;            // their union
    int row0, tokens;          // first row of q, new tokens (both row tiles); tokens < 0: no more units
    int pos0;                  // position of the first token: its last visible key if causal
    int L, r, g;               // keys of the request, the request, the head group
    int lo, hi;                // keys that some row sees
    int slot;                  // the piece's place in the workspace; -1: the whole unit is done here
    int pad;
};

// Shared memory of the plan, between the pipeline's barriers and the staging and behind it: the
// queue's barriers (full, empty), its entries, and the coarse counts.
template <class C>
struct PlanSmem {
    static constexpr int BARS = C::SMEM_MISC + 16;
    static constexpr int UNITS = BARS + 2 * kQueue * 8;
    static constexpr int COARSE = UNITS + kQueue * int(sizeof(PagedUnit));
    static constexpr int STEPS = C::SMEM_OST + 4 * C::NQT * C::OST_BYTES;   // behind the staging
    static constexpr int RANGE = STEPS + (kCoarse + 1) * 8;                // this CTA's cut and the cuts beside it
    static constexpr int BYTES = C::SMEM_BYTES + 1024;
    static_assert(COARSE + (kCoarse + 1) * 4 <= C::SMEM_OST, "the plan lies before the staging");
    static_assert(RANGE + 64 + 1024 <= BYTES && BYTES <= 232448, "shared memory budget");
    static_assert(BARS % 8 == 0 && sizeof(PagedUnit) == 64, "alignment");
    // who hands an entry back: the TMA warp, the MMA warp and each softmax warp
    static constexpr int READERS = 2 + C::SOFTMAX_WARPS;
};
constexpr int kSiteUnitFull = 14, kSiteUnitEmpty = 15;   // waits of the queue (bits 8..15 of the status word)

// A role's end of the queue.
template <class C, int ROLE>
struct PagedUnits {
    using Unit = PagedUnit;
    uint32_t sbase;
    uint8_t *smem;
    const Ctl &ctl;
    int box_rows;
    uint32_t n;

    __device__ __forceinline__ bool next(PagedUnit &w) {
        const int i = int(n % kQueue);
        const uint32_t bars = sbase + PlanSmem<C>::BARS;
        if (!warp_wait_bar<ROLE>(bars + 8u * i, (n / kQueue) & 1u, ctl, kSiteUnitFull)) return false;
        w = *reinterpret_cast<const PagedUnit *>(smem + PlanSmem<C>::UNITS + i * int(sizeof(PagedUnit)));
        __syncwarp();
        if (threadIdx.x % 32 == 0) sm100::mbar_arrive(bars + 8u * (kQueue + i));
        ++n;
        return w.tokens >= 0;
    }

    // Rows of the V tile from the request's length to the end of the box that holds it.
    __device__ __forceinline__ void v_landed(const PagedUnit &w, int j, uint32_t tile) const {
        const int a = w.L - j * C::BC;
        if (a <= 0 || a >= C::BC || a % box_rows == 0) return;
        const int b = (a / box_rows + 1) * box_rows;
#pragma unroll 1
        for (int c = 0; c < C::NCH; ++c)
#pragma unroll 1
            for (int i = a * C::RB + int(threadIdx.x % 32) * 16; i < b * C::RB; i += 512)
                sm100::st_shared_v4(tile + uint32_t(c * C::KV_CHUNK + i), 0u, 0u, 0u, 0u);
        sm100::fence_proxy_async_smem();   // the MMA reads through the async proxy
        __syncwarp();
    }
};

// The planner: one warp walks this CTA's units (its whole ones, then its range of the line) and queues
// them, so that the other roles do none of the plan's arithmetic.
template <class C>
__device__ void paged_plan_role(const PagedTileParams &p, int seg, int whole_units, uint32_t sbase, uint8_t *smem, const Ctl &ctl) {
    const int lane = int(threadIdx.x) % 32, cta = int(blockIdx.x);
    const int *units_before = reinterpret_cast<const int *>(smem + PlanSmem<C>::COARSE);
    const long long *steps_before = reinterpret_cast<const long long *>(smem + PlanSmem<C>::STEPS);
    const long long *range = reinterpret_cast<const long long *>(smem + PlanSmem<C>::RANGE);
    const long long x0 = range[0], x1 = range[1], total = range[2];
    const uint32_t bars = sbase + PlanSmem<C>::BARS;
    Walk walk{};
    bool found = false;
    int k = cta;
#pragma unroll 1
    for (uint32_t n = 0;; ++n) {
        PagedUnit w{};
        w.tokens = -1;
        Piece piece{};
        if (k < whole_units) {
            piece.u = plan_unit<C::BC>(p.plan, units_before, kCoarse, seg, k);
            piece.js = piece.u.js;
            piece.je = piece.u.je;
            k += p.plan.workers;
            w.tokens = 0;
        } else {
            if (!found) {   // where the range begins, and what the merge has to do at that cut
                found = true;
                MergeJob job{};
                if (x0 < total) {
                    walk.u = plan_find<C::BC>(p.plan, steps_before, kCoarse, seg, x0);
                    walk.o = x0 - walk.u.begin;
                    walk.left = x1 - x0;
                    walk.first = true;
                    if (cta > 0) job = merge_job(p.plan, walk.u, cta, p.plan.workers, [&](int c) { return p.cuts[cta * (kMaxPagedCtas + 1) + c]; });
                }
                if (lane == 0) p.jobs[cta] = job;
            }
            if (walk_next<C::BC>(p.plan, walk, piece)) w.tokens = 0;
        }
        if (w.tokens == 0) {
            const Unit &u = piece.u;
            const long long diag = (long long)u.q.L - u.q.n;
            const int tok0 = u.b * p.plan.tpb;
            w.slot = piece.js == u.js && piece.je == u.je ? -1 : 2 * cta + (piece.first ? 0 : 1);
            w.row0 = u.q.q0 + tok0;
            w.tokens = min(u.q.n - tok0, p.plan.tpb);
            w.pos0 = int(tok0 + diag);
            w.L = u.q.L;
            w.r = u.r;
            w.g = u.g;
            unit_keys(p.plan, u, w.lo, w.hi);
            w.j_lo = 0x7fffffff;
#pragma unroll
            for (int t = 0; t < C::NQT; ++t) {
                const int t0 = t * p.tq, t1 = min(w.tokens, t0 + p.tq);
                if (t0 >= t1) continue;
                const int last = p.plan.causal ? w.pos0 + t1 - 1 : w.L - 1;
                // in 64 bits: a position below 0 (more new tokens than keys) less a window near 2^31
                const long long from = p.plan.window > 0 ? (long long)w.pos0 + t0 - p.plan.window + 1 : 0;
                const int js = max(int(max(from, 0LL)) / C::BC, piece.js), je = min(max(last, 0) / C::BC + 1, piece.je);
                if (je <= js) continue;
                w.js[t] = js;
                w.je[t] = je;
                w.j_lo = min(w.j_lo, js);
                w.j_hi = max(w.j_hi, je);
            }
            if (w.j_hi == 0) w.j_lo = 0;
        }
        const int i = int(n % kQueue);
        if (!warp_wait_bar<kRoleControl>(bars + 8u * (kQueue + i), ((n / kQueue) & 1u) ^ 1u, ctl, kSiteUnitEmpty)) return;
        if (lane == 0) {
            *reinterpret_cast<PagedUnit *>(smem + PlanSmem<C>::UNITS + i * int(sizeof(PagedUnit))) = w;
            sm100::mbar_arrive(bars + 8u * i);
        }
        if (w.tokens < 0) return;
    }
}

template <class C>
__device__ void paged_producer_role(const CUtensorMap *tm_q, const CUtensorMap *tm_k, const CUtensorMap *tm_v,
                                    const PagedTileParams &p, PagedUnits<C, kRoleControl> units, uint32_t sbase, const Ctl &ctl) {
    auto bar = [&](int i) { return sbase + C::SMEM_BAR + 8u * uint32_t(i); };
    sm100::prefetch_tensormap(tm_q);
    sm100::prefetch_tensormap(tm_k);
    sm100::prefetch_tensormap(tm_v);
    const int lane = int(threadIdx.x) % 32;
    const int boxes = C::BC / p.run;
    const uint32_t q_bytes = uint32_t(C::NCH * C::RB * p.tq * p.pack);
    uint32_t kv_cnt = 0;
    uint32_t qcnt[2] = {0, 0};
    bool ok = true;
    PagedUnit w;
    while (ok && units.next(w)) {
        if (w.j_hi == w.j_lo) continue;
        const int kvh = w.g * p.pack / p.n_rep;
        const int *table = p.table + w.r * p.table_stride;
        // Block and slot of box `lane` of key tile j (a block past the cache: zeros).
        auto find_box = [&](int j, int &block, int &slot) {
            const int key = j * C::BC + lane * p.run;
            const bool seen = lane < boxes && key <= w.hi && key + p.run > w.lo;
            const int page = seen ? key / p.page : 0;
            slot = seen ? key - page * p.page : 0;
            block = seen ? __ldg(table + page) : p.num_blocks;
        };
        auto slot_named = [&](int j) {   // the table was asked for this box
            const int key = j * C::BC + lane * p.run;
            return lane < boxes && key <= w.hi && key + p.run > w.lo;
        };
        int block, slot;
        find_box(w.j_lo, block, slot);
#pragma unroll
        for (int t = 0; t < C::NQT; ++t) {
            if (!ok || w.je[t] == w.js[t]) continue;
            const int qb = int(qcnt[t] % C::NQB);
            if (!warp_wait_bar<kRoleControl>(bar(C::B_QEMPTY + t * C::NQB + qb), ((qcnt[t] / C::NQB) & 1u) ^ 1u, ctl, kSiteQEmpty)) {
                ok = false;
                break;
            }
            ++qcnt[t];
            const uint32_t fb = bar(C::B_QFULL + t * C::NQB + qb);
            sm100::mbar_arrive_expect_tx_elected(fb, q_bytes);
            const uint32_t dst = sbase + C::SMEM_Q + (t * C::NQB + qb) * C::Q_TILE;
#pragma unroll
            for (int c = 0; c < C::NCH; ++c)
                sm100::tma_load_4d_elected(dst + c * C::Q_CHUNK, tm_q, fb, c * C::CW, w.g * p.pack, w.row0 + t * p.tq, 0);
        }
        for (int j = w.j_lo; ok && j < w.j_hi; ++j) {
            int next_block = 0, next_slot = 0;
            if (j + 1 < w.j_hi) find_box(j + 1, next_block, next_slot);   // looked up while this tile's slots are waited for
            if (block < 0 || block > p.num_blocks || (block == p.num_blocks && slot_named(j))) {
                fa_host::report_range(p.plan.status, fa_host::kSiteTableId, w.r);
                block = p.num_blocks;
            }
#pragma unroll 1
            for (int which = 0; which < 2; ++which) {
                const int s = int(kv_cnt % C::NS);
                if (!warp_wait_bar<kRoleControl>(bar(C::B_EMPTY + s), ((kv_cnt / C::NS) & 1u) ^ 1u, ctl, kSiteKvEmpty)) { ok = false; break; }
                const uint32_t fb = bar(C::B_FULL + s);
                sm100::mbar_arrive_expect_tx_elected(fb, C::KV_TILE);
                const uint32_t dst = sbase + C::SMEM_KV + s * C::KV_TILE;
                const CUtensorMap *m = which ? tm_v : tm_k;
#pragma unroll 1
                for (int i = 0; i < boxes; ++i) {
                    const int b = __shfl_sync(0xffffffffu, block, i), sl = __shfl_sync(0xffffffffu, slot, i);
                    const int c1 = p.slot_first ? sl : kvh, c2 = p.slot_first ? kvh : sl;
#pragma unroll
                    for (int c = 0; c < C::NCH; ++c)
                        sm100::tma_load_4d_elected(dst + uint32_t(c * C::KV_CHUNK + i * p.run * C::RB), m, fb, c * C::CW, c1, c2, b);
                }
                ++kv_cnt;
            }
            block = next_block;
            slot = next_slot;
        }
    }
    if (!ok || *ctl.abort_flag) producer_unwind<C>(sbase, kv_cnt, qcnt, ctl);
}

template <class C>
__device__ void paged_softmax_role(const PagedTileParams &p, PagedUnits<C, kRoleSoftmax> units, uint32_t sbase, uint32_t tmem, const Ctl &ctl,
                                   int warp, int lane) {
    auto bar = [&](int i) { return sbase + C::SMEM_BAR + 8u * uint32_t(i); };
    constexpr int D = C::D;
    const int t = warp / 4, quarter = warp % 4;
    const int row_in_tile = quarter * 32 + lane;
    const int i_tok = row_in_tile / p.pack, i_head = row_in_tile - i_tok * p.pack;
    const uint32_t o_taddr = tmem + (uint32_t(quarter * 32) << 16) + uint32_t(C::O_COL0 + t * C::OST);
    uint32_t scnt = 0, ocnt = 0, ofin = 0;
    PagedUnit w;
    while (units.next(w)) {
        const int js = w.js[t], je = w.je[t], nk = je - js;
        const int token = t * p.tq + i_tok;            // of the unit
        const int at0 = w.pos0 + t * p.tq, at = at0 + i_tok;   // positions: the row tile's first token, this row's
        const bool window = p.plan.window > 0;
        // (rows before the first key see none: their lower bound does not matter, and -1 keeps it within 32 bits)
        const RowKeys keys{w.L, p.plan.causal ? at : 0x7fffffff, window ? max(at, -1) - p.plan.window + 1 : -0x7fffffff,
                           p.plan.causal ? at0 : 0x7fffffff, window ? max(at0 + p.tq - 1, -1) - p.plan.window + 1 : -0x7fffffff};
        float m_ref = -INFINITY, l = 0.f;
        if (!softmax_tiles<C>(sbase, tmem, ctl, t, quarter, p.scale_log2, keys, js, je, scnt, ocnt, m_ref, l)) goto unwind;
        if (nk > 0) {
            if (!warp_wait_bar(bar(C::B_OFINAL + t), ofin & 1u, ctl, kSiteOFinal)) goto unwind;
            ++ofin;
            sm100::tc_fence_after_sync();
        }
        ocnt += uint32_t(nk);
        {
            const float inv_l = l == 0.f ? 0.f : 1.f / l;   // (a sum that is NaN stays NaN, in both)
            const float lse = l == 0.f ? -INFINITY : (m_ref + log2f(l)) * kLn2;
            const bool store = i_tok < p.tq && token < w.tokens;
            const bool whole = w.slot < 0;
            const long long row = w.row0 + token;
            const int head = w.g * p.pack + i_head;
            const long long o_off = store ? (row * p.Hq + head) * D : -1;
            const long long piece = ((long long)w.slot * C::NQT + t) * kBlockQ + row_in_tile;
            if (whole && C::OSTAGE) {
                // 64 columns a pass through this warp's staging buffer (rows of 128 bytes, 16-byte unit i
                // of row r at i ^ (r % 8)), so that eight lanes write one row's 128 bytes together.
                const uint32_t stage = sbase + uint32_t(C::SMEM_OST + warp * C::OST_BYTES);
#pragma unroll
                for (int c2 = 0; c2 < (D + 63) / 64; ++c2) {
                    uint32_t pk[32];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t o[32];
                        if (nk > 0) {
                            sm100::tmem_ld32_sync(o_taddr + uint32_t(64 * c2 + 32 * h), o);
                        } else {
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = 0u;
                        }
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            pk[16 * h + i] = sm100::pack_x2<C::F16>(__uint_as_float(o[2 * i]) * inv_l, __uint_as_float(o[2 * i + 1]) * inv_l);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sm100::st_shared_v4(stage + uint32_t(lane * 128 + ((i ^ (lane & 7)) * 16)), pk[4 * i], pk[4 * i + 1],
                                            pk[4 * i + 2], pk[4 * i + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = 4 * i + lane / 8, col = 64 * c2 + 8 * (lane % 8);
                        const long long off = __shfl_sync(0xffffffffu, o_off, rr);
                        uint32_t x[4];
                        sm100::ld_shared_v4(x, stage + uint32_t(rr * 128 + (((lane % 8) ^ (rr & 7)) * 16)));
                        if (off >= 0 && col < D) *reinterpret_cast<uint4 *>(p.out + off + col) = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    __syncwarp();
                }
            } else if (!whole && C::OSTAGE) {
                // the piece's fp32 rows, 32 columns a pass through the same buffer
                const uint32_t stage = sbase + uint32_t(C::SMEM_OST + warp * C::OST_BYTES);
                const unsigned stored = __ballot_sync(0xffffffffu, store);
                float *dst = p.o_part + (piece - lane) * D;   // the warp's first row
#pragma unroll 1
                for (int c = 0; c < C::O_CHUNKS; ++c) {
                    uint32_t o[32];
                    if (nk > 0) {
                        sm100::tmem_ld32_sync(o_taddr + uint32_t(32 * c), o);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * inv_l);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        sm100::st_shared_v4(stage + uint32_t(lane * 128 + ((i ^ (lane & 7)) * 16)), o[4 * i], o[4 * i + 1], o[4 * i + 2],
                                            o[4 * i + 3]);
                    __syncwarp();
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int rr = 4 * i + lane / 8, col = 32 * c + 4 * (lane % 8);
                        uint32_t x[4];
                        sm100::ld_shared_v4(x, stage + uint32_t(rr * 128 + (((lane % 8) ^ (rr & 7)) * 16)));
                        if ((stored >> rr & 1u) && col < D)
                            *reinterpret_cast<uint4 *>(dst + rr * D + col) = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                    __syncwarp();
                }
            } else {
                // d = 32: a row's 64 (whole) or 128 bytes by its own thread
#pragma unroll
                for (int c = 0; c < C::O_CHUNKS; ++c) {
                    uint32_t o[32];
                    if (nk > 0) {
                        sm100::tmem_ld32_sync(o_taddr + uint32_t(32 * c), o);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = 0u;
                    }
                    if (!store) continue;
                    if (!whole) {
                        float *dst = p.o_part + piece * D + 32 * c;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            *reinterpret_cast<float4 *>(dst + 4 * i) =
                                make_float4(__uint_as_float(o[4 * i]) * inv_l, __uint_as_float(o[4 * i + 1]) * inv_l,
                                            __uint_as_float(o[4 * i + 2]) * inv_l, __uint_as_float(o[4 * i + 3]) * inv_l);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                x[e] = sm100::pack_x2<C::F16>(__uint_as_float(o[8 * i + 2 * e]) * inv_l, __uint_as_float(o[8 * i + 2 * e + 1]) * inv_l);
                            *reinterpret_cast<uint4 *>(p.out + o_off + 32 * c + 8 * i) = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    }
                }
            }
            sm100::tc_fence_before_sync();
            sm100::mbar_arrive(bar(C::B_OEMPTY + t));
            if (store) {
                if (!whole) p.lse_part[piece] = lse;
                else if (p.lse != nullptr) p.lse[(long long)head * p.plan.T + row] = lse;
            }
        }
    }
unwind:
    sm100::tmem_st_wait();
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
fa_paged_tiles_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedTileParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = sm100::smem_u32(smem);
    const int warp = int(threadIdx.x) / 32, lane = int(threadIdx.x) % 32;
    uint32_t *tmem_holder = reinterpret_cast<uint32_t *>(smem + C::SMEM_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::SMEM_MISC + 4);
    const Ctl ctl{abort_flag, p.plan.status, kWaitLimitNs};
    // The few-rows kernel of a mixed call takes the SMs as this one's CTAs end; then the merge.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    if (threadIdx.x == 0) {
        init_barriers<C>(sbase);
        for (int i = 0; i < kQueue; ++i) {
            sm100::mbar_init(sbase + PlanSmem<C>::BARS + 8u * i, 1);
            sm100::mbar_init(sbase + PlanSmem<C>::BARS + 8u * (kQueue + i), PlanSmem<C>::READERS);
        }
        *abort_flag = 0;
        sm100::fence_mbar_init();
    }
    if (warp == 0) {
        sm100::tmem_alloc(sm100::smem_u32(tmem_holder), C::TMEM_COLS);
        sm100::tmem_relinquish();
    }
    // The plan uses the K/V ring's memory before the first copy goes there, but for the coarse counts.
    struct Plan {
        PlanScan<C::THREADS> scan;
        long long cuts[kMaxPagedCtas + 1];
    };
    static_assert(sizeof(Plan) <= size_t(C::NS) * C::KV_TILE, "plan in the ring");
    static_assert(C::THREADS % kCoarse == 0 && C::THREADS > kMaxPagedCtas, "segments, and a thread for each cut");
    Plan &plan = *reinterpret_cast<Plan *>(smem + C::SMEM_KV);
    const int tid = int(threadIdx.x), seg = (p.plan.R + C::THREADS - 1) / C::THREADS, cta = int(blockIdx.x);
    const long long total = plan_scan<C::BC>(p.plan, plan.scan, tid, cta == 0 && p.say != 0);
    const int rounds = plan_schedule<C::BC>(p.plan, plan.scan, total, plan.cuts, tid);
    if (tid <= kCoarse) {
        reinterpret_cast<int *>(smem + PlanSmem<C>::COARSE)[tid] = plan.scan.seg_units[tid * (C::THREADS / kCoarse)];
        reinterpret_cast<long long *>(smem + PlanSmem<C>::STEPS)[tid] = plan.scan.seg_start[tid * (C::THREADS / kCoarse)];
    }
    if (tid == 0) {
        long long *range = reinterpret_cast<long long *>(smem + PlanSmem<C>::RANGE);
        range[0] = plan.cuts[cta];
        range[1] = plan.cuts[cta + 1];
        range[2] = total;
    }
    if (tid <= p.plan.workers) p.cuts[cta * (kMaxPagedCtas + 1) + tid] = plan.cuts[tid];   // the planner and the merge read them
    __syncthreads();
    sm100::fence_proxy_async_smem();   // those reads and writes come before the copies into the ring
    sm100::tc_fence_before_sync();
    __syncthreads();
    sm100::tc_fence_after_sync();
    const uint32_t tmem = *tmem_holder;

    if (warp < C::SOFTMAX_WARPS) {
        if constexpr (C::REALLOC_REGS) sm100::regs_increase<C::SOFTMAX_REGS>();
        paged_softmax_role<C>(p, PagedUnits<C, kRoleSoftmax>{sbase, smem, ctl, p.run, 0}, sbase, tmem, ctl, warp, lane);
    } else {
        if constexpr (C::REALLOC_REGS) sm100::regs_decrease<C::CONTROL_REGS>();
        const PagedUnits<C, kRoleControl> units{sbase, smem, ctl, p.run, 0};
        if (warp == C::TMA_WARP) paged_producer_role<C>(&tm_q, &tm_k, &tm_v, p, units, sbase, ctl);
        else if (warp == C::MMA_WARP) mma_role<C>(units, sbase, tmem, ctl);
        else if (warp == C::MMA_WARP + 1)
            paged_plan_role<C>(p, seg * (C::THREADS / kCoarse), rounds * p.plan.workers, sbase, smem, ctl);
    }
    __syncwarp();

    sm100::tc_fence_before_sync();
    __syncthreads();
    sm100::tc_fence_after_sync();
    if (warp == 0) sm100::tmem_dealloc(tmem, C::TMEM_COLS);
}

// The merge after the tile kernel: blocks of 32 rows a cut, then (where the call has a kernel of few
// rows too) that one's cuts.
template <class C, int FEW>
__global__ void __launch_bounds__(256) fa_paged_merge_kernel(const __grid_constant__ PagedTileParams p,
                                                             const __grid_constant__ PagedParams few) {
    constexpr int kRows = C::NQT * kBlockQ, kPer = kRows / 32;
    const int tile_blocks = (p.plan.workers - 1) * kPer, i = int(blockIdx.x);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the pieces, cuts and jobs are written
    if (i < tile_blocks) {
        const int w = i / kPer + 1;
        const MergeJob job = p.jobs[w];
        if (job.parts > 0)
            merge_unit<C::D, C::F16, kRows, kBlockQ>(p, job, w, i % kPer * 32, 32, [&](int s) { return p.cuts[w - 1 + s] < p.cuts[w + s]; });
    } else {
        merge_rows<C::D, C::F16, FEW>(few, i - tile_blocks + 1);
    }
}

}  // namespace fa
