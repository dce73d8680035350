// fa_paged_tiles.cuh -- attention over a paged cache for chunks of new tokens, on the tensor cores
// (tcgen05): the roles and tilings of the dense forward (fa_kernel.cuh) over gathered pages.
//
// Bound by the tensor cores: a unit's 256 rows (NQT = 2) make 256 flops a byte of K and V.  What is
// different from the dense forward:
//   * a row tile stacks `pack` query heads of one KV head over 128 / pack tokens (flat row
//     token * pack + head), so a short chunk still fills it, and the heads share every K/V load;
//   * the work is one line of key-tile steps cut evenly over the CTAs (fa_paged_plan.cuh): a single
//     long request keeps every SM busy to the end.  A CTA cuts at most two units, their pieces go to
//     the workspace and the merge kernel combines them;
//   * K and V tiles are put together from the largest power-of-two runs of slots that divide a page
//     (8 rows at least: one swizzle atom), one TMA box each; runs that no row of the unit sees take a
//     block index past the cache and are filled with zeros by the copy engine.  Slots of the last run
//     behind the request's last key may hold anything (0 x NaN = NaN in P V), so the MMA warp zeroes
//     those rows of V in shared memory before it multiplies; K needs nothing, its scores are masked.
#pragma once

#include "fa_kernel.cuh"
#include "fa_paged_rows.cuh"

namespace fa {

struct PagedTileParams : PagedParams {
    int tq;            // tokens a row tile: 128 / pack
    int box_rows;      // slots a K/V box
    int slot_first;    // the tensor map's second axis is the slot (else the head)
};

// A unit as one CTA does it: its key tiles clipped to the CTA's range.
struct PagedUnit {
    Unit u;
    int js[2], je[2], j_lo, j_hi;   // as UnitInfo
    bool whole;                     // the unit lies wholly in this range
    int slot;                       // else: where in the workspace its piece goes
};

template <class C>
struct PagedUnits {
    using Unit = PagedUnit;
    const PagedTileParams &p;
    Cursor at;                      // the next piece
    bool first;                     // it begins where the range does

    __device__ __forceinline__ bool next(PagedUnit &w) {
        if (at.left <= 0) return false;
        const int pjs = at.j, pje = min(at.u.je, at.j + at.left);
        w.u = at.u;
        w.whole = pjs == at.u.js && pje == at.u.je;
        w.slot = 2 * int(blockIdx.x) + (first ? 0 : 1);
        const long long diag = (long long)w.u.q.L - w.u.q.n;
        w.j_lo = 0x7fffffff;
        w.j_hi = 0;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            int js = 0, je = 0;
            const int tok0 = w.u.b * p.plan.tpb + t * p.tq, tok1 = min(w.u.q.n, tok0 + p.tq);
            if (t < C::NQT && tok0 < tok1) {
                const long long last = p.plan.causal ? tok1 - 1 + diag : (long long)w.u.q.L - 1;
                const long long from = p.plan.window > 0 ? tok0 + diag - p.plan.window + 1 : 0;
                js = max(int(max(from, 0LL) / C::BC), pjs);
                je = min(int(max(last, 0LL) / C::BC) + 1, pje);
                if (je <= js) js = je = 0;
            }
            w.js[t] = js;
            w.je[t] = je;
            if (je > js) {
                w.j_lo = min(w.j_lo, js);
                w.j_hi = max(w.j_hi, je);
            }
        }
        if (w.j_hi == 0) w.j_lo = 0;
        at.left -= pje - pjs;
        first = false;
        if (at.left > 0) {
            plan_next<C::BC>(p.plan, at.u);
            at.j = at.u.js;
        }
        return true;
    }

    // Rows of the V tile from the request's length to the end of the box that holds it.
    __device__ __forceinline__ void v_landed(const PagedUnit &w, int j, uint32_t tile) const {
        const int a = w.u.q.L - j * C::BC;
        if (a <= 0 || a >= C::BC || a % p.box_rows == 0) return;
        const int b = (a / p.box_rows + 1) * p.box_rows;
#pragma unroll
        for (int c = 0; c < C::NCH; ++c)
            for (int i = a * C::RB + int(threadIdx.x % 32) * 16; i < b * C::RB; i += 512)
                sm100::st_shared_v4(tile + uint32_t(c * C::KV_CHUNK + i), 0u, 0u, 0u, 0u);
        sm100::fence_proxy_async_smem();   // the MMA reads through the async proxy
        __syncwarp();
    }
};

template <class C>
__device__ void paged_producer_role(const CUtensorMap *tm_q, const CUtensorMap *tm_k, const CUtensorMap *tm_v,
                                    const PagedTileParams &p, PagedUnits<C> units, uint32_t sbase, const Ctl &ctl) {
    auto bar = [&](int i) { return sbase + C::SMEM_BAR + 8u * uint32_t(i); };
    sm100::prefetch_tensormap(tm_q);
    sm100::prefetch_tensormap(tm_k);
    sm100::prefetch_tensormap(tm_v);
    const int lane = int(threadIdx.x) % 32;
    const int boxes = C::BC / p.box_rows;
    const uint32_t q_bytes = uint32_t(C::NCH * C::RB * p.tq * p.pack);
    uint32_t kv_cnt = 0;
    uint32_t qcnt[2] = {0, 0};
    bool ok = true;
    PagedUnit w;
    while (ok && units.next(w)) {
        if (w.j_hi == w.j_lo) continue;
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
                sm100::tma_load_4d_elected(dst + c * C::Q_CHUNK, tm_q, fb, c * C::CW, w.u.g * p.pack,
                                           w.u.q.q0 + w.u.b * p.plan.tpb + t * p.tq, 0);
        }
        int lo, hi;
        unit_keys(p.plan, w.u, lo, hi);
        const int kvh = w.u.g * p.pack / p.n_rep;
        // Block and slot of box `lane` of key tile j (a block past the cache: zeros).
        auto find_box = [&](int j, int &block, int &slot) {
            block = p.num_blocks;
            slot = 0;
            const int key = j * C::BC + lane * p.box_rows;
            if (lane >= boxes || key > hi || key + p.box_rows <= lo) return;
            const int page = key / p.page;
            const int id = __ldg(p.table + w.u.r * p.table_stride + page);
            slot = key - page * p.page;
            if (id >= 0 && id < p.num_blocks) block = id;
            else fa_host::report_range(p.plan.status, fa_host::kSiteTableId, w.u.r);
        };
        int block, slot;
        find_box(w.j_lo, block, slot);
        for (int j = w.j_lo; ok && j < w.j_hi; ++j) {
            int next_block = 0, next_slot = 0;
            if (j + 1 < w.j_hi) find_box(j + 1, next_block, next_slot);   // looked up while this tile's slots are waited for
#pragma unroll
            for (int which = 0; which < 2; ++which) {
                const int s = int(kv_cnt % C::NS);
                if (!warp_wait_bar<kRoleControl>(bar(C::B_EMPTY + s), ((kv_cnt / C::NS) & 1u) ^ 1u, ctl, kSiteKvEmpty)) { ok = false; break; }
                const uint32_t fb = bar(C::B_FULL + s);
                sm100::mbar_arrive_expect_tx_elected(fb, C::KV_TILE);
                const uint32_t dst = sbase + C::SMEM_KV + s * C::KV_TILE;
                const CUtensorMap *m = which ? tm_v : tm_k;
                for (int i = 0; i < boxes; ++i) {
                    const int b = __shfl_sync(0xffffffffu, block, i), sl = __shfl_sync(0xffffffffu, slot, i);
                    const int c1 = p.slot_first ? sl : kvh, c2 = p.slot_first ? kvh : sl;
#pragma unroll
                    for (int c = 0; c < C::NCH; ++c)
                        sm100::tma_load_4d_elected(dst + uint32_t(c * C::KV_CHUNK + i * p.box_rows * C::RB), m, fb, c * C::CW, c1, c2, b);
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
__device__ void paged_softmax_role(const PagedTileParams &p, PagedUnits<C> units, uint32_t sbase, uint32_t tmem, const Ctl &ctl,
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
        const int tok0 = w.u.b * p.plan.tpb + t * p.tq, token = tok0 + i_tok;
        const int diag = w.u.q.L - w.u.q.n;
        const bool window = p.plan.window > 0;
        const RowKeys keys{w.u.q.L, p.plan.causal ? token + diag : 0x7fffffff,
                           window ? token + diag - p.plan.window + 1 : -0x7fffffff, p.plan.causal ? tok0 + diag : 0x7fffffff,
                           window ? tok0 + p.tq - 1 + diag - p.plan.window + 1 : -0x7fffffff};
        float m_ref = -INFINITY, l = 0.f;
        if (!softmax_tiles<C>(sbase, tmem, ctl, t, quarter, p.scale_log2, keys, js, je, scnt, ocnt, m_ref, l)) goto unwind;
        if (nk > 0) {
            if (!warp_wait_bar(bar(C::B_OFINAL + t), ofin & 1u, ctl, kSiteOFinal)) goto unwind;
            ++ofin;
            sm100::tc_fence_after_sync();
        }
        ocnt += uint32_t(nk);
        {
            const float inv_l = l > 0.f ? 1.f / l : 0.f;
            const float lse = l > 0.f ? (m_ref + log2f(l)) * kLn2 : -INFINITY;
            const bool store = i_tok < p.tq && token < w.u.q.n;
            const long long row = w.u.q.q0 + token;
            const int head = w.u.g * p.pack + i_head;
            const long long o_off = store ? (row * p.Hq + head) * D : -1;
            const long long piece = ((long long)w.slot * C::NQT + t) * kBlockQ + row_in_tile;
            if (w.whole && C::OSTAGE) {
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
            } else {
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
                    if (!w.whole) {
                        float *dst = p.o_part + piece * D + 32 * c;
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (32 * c + 4 * i < D)
                                *reinterpret_cast<float4 *>(dst + 4 * i) =
                                    make_float4(__uint_as_float(o[4 * i]) * inv_l, __uint_as_float(o[4 * i + 1]) * inv_l,
                                                __uint_as_float(o[4 * i + 2]) * inv_l, __uint_as_float(o[4 * i + 3]) * inv_l);
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (32 * c + 8 * i >= D) continue;
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
                if (!w.whole) p.lse_part[piece] = lse;
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
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the merge may be set up meanwhile

    if (threadIdx.x == 0) {
        init_barriers<C>(sbase);
        *abort_flag = 0;
        sm100::fence_mbar_init();
    }
    if (warp == 0) {
        sm100::tmem_alloc(sm100::smem_u32(tmem_holder), C::TMEM_COLS);
        sm100::tmem_relinquish();
    }
    // The plan's sums use the K/V ring's memory before the first copy goes there.
    static_assert(sizeof(PlanScan<C::THREADS>) + sizeof(Cursor) <= size_t(C::KV_TILE), "plan in the ring");
    auto &scan = *reinterpret_cast<PlanScan<C::THREADS> *>(smem + C::SMEM_KV);
    auto &start = *reinterpret_cast<Cursor *>(smem + C::SMEM_KV + sizeof(PlanScan<C::THREADS>));
    const long long total = plan_scan<C::BC>(p.plan, scan, int(threadIdx.x), blockIdx.x == 0);
    if (threadIdx.x == 0) {
        const long long x0 = range_start(total, p.plan.workers, int(blockIdx.x));
        const long long x1 = range_start(total, p.plan.workers, int(blockIdx.x) + 1);
        Cursor c{};
        if (x0 < x1) {
            c.u = plan_find<C::BC>(p.plan, scan, x0);
            c.j = c.u.js + int(x0 - c.u.begin);
            c.left = int(x1 - x0);
        }
        start = c;
    }
    __syncthreads();
    const PagedUnits<C> units{p, start, true};
    sm100::fence_proxy_async_smem();   // those reads and writes come before the copies into the ring
    sm100::tc_fence_before_sync();
    __syncthreads();
    sm100::tc_fence_after_sync();
    const uint32_t tmem = *tmem_holder;

    if (warp < C::SOFTMAX_WARPS) {
        if constexpr (C::REALLOC_REGS) sm100::regs_increase<C::SOFTMAX_REGS>();
        paged_softmax_role<C>(p, units, sbase, tmem, ctl, warp, lane);
    } else {
        if constexpr (C::REALLOC_REGS) sm100::regs_decrease<C::CONTROL_REGS>();
        if (warp == C::TMA_WARP) paged_producer_role<C>(&tm_q, &tm_k, &tm_v, p, units, sbase, ctl);
        else if (warp == C::MMA_WARP) mma_role<C>(units, sbase, tmem, ctl);
    }
    __syncwarp();

    sm100::tc_fence_before_sync();
    __syncthreads();
    sm100::tc_fence_after_sync();
    if (warp == 0) sm100::tmem_dealloc(tmem, C::TMEM_COLS);
}

}  // namespace fa
