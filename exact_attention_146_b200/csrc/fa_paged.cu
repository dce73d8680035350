// fa_paged.cu -- attention of new tokens over a paged cache (fa_paged_fwd, declared in include/fa.h):
// argument checks, workspace layout, choice and launches of the kernels in fa_paged_rows.cuh (few rows)
// and fa_paged_tiles.cuh (many).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_cache.h"
#include "fa_host.h"
#include "fa_paged_rows.cuh"
#include "fa_paged_tiles.cuh"

namespace {

using namespace fa;
using namespace fa_host;

constexpr int kMaxRowWorkers = kMaxPagedCtas * 10;

// The few-rows kernel's shape for each head dim: stages of 4 to 16 KB, and as many warps as leave each at
// least three of them.  Decoding 48 requests of 4k to 16k keys (Hkv 8, slots of a page apart by all heads):
//   d = 128: 32 keys, 4 warps 248 us (6.55 TB/s); 16 keys, 8 warps 252 us
//   d = 64: 32 keys, 8 warps 152 us; 16 keys, 8 warps 180 us        d = 32: 32 keys, 10 warps 87 us; 8 warps 123 us
//   d = 192: 16 keys, 5 warps 372 us; 4 warps 409 us                d = 256: 16 keys, 4 warps 482 us; 3 warps 577 us
// Calls too small to fill the GPU take a worker's chain of steps, which 32 keys shorten: one request of
// 40,000 keys 40 us against 44 us.
template <int D> struct RowShape { static constexpr int KEYS = 32, WARPS = 4; };
template <> struct RowShape<32> { static constexpr int KEYS = 32, WARPS = 10; };
template <> struct RowShape<64> { static constexpr int KEYS = 32, WARPS = 8; };
template <> struct RowShape<192> { static constexpr int KEYS = 16, WARPS = 5; };
template <> struct RowShape<256> { static constexpr int KEYS = 16, WARPS = 4; };
template <int D, bool F16, int ROWS, bool TMA> using RowsOf = RowCfg<D, F16, RowShape<D>::KEYS, RowShape<D>::WARPS, ROWS, TMA>;

size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

// Workspace: the pieces' O (fp32), then their LSE; two pieces a worker at most (its range's first
// and last unit).
size_t part_o_bytes(int workers, int rows, int d) { return align256(size_t(workers) * 2 * rows * d * 4); }
size_t part_bytes(int workers, int rows, int d) { return part_o_bytes(workers, rows, d) + align256(size_t(workers) * 2 * rows * 4); }
size_t job_bytes(int workers) { return align256(size_t(workers) * sizeof(MergeJob)); }

int largest_divisor(int n, int most) {
    for (int x = std::min(n, most); x > 1; --x)
        if (n % x == 0) return x;
    return 1;
}

// Launches `kern` so that its blocks may be set up while the kernel before it in the stream still
// runs (it waits for that kernel's end itself, by griddepcontrol.wait).
template <class... P, class... A>
int launch_after(void (*kern)(P...), unsigned grid, int threads, size_t smem, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(unsigned(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    return FA_OK;
}

// What is kept per kernel and device: its shared-memory limit has been raised, and its registers are
// those that it was written for (0 not looked at, 1 usable, -1 not).
template <class Kernel>
int make_ready(Kernel kern, int smem, int regs, int &state) {
    std::lock_guard<std::mutex> lock(g_mutex);
    if (state == 0) {
        cudaFuncAttributes a{};
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess ||
            cudaFuncGetAttributes(&a, kern) != cudaSuccess) {
            cudaGetLastError();
            return FA_ERR_CUDA;
        }
        state = (regs == 0 || a.numRegs == regs) ? 1 : -1;
    }
    return state == 1 ? FA_OK : FA_ERR_CUDA;
}

// The largest power of two, up to a key tile, that divides a page.
int box_rows(int page, int most) {
    int g = 1;
    while (g < most && page % (2 * g) == 0) g *= 2;
    return g;
}

// A [T, H, d] array of rows `stride` apart: box (cw columns, heads, rows).
struct View {
    const void *base;
    long long dims[3], strides[3];   // elements; the axes after d
    int box[3];
};

// The caches as the tensor maps see them: the axes after d, the nearer of head and slot first.
View cache_view(const PagedParams &p, int Hkv) {
    View kv{p.k, {Hkv, p.page, p.num_blocks}, {p.head_stride, p.slot_stride, p.block_stride}, {1, 1, 1}};
    if (p.slot_first) {
        std::swap(kv.dims[0], kv.dims[1]);
        std::swap(kv.strides[0], kv.strides[1]);
    }
    return kv;
}

// Tensor maps of K and V with boxes of cw columns and `run` slots.
int encode_cache(CUtensorMap *mk, CUtensorMap *mv, const PagedParams &p, View kv, int d, int cw, int run, bool f16) {
    kv.box[p.slot_first ? 0 : 1] = run;
    // L2 fetches no more at once than lies in the row, where the bytes behind it are another head's: those are
    // read at other times by other workers (d = 80, 48 requests: 160-byte rows fetched as whole lines took 1.6 times the bytes).
    const int row = 2 * d, line = p.slot_stride == d || row % 256 == 0 ? 256 : row % 128 == 0 ? 128 : 64;
    const int rc = encode_view(mk, p.k, d, kv.dims, kv.strides, cw, kv.box, f16 ? 1 : 0, line);
    return rc != FA_OK ? rc : encode_view(mv, p.v, d, kv.dims, kv.strides, cw, kv.box, f16 ? 1 : 0, line);
}

// What a unit of the few-rows kernel costs besides its steps (its Q, the first look-up, what it writes):
// 64 requests of up to 500 keys took 41 us without it and with the lengths read from memory, 21 us with both.
constexpr int kRowOverhead = 2;

// The kernel of few rows; fills what it adds to `p`.
template <class C>
int launch_rows_as(PagedParams &p, const View &kv, bool after_tiles, char *workspace, int ctas, int dev, cudaStream_t st) {
    static int state[kMaxDevices] = {};
    int rc = make_ready(fa_paged_rows_kernel<C>, C::SMEM, 0, state[dev]);
    if (rc != FA_OK) return rc;
    CUtensorMap mk{}, mv{};
    if (C::TMA) {
        p.run = box_rows(p.page, C::KEYS);
        if ((rc = encode_cache(&mk, &mv, p, kv, C::D, C::CW, p.run, C::F16)) != FA_OK) return rc;
    }
    p.pack = largest_divisor(p.n_rep, C::ROWS);
    p.plan.groups = p.Hq / p.pack;
    p.plan.tpb = C::ROWS / p.pack;
    p.plan.workers = ctas * C::WARPS;
    p.plan.overhead = kRowOverhead;
    p.o_part = reinterpret_cast<float *>(workspace);
    p.lse_part = reinterpret_cast<float *>(workspace + part_o_bytes(p.plan.workers, C::ROWS, C::D));
    p.jobs = reinterpret_cast<MergeJob *>(workspace + part_bytes(p.plan.workers, C::ROWS, C::D));
    // after the tile kernel, which began when the inputs were complete: beside its last CTAs
    if (after_tiles) return launch_after(fa_paged_rows_kernel<C>, unsigned(ctas), C::THREADS, C::SMEM, st, mk, mv, p);
    fa_paged_rows_kernel<C><<<unsigned(ctas), C::THREADS, C::SMEM, st>>>(mk, mv, p);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Pages of whole swizzle atoms come by TMA, any other row by row.
template <int D, bool F16, int ROWS>
int launch_rows(PagedParams &p, const View &kv, bool after_tiles, char *workspace, int ctas, int dev, cudaStream_t st) {
    return p.page % 8 == 0 && p.num_blocks > 0 ? launch_rows_as<RowsOf<D, F16, ROWS, true>>(p, kv, after_tiles, workspace, ctas, dev, st)
                                               : launch_rows_as<RowsOf<D, F16, ROWS, false>>(p, kv, after_tiles, workspace, ctas, dev, st);
}

template <int D, bool F16, int ROWS>
int launch_rows_only(PagedParams p, const View &kv, char *workspace, int ctas, int dev, cudaStream_t st) {
    const int rc = launch_rows<D, F16, ROWS>(p, kv, false, workspace, ctas, dev, st);
    if (rc != FA_OK) return rc;
    return launch_after(fa_paged_merge_rows_kernel<D, F16, ROWS>, unsigned(p.plan.workers - 1), 256, 0, st, p);
}

// The dense forward's tilings (fa_fwd.cu says why each).
template <bool H> using Tile32 = TileCfg<32, 128, 2, 8, 2, 1, true, 2, H>;
template <bool H> using Tile64 = TileCfg<64, 128, 2, 8, 2, 1, true, 2, H>;
template <bool H> using Tile80 = TileCfg<80, 128, 2, 4, 1, 1, true, 0, H, false, false, true>;
template <bool H> using Tile96 = TileCfg<96, 128, 2, 4, 1, 1, true, 0, H, false, false, true>;
template <bool H> using Tile128 = TileCfg<128, 128, 2, 4, 1, 1, true, 0, H, false, false, true>;
template <bool H> using Tile192 = TileCfg<192, 64, 2, 4, 1, 1, true, 0, H, false, false, true>;
template <bool H> using Tile256 = TileCfg<256, 64, 1, 4, 1, 2, false, 0, H>;

// What a unit of the tile kernel costs besides its key tiles (Q, the first tile's way through the
// pipeline with nothing beside it, the epilogue), in key tiles of 1.9 to 2.2 us.  8 requests of up to 512
// new tokens (d = 128): 203 us with 2, 206 with 3, 210 with 6, 235 without; 37 ragged prompts of 4 KV heads
// (d = 64): 93, 97, 96 us with 2, 3, 4.
constexpr int kTileOverhead = 2;

// Chunks on the tensor cores; requests of at most `few` new tokens (few > 0) by the kernel of few rows
// behind it, whose CTAs start as the tile kernel's end: those end up to a quarter of the time apart, and the
// other's work fills that.
template <class C, int FEW>
int launch_tiles(const PagedParams &base, const View &q, const View &kv, int few, char *workspace, int ctas, int dev,
                 cudaStream_t st) {
    static int state[kMaxDevices] = {};
    // the register split inside the kernel counts on exactly this launch budget
    int rc = make_ready(fa_paged_tiles_kernel<C>, PlanSmem<C>::BYTES, C::REALLOC_REGS ? C::LAUNCH_REGS : 0, state[dev]);
    if (rc != FA_OK) return rc;
    PagedTileParams p{};
    static_cast<PagedParams &>(p) = base;
    p.tq = kBlockQ / p.pack;
    p.plan.groups = p.Hq / p.pack;
    p.plan.tpb = C::NQT * p.tq;
    p.plan.workers = ctas;
    p.plan.overhead = kTileOverhead;
    p.plan.n_lo = few + 1;
    p.run = box_rows(p.page, C::BC);
    constexpr int rows = C::NQT * kBlockQ;
    char *const ws = workspace + part_bytes(kMaxRowWorkers, kRowRows, C::D) + job_bytes(kMaxRowWorkers);
    p.o_part = reinterpret_cast<float *>(ws);
    p.lse_part = reinterpret_cast<float *>(ws + part_o_bytes(ctas, rows, C::D));
    p.jobs = reinterpret_cast<MergeJob *>(ws + part_bytes(ctas, rows, C::D));
    p.cuts = reinterpret_cast<long long *>(ws + part_bytes(ctas, rows, C::D) + job_bytes(ctas));
    CUtensorMap mq, mk, mv;
    const int elem = C::F16 ? 1 : 0;
    if ((rc = encode_view(&mq, q.base, C::D, q.dims, q.strides, C::CW, q.box, elem)) != FA_OK) return rc;
    if ((rc = encode_cache(&mk, &mv, p, kv, C::D, C::CW, p.run, C::F16)) != FA_OK) return rc;
    PagedParams pf = base;
    pf.plan.n_hi = few;
    pf.say = 0;
    fa_paged_tiles_kernel<C><<<unsigned(ctas), C::THREADS, PlanSmem<C>::BYTES, st>>>(mq, mk, mv, p);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    if (few > 0 && (rc = launch_rows<C::D, C::F16, FEW>(pf, kv, true, workspace, ctas, dev, st)) != FA_OK) return rc;
    const int blocks = (ctas - 1) * (rows / 32) + (few > 0 ? pf.plan.workers - 1 : 0);
    if (blocks == 0) return FA_OK;
    return launch_after(fa_paged_merge_kernel<C, FEW>, unsigned(blocks), 256, 0, st, p, pf);
}

template <bool F16, int FEW>
int dispatch_tiles(PagedParams p, const View &kv, int d, int few, char *workspace, int ctas, int dev, cudaStream_t st) {
    p.pack = largest_divisor(p.n_rep, kBlockQ);
    const View q{p.q, {p.Hq, p.plan.T, 1}, {d, p.q_stride, p.q_stride * p.plan.T}, {p.pack, kBlockQ / p.pack, 1}};
    switch (d) {
        case 32: return launch_tiles<Tile32<F16>, FEW>(p, q, kv, few, workspace, ctas, dev, st);
        case 64: return launch_tiles<Tile64<F16>, FEW>(p, q, kv, few, workspace, ctas, dev, st);
        case 80: return launch_tiles<Tile80<F16>, FEW>(p, q, kv, few, workspace, ctas, dev, st);
        case 96: return launch_tiles<Tile96<F16>, FEW>(p, q, kv, few, workspace, ctas, dev, st);
        case 128: return launch_tiles<Tile128<F16>, FEW>(p, q, kv, few, workspace, ctas, dev, st);
        case 192: return launch_tiles<Tile192<F16>, FEW>(p, q, kv, few, workspace, ctas, dev, st);
        default: return launch_tiles<Tile256<F16>, FEW>(p, q, kv, few, workspace, ctas, dev, st);
    }
}

template <bool F16, int ROWS>
int dispatch_rows(const PagedParams &p, const View &kv, int d, char *workspace, int ctas, int dev, cudaStream_t st) {
    switch (d) {
        case 32: return launch_rows_only<32, F16, ROWS>(p, kv, workspace, ctas, dev, st);
        case 64: return launch_rows_only<64, F16, ROWS>(p, kv, workspace, ctas, dev, st);
        case 80: return launch_rows_only<80, F16, ROWS>(p, kv, workspace, ctas, dev, st);
        case 96: return launch_rows_only<96, F16, ROWS>(p, kv, workspace, ctas, dev, st);
        case 128: return launch_rows_only<128, F16, ROWS>(p, kv, workspace, ctas, dev, st);
        case 192: return launch_rows_only<192, F16, ROWS>(p, kv, workspace, ctas, dev, st);
        default: return launch_rows_only<256, F16, ROWS>(p, kv, workspace, ctas, dev, st);
    }
}

int paged_fwd(const void *q, long long q_stride, const fa_paged_cache *given, const int *block_table,
              long long table_stride, int max_blocks, const int *cu_seqlens, const int *seq_lens, int R, int T, int Hq,
              int max_new, float scale, int causal, int window, void *out, float *lse, void *workspace,
              size_t workspace_bytes, bool f16, void *stream) {
    // ---- host-only validation
    if (given == nullptr || R < 0 || T < 0 || Hq <= 0 || Hq > 65535 || max_new < 0 || max_blocks < 0) return FA_ERR_INVALID_ARG;
    const fa_paged_cache tidy = tidy_cache(*given), *cache = &tidy;
    int rc = valid_cache(cache);
    if (rc != FA_OK) return rc;
    const int d = cache->d, Hkv = cache->Hkv;
    if (Hq % Hkv != 0 || (causal != 0 && causal != 1) || window < 0 || (window > 0 && !causal)) return FA_ERR_INVALID_ARG;
    if (!std::isfinite(scale) || !(scale > 0.f)) return FA_ERR_INVALID_ARG;
    if ((table_stride != 0 && table_stride < max_blocks) || (long long)max_blocks * cache->page_size > 0x7fffffffLL - 4096)
        return FA_ERR_INVALID_ARG;   // (keys of the last tile stay within 32 bits)
    if (q_stride < (long long)Hq * d || q_stride % 8 != 0) return FA_ERR_INVALID_ARG;
    if (R == 0 || T == 0) return FA_OK;
    const size_t q_b = (size_t(T - 1) * size_t(q_stride) + size_t(Hq) * d) * 2, out_b = size_t(T) * Hq * d * 2;
    const size_t lse_b = lse != nullptr ? size_t(T) * Hq * 4 : 0, kv_b = cache_bytes(cache);
    const size_t tab_b = max_blocks > 0 ? (size_t(R - 1) * size_t(table_stride) + size_t(max_blocks)) * 4 : 0;
    const size_t ws_b = fa_paged_workspace_bytes(Hq, Hkv, d);
    if (q == nullptr || out == nullptr || cu_seqlens == nullptr || seq_lens == nullptr) return FA_ERR_INVALID_ARG;
    if ((tab_b > 0 && block_table == nullptr) || (kv_b > 0 && (cache->k == nullptr || cache->v == nullptr))) return FA_ERR_INVALID_ARG;
    if (workspace == nullptr || workspace_bytes < ws_b) return FA_ERR_INVALID_ARG;
    const Span in[] = {{q, q_b, 16}, {cache->k, kv_b, 16}, {cache->v, kv_b, 16}, {block_table, tab_b, 4},
                       {cu_seqlens, (size_t(R) + 1) * 4, 4}, {seq_lens, size_t(R) * 4, 4}};
    const Span outs[] = {{out, out_b, 16}, {lse, lse_b, 4}, {workspace, ws_b, 256}};
    if ((rc = check_layout(in, 6, outs, 3, [](int, int) { return false; })) != FA_OK) return rc;

    // ---- device checks
    DeviceState *dev = nullptr;
    int dev_id = -1;
    if ((rc = current_device(&dev, &dev_id)) != FA_OK) return rc;
    SpanRanges seen;
    if ((rc = check_spans(&seen, in, 6, dev_id)) != FA_OK || (rc = check_spans(&seen, outs, 3, dev_id)) != FA_OK) return rc;

    PagedParams p{};
    p.plan.cu = cu_seqlens;
    p.plan.lens = seq_lens;
    p.plan.status = dev->status_ptr;
    p.plan.max_len = (long long)max_blocks * cache->page_size;
    p.plan.R = R;
    p.plan.T = T;
    p.plan.max_new = max_new;
    p.plan.causal = causal;
    p.plan.window = window;
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(cache->k);
    p.v = static_cast<const uint16_t *>(cache->v);
    p.out = static_cast<uint16_t *>(out);
    p.lse = lse;
    p.table = block_table;
    p.table_stride = table_stride;
    p.q_stride = q_stride;
    p.block_stride = cache->block_stride;
    p.slot_stride = cache->slot_stride;
    p.head_stride = cache->head_stride;
    p.Hq = Hq;
    p.n_rep = Hq / Hkv;
    p.page = cache->page_size;
    p.num_blocks = cache->num_blocks;
    p.scale_log2 = scale * 1.4426950408889634f;
    const int ctas = std::min(dev->num_sms, kMaxPagedCtas);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    p.plan.n_lo = 1;
    p.plan.n_hi = max_new;
    p.say = 1;
    p.slot_first = p.slot_stride < p.head_stride ? 1 : 0;
    const View kv = cache_view(p, Hkv);
    char *const ws = static_cast<char *>(workspace);
    // Calls of up to 16 rows a KV head, and in a mixed call the requests of so few, take the kernel of few rows.  48
    // requests of 4k to 16k keys (d 128), whose K and V cost 281 us at the copy rate: 4 rows 281 us, 16 rows 316 us;
    // by the tile kernel 449 us for 20 rows and 457 us for 124.  (Two units of 16 rows would read K and V twice, 563 us.)
    // Row tiles of 128 need pages of whole swizzle atoms (8 slots), so prompts over any other page take the kernel of
    // few rows too, which reads K and V once per 16 rows: 4096 new tokens over 28672 keys (Hq 32, Hkv 8, d 128) take 40 ms
    // with pages of 1, 4 or 100, against 1.71 ms with 128, 1.96 with 16, 2.85 with 8.
    const bool eight = p.n_rep <= 8;   // a unit of 8 rows holds a decoding step; else one of 16
    const int few = kRowRows / p.n_rep;   // new tokens whose rows fit a unit
    if (max_new > few && p.page % 8 == 0 && p.num_blocks > 0) {
        const int split = R == 1 ? 0 : eight ? 8 / p.n_rep : few;
        if (eight)
            return f16 ? dispatch_tiles<true, 8>(p, kv, d, split, ws, ctas, dev_id, st)
                       : dispatch_tiles<false, 8>(p, kv, d, split, ws, ctas, dev_id, st);
        return f16 ? dispatch_tiles<true, kRowRows>(p, kv, d, split, ws, ctas, dev_id, st)
                   : dispatch_tiles<false, kRowRows>(p, kv, d, split, ws, ctas, dev_id, st);
    }
    // Rows are the narrow side of the kernel's products: 8 where they fit (a decoding step of up to 8 heads a KV
    // head), which halves the products.
    if ((long long)max_new * p.n_rep <= 8)
        return f16 ? dispatch_rows<true, 8>(p, kv, d, ws, ctas, dev_id, st) : dispatch_rows<false, 8>(p, kv, d, ws, ctas, dev_id, st);
    return f16 ? dispatch_rows<true, kRowRows>(p, kv, d, ws, ctas, dev_id, st) : dispatch_rows<false, kRowRows>(p, kv, d, ws, ctas, dev_id, st);
}

}  // namespace

extern "C" {

size_t fa_paged_workspace_bytes(int Hq, int Hkv, int d) {
    if (Hq <= 0 || Hkv <= 0 || Hq % Hkv != 0 || fa_tile_config(d, nullptr, nullptr, nullptr, nullptr) != FA_OK) return 0;
    return part_bytes(kMaxRowWorkers, kRowRows, d) + job_bytes(kMaxRowWorkers) +
           part_bytes(kMaxPagedCtas, d == 256 ? kBlockQ : 2 * kBlockQ, d) + job_bytes(kMaxPagedCtas) +
           align256(size_t(kMaxPagedCtas) * (kMaxPagedCtas + 1) * sizeof(long long));
}

int fa_paged_fwd(const void *q, long long q_stride, const fa_paged_cache *cache, const int *block_table,
                 long long table_stride, int max_blocks, const int *cu_seqlens, const int *seq_lens, int R, int T, int Hq,
                 int max_new, float scale, int causal, int window, void *out, float *lse, void *workspace,
                 size_t workspace_bytes, void *stream) {
    return paged_fwd(q, q_stride, cache, block_table, table_stride, max_blocks, cu_seqlens, seq_lens, R, T, Hq, max_new,
                     scale, causal, window, out, lse, workspace, workspace_bytes, false, stream);
}

int fa_paged_fwd_f16(const void *q, long long q_stride, const fa_paged_cache *cache, const int *block_table,
                     long long table_stride, int max_blocks, const int *cu_seqlens, const int *seq_lens, int R, int T,
                     int Hq, int max_new, float scale, int causal, int window, void *out, float *lse, void *workspace,
                     size_t workspace_bytes, void *stream) {
    return paged_fwd(q, q_stride, cache, block_table, table_stride, max_blocks, cu_seqlens, seq_lens, R, T, Hq, max_new,
                     scale, causal, window, out, lse, workspace, workspace_bytes, true, stream);
}

}  // extern "C"
