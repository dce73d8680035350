// fa_tables.cu -- block tables, slot maps and the free-block stack of a paged key/value cache,
// built on the GPU from request lengths (fa_kv_reserve, fa_kv_release; declared in include/fa.h).
//
// With held_r = ceil(ctx_r / page), want_r = ceil((ctx_r + new_r) / page) and the exclusive prefix
// sums cu (of new) and off (of want - held):
//     table[r][held_r + n] = free[count - 1 - (off_r + n)],
//     token t of request r: position ctx_r + t - cu_r, slot = block(position / page) * page + position % page.
// A new block's id is taken from the free stack directly, so no token waits for a table entry
// that another thread writes.
//
// The work is a few hundred kilobytes at most (12 bytes a token), so the time is latency: one
// launch, one round trip for the lengths, one for the table entries.  One thread-block cluster of
// up to eight CTAs runs it; every CTA sums all lengths itself (no exchange), takes every n-th
// token, and the cluster barrier orders the reads of the lengths and the free count before their
// updated values are written, which is what lets both be updated in place.  A step of many tokens
// goes over the whole GPU instead, and a second small kernel, set up meanwhile, writes those values
// (1500 requests, 100,000 tokens: 15.9 us against 28 us by the cluster).  16 decoding requests
// take 4.3 us, of which a launch alone is 2.2.
#include <algorithm>
#include <cstdint>

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_cache.h"
#include "fa_host.h"

namespace {

using namespace fa_host;
namespace cg = cooperative_groups;

constexpr int kTableThreads = 1024;
constexpr int kMaxCluster = 8;
constexpr int kMostItems = 1 << 30;   // requests, tokens, blocks: strided loops stay within 32 bits
// Tokens up to which one cluster does a step.
constexpr int kClusterTokens = 16384;
constexpr int kBatch = 4;   // tokens or blocks a thread has in flight
// Tokens and blocks of a chunk of kTableThreads requests are summed in the halves of one 64-bit word.  A
// request has at most T new tokens and no more new blocks than tokens, so neither half carries while T
// is below this; from here on the totals are summed apart before the halves are relied on.
constexpr int kPackedTokens = 1 << 22;
static_assert((long long)kTableThreads * (kPackedTokens - 1) < 1LL << 32, "a chunk's tokens fit 32 bits");

__device__ __forceinline__ int blocks_of(int tokens, int page) {   // tokens + page - 1 may pass 2^31
    return int((unsigned(tokens) + unsigned(page) - 1u) / unsigned(page));
}

// Inclusive scan over a warp.
__device__ __forceinline__ unsigned long long warp_scan(unsigned long long x) {
    const int lane = int(threadIdx.x) % 32;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}

// Inclusive scan over the block.  `warp_sums`: 32 words of shared memory; `flag` becomes its OR over the
// block.
__device__ __forceinline__ unsigned long long block_scan(unsigned long long x, unsigned long long *warp_sums,
                                                         unsigned long long *total, int &flag) {
    const int lane = int(threadIdx.x) % 32, warp = int(threadIdx.x) / 32, warps = int(blockDim.x) / 32;
    x = warp_scan(x);
    __syncthreads();   // the previous scan's sums have been read
    if (lane == 31) warp_sums[warp] = x;
    flag = __syncthreads_or(flag);
    const unsigned long long upto = warp_scan(lane < warps ? warp_sums[lane] : 0ull);   // each warp scans them again
    *total = __shfl_sync(0xffffffffu, upto, 31);
    const unsigned long long before = __shfl_sync(0xffffffffu, upto, (warp + 31) % 32);
    return x + (warp > 0 ? before : 0ull);
}

// The last entry of `starts` (ascending, n entries, starts[0] <= x) that is <= x: the request that
// holds token (or new block) x; requests without any have equal starts and are passed over.
__device__ __forceinline__ int holder(const int *starts, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (starts[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

struct ReserveParams {
    const int *ctx, *fresh;      // [R] tokens held, tokens to come
    int *table;                  // [R, max_blocks], row stride `table_stride`
    long long table_stride;
    const int *free_blocks;      // [num_blocks] stack
    const int *free_count;       // [1]
    int *free_count_out;         // [1], may be free_count
    int *cu;                     // [R + 1]
    int *seq_lens;               // [R], may be ctx
    int *positions;              // [T]
    long long *slots;            // [T]
    int *status;
    int R, T, max_blocks, num_blocks, page;
};

// What a launch does: all of it by one cluster, the tokens and the table by any grid, or the values
// that may be updated in place (after that grid) by one CTA.
enum class ReservePart { All, Tokens, Lengths };

template <ReservePart PART>
__global__ void __launch_bounds__(kTableThreads) fa_kv_reserve_kernel(const __grid_constant__ ReserveParams p) {
    __shared__ unsigned long long warp_sums[32];
    __shared__ int s_cu[kTableThreads], s_off[kTableThreads], s_ctx[kTableThreads], s_held[kTableThreads];
    if (PART == ReservePart::Tokens) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int rank = int(blockIdx.x), ranks = int(gridDim.x);   // (the cluster is the grid)
    const int tid = int(threadIdx.x), nt = int(blockDim.x);
    const int count = *p.free_count;

    // Totals, and whether every length fits: a step that does not fit is refused whole.
    long long tokens = 0, blocks = 0;
    unsigned long long my_tokens = 0, my_blocks = 0;   // this thread's requests
    int bad = 0;
    int ctx0 = 0, new0 = 0;   // this thread's request of the first chunk
    unsigned long long upto0 = 0, total0 = 0;
    for (int base = 0; base < p.R; base += nt) {
        const int r = base + tid;
        const int c = r < p.R ? p.ctx[r] : 0, n = r < p.R ? p.fresh[r] : 0;
        unsigned long long mine = 0;
        int off = 0;
        if (c < 0 || n < 0 || (long long)c + n > (long long)p.max_blocks * p.page || n > p.T) {
            off = 1;
            if (rank == 0 && PART != ReservePart::Lengths)
                report_range(p.status, n > p.T && c >= 0 ? kSiteTokens : kSiteLengths, r);
        } else {
            const unsigned need = unsigned(blocks_of(c + n, p.page) - blocks_of(c, p.page));
            mine = (unsigned long long)(unsigned)n | ((unsigned long long)need << 32);
            my_tokens += unsigned(n);
            my_blocks += need;
        }
        unsigned long long total = 0;
        const unsigned long long upto = block_scan(mine, warp_sums, &total, off);
        bad |= off;
        tokens += (long long)(total & 0xffffffffu);
        blocks += (long long)(total >> 32);
        if (base == 0) ctx0 = c, new0 = n, upto0 = upto - mine, total0 = total;
    }
    if (p.T >= kPackedTokens) {   // (a step that passes has at most 2^30 of each, and its packed sums are right)
        unsigned long long all = 0;
        int none = 0;
        block_scan(my_tokens, warp_sums, &all, none);
        tokens = (long long)all;
        block_scan(my_blocks, warp_sums, &all, none);
        blocks = (long long)all;
    }
    if (!bad && tokens > p.T) {
        bad = 1;
        if (rank == 0 && tid == 0 && PART != ReservePart::Lengths) report_range(p.status, kSiteTokens, 0);
    }
    if (!bad && (count < 0 || count > p.num_blocks || blocks > count)) {
        bad = 1;
        if (rank == 0 && tid == 0 && PART != ReservePart::Lengths) report_range(p.status, kSiteBlocks, 0);
    }

    // the lengths have been read; and this kernel ends after the tokens' one
    if (PART == ReservePart::Lengths) asm volatile("griddepcontrol.wait;" ::: "memory");
    int tok_base = 0, blk_base = 0;
    if (!bad) {
        for (int base = 0; base < p.R; base += nt) {
            const int r = base + tid, n_here = min(nt, p.R - base);
            const int c = base == 0 ? ctx0 : (r < p.R ? p.ctx[r] : 0);
            const int n = base == 0 ? new0 : (r < p.R ? p.fresh[r] : 0);
            const int held = blocks_of(c, p.page);
            unsigned long long upto = upto0, total = total0;
            if (base > 0) {
                const unsigned long long mine = (unsigned long long)(unsigned)n | ((unsigned long long)(unsigned)(blocks_of(c + n, p.page) - held) << 32);
                int none = 0;
                upto = block_scan(mine, warp_sums, &total, none) - mine;
            }
            const int tok_end = tok_base + int(total & 0xffffffffu), blk_end = blk_base + int(total >> 32);
            if (PART == ReservePart::Lengths) {
                if (r < p.R) {
                    p.cu[r] = tok_base + int(upto & 0xffffffffu);
                    p.seq_lens[r] = c + n;
                }
                tok_base = tok_end;
                blk_base = blk_end;
                continue;
            }
            s_cu[tid] = tok_base + int(upto & 0xffffffffu);
            s_off[tid] = blk_base + int(upto >> 32);
            s_ctx[tid] = c;
            s_held[tid] = held;
            if (PART == ReservePart::All && rank == 0 && r < p.R) p.cu[r] = s_cu[tid];
            __syncthreads();
            // kBatch tokens a thread at a time: their searches and loads overlap
            const int step = ranks * nt;
            for (int t0 = tok_base + rank * nt + tid; t0 < tok_end; t0 += kBatch * step) {
                int id[kBatch], pos[kBatch], in_page[kBatch], at[kBatch];
                bool old[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int t = min(t0 + k * step, tok_end - 1), i = holder(s_cu, n_here, t);
                    pos[k] = s_ctx[i] + t - s_cu[i];
                    const int lb = pos[k] / p.page;
                    in_page[k] = pos[k] - lb * p.page;
                    at[k] = base + i;
                    old[k] = lb < s_held[i];
                    id[k] = old[k] ? p.table[(long long)(base + i) * p.table_stride + lb]
                                   : p.free_blocks[count - 1 - (s_off[i] + lb - s_held[i])];
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int t = t0 + k * step;
                    if (t >= tok_end) break;
                    long long slot = (long long)id[k] * p.page + in_page[k];
                    if (id[k] < 0 || id[k] >= p.num_blocks) {
                        report_range(p.status, old[k] ? kSiteTableId : kSiteFreeId, at[k]);
                        slot = -1;
                    }
                    p.positions[t] = pos[k];
                    p.slots[t] = slot;
                }
            }
            for (int b = blk_base + rank * nt + tid; b < blk_end; b += ranks * nt) {
                const int i = holder(s_off, n_here, b);
                const int id = p.free_blocks[count - 1 - b];
                if (id < 0 || id >= p.num_blocks) report_range(p.status, kSiteFreeId, base + i);
                p.table[(long long)(base + i) * p.table_stride + s_held[i] + (b - s_off[i])] = id;
            }
            tok_base = tok_end;
            blk_base = blk_end;
            __syncthreads();
        }
    } else if (PART != ReservePart::Tokens && rank == 0) {
        for (int r = tid; r < p.R; r += nt) {
            p.cu[r] = 0;
            if (PART == ReservePart::Lengths) p.seq_lens[r] = p.ctx[r];
        }
    }
    if (PART != ReservePart::Lengths)
        for (int t = tok_base + rank * nt + tid; t < p.T; t += ranks * nt) {
            p.positions[t] = 0;
            p.slots[t] = -1;
        }
    if (PART == ReservePart::Tokens) return;
    if (PART == ReservePart::All) {
        cg::this_cluster().sync();   // every CTA has read the lengths and the count: they may be updated in place
        if (rank == 0)
            for (int r = tid; r < p.R; r += nt) p.seq_lens[r] = bad ? p.ctx[r] : p.ctx[r] + p.fresh[r];
    }
    if (rank == 0 && tid == 0) {
        p.cu[p.R] = tok_base;
        *p.free_count_out = count - blk_base;
    }
}

struct ReleaseParams {
    const int *lens, *done;      // [R]
    const int *table;
    long long table_stride;
    int *free_blocks;            // [num_blocks] stack
    const int *free_count;
    int *free_count_out;         // may be free_count
    int *lens_out;               // [R], may be lens
    int *status;
    int R, max_blocks, num_blocks, page;
};

__global__ void __launch_bounds__(kTableThreads) fa_kv_release_kernel(const __grid_constant__ ReleaseParams p) {
    __shared__ unsigned long long warp_sums[32];
    __shared__ int s_off[kTableThreads];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = int(cluster.block_rank()), ranks = int(cluster.num_blocks());
    const int tid = int(threadIdx.x), nt = int(blockDim.x);
    const int count = *p.free_count;

    long long blocks = 0;
    int bad = 0;
    unsigned long long upto0 = 0, total0 = 0;
    for (int base = 0; base < p.R; base += nt) {
        const int r = base + tid;
        int held = 0, off = 0;
        if (r < p.R && p.done[r] != 0) {
            const int n = p.lens[r];
            if (n < 0 || n > (long long)p.max_blocks * p.page) {
                off = 1;
                if (rank == 0) report_range(p.status, kSiteLengths, r);
            } else {
                held = blocks_of(n, p.page);
            }
        }
        unsigned long long total = 0;
        const unsigned long long upto = block_scan((unsigned long long)(unsigned)held, warp_sums, &total, off);
        bad |= off;
        blocks += (long long)total;
        if (base == 0) upto0 = upto - (unsigned)held, total0 = total;
    }
    if (!bad && (count < 0 || count + blocks > p.num_blocks)) {   // more blocks than the stack can hold
        bad = 1;
        if (rank == 0 && tid == 0) report_range(p.status, kSiteBlocks, 0);
    }
    int blk_base = 0;
    if (!bad) {
        for (int base = 0; base < p.R; base += nt) {
            const int r = base + tid, n_here = min(nt, p.R - base);
            unsigned long long upto = upto0, total = total0;
            if (base > 0) {
                const int held = (r < p.R && p.done[r] != 0) ? blocks_of(p.lens[r], p.page) : 0;
                int none = 0;
                upto = block_scan((unsigned long long)(unsigned)held, warp_sums, &total, none) - (unsigned)held;
            }
            s_off[tid] = blk_base + int(upto);
            __syncthreads();
            const int blk_end = blk_base + int(total);
            const int step = ranks * nt;
            for (int b0 = blk_base + rank * nt + tid; b0 < blk_end; b0 += kBatch * step) {
                int id[kBatch], at[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int b = min(b0 + k * step, blk_end - 1), i = holder(s_off, n_here, b);
                    at[k] = base + i;
                    id[k] = p.table[(long long)(base + i) * p.table_stride + (b - s_off[i])];
                }
#pragma unroll
                for (int k = 0; k < kBatch; ++k) {
                    const int b = b0 + k * step;
                    if (b >= blk_end) break;
                    if (id[k] < 0 || id[k] >= p.num_blocks) report_range(p.status, kSiteTableId, at[k]);
                    p.free_blocks[count + b] = id[k];
                }
            }
            blk_base = blk_end;
            __syncthreads();
        }
    }
    cluster.sync();
    if (rank == 0) {
        for (int r = tid; r < p.R; r += nt) p.lens_out[r] = (!bad && p.done[r] != 0) ? 0 : p.lens[r];
        if (tid == 0) *p.free_count_out = count + blk_base;
    }
}

// One cluster: CTAs of 256 threads while a chunk of 256 requests and a few tokens a thread do,
// else of 1024; as many CTAs (up to eight) as leave each thread about four items.
template <class P>
int launch_cluster(void (*kern)(P), const P &p, long long items, int R, cudaStream_t st) {
    const int threads = (R <= 256 && items <= 1024) ? 256 : kTableThreads;
    const long long want = (items + 4LL * threads - 1) / (4LL * threads);
    int ctas = 1;
    while (ctas < kMaxCluster && ctas < want) ctas *= 2;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(ctas));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(ctas);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    return FA_OK;
}

size_t table_bytes(int R, long long stride, int max_blocks) {
    return R == 0 ? 0 : (size_t(R - 1) * size_t(stride) + size_t(max_blocks)) * 4;
}

}  // namespace

extern "C" {

int fa_kv_reserve(const int *ctx_lens, const int *new_lens, int R, int *block_table, long long table_stride,
                  int max_blocks, const int *free_blocks, const int *free_count, int num_blocks, int page_size,
                  int T, int *cu_seqlens, int *seq_lens, int *positions, long long *slots, int *free_count_out,
                  void *stream) {
    if (R < 0 || T < 0 || max_blocks < 0 || num_blocks < 0 || page_size < 1) return FA_ERR_INVALID_ARG;
    if (table_stride < max_blocks) return FA_ERR_INVALID_ARG;
    if (std::max({R, T, num_blocks}) > kMostItems) return FA_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_size > 0x7fffffffLL) return FA_ERR_INVALID_ARG;   // lengths are 32-bit
    const size_t lens_b = size_t(R) * 4, tab_b = max_blocks > 0 ? table_bytes(R, table_stride, max_blocks) : 0;
    const size_t free_b = size_t(num_blocks) * 4, cu_b = (size_t(R) + 1) * 4, pos_b = size_t(T) * 4, slot_b = size_t(T) * 8;
    if (cu_seqlens == nullptr || free_count == nullptr || free_count_out == nullptr) return FA_ERR_INVALID_ARG;
    if (R > 0 && (ctx_lens == nullptr || new_lens == nullptr || seq_lens == nullptr)) return FA_ERR_INVALID_ARG;
    if ((tab_b > 0 && block_table == nullptr) || (free_b > 0 && free_blocks == nullptr)) return FA_ERR_INVALID_ARG;
    if (T > 0 && (positions == nullptr || slots == nullptr)) return FA_ERR_INVALID_ARG;
    const Span in[] = {{ctx_lens, lens_b, 4}, {new_lens, lens_b, 4}, {free_blocks, free_b, 4}, {free_count, 4, 4}};
    const Span out[] = {{block_table, tab_b, 4}, {cu_seqlens, cu_b, 4}, {seq_lens, lens_b, 4}, {positions, pos_b, 4},
                        {slots, slot_b, 8}, {free_count_out, 4, 4}};
    int rc = check_layout(in, 4, out, 6, [&](int i, int o) {   // updated in place: exactly the same array
        return (i == 0 && o == 2 && ctx_lens == seq_lens) || (i == 3 && o == 5 && free_count == free_count_out);
    });
    if (rc != FA_OK) return rc;
    DeviceState *dev = nullptr;
    int dev_id = -1;
    if ((rc = current_device(&dev, &dev_id)) != FA_OK) return rc;
    SpanRanges seen;
    if ((rc = check_spans(&seen, in, 4, dev_id)) != FA_OK || (rc = check_spans(&seen, out, 6, dev_id)) != FA_OK) return rc;
    ReserveParams p{};
    p.ctx = ctx_lens;
    p.fresh = new_lens;
    p.table = block_table;
    p.table_stride = table_stride;
    p.free_blocks = free_blocks;
    p.free_count = free_count;
    p.free_count_out = free_count_out;
    p.cu = cu_seqlens;
    p.seq_lens = seq_lens;
    p.positions = positions;
    p.slots = slots;
    p.status = dev->status_ptr;
    p.R = R;
    p.T = T;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.page = page_size;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T <= kClusterTokens) return launch_cluster(fa_kv_reserve_kernel<ReservePart::All>, p, std::max(R, T), R, st);
    const unsigned ctas = unsigned(std::min((T + 4 * kTableThreads - 1) / (4 * kTableThreads) * 4, dev->num_sms));
    fa_kv_reserve_kernel<ReservePart::Tokens><<<ctas, kTableThreads, 0, st>>>(p);
    if (cudaGetLastError() != cudaSuccess) return FA_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kTableThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;   // set up while the tokens are written
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, fa_kv_reserve_kernel<ReservePart::Lengths>, p) != cudaSuccess) {
        cudaGetLastError();
        return FA_ERR_CUDA;
    }
    return FA_OK;
}

int fa_kv_release(const int *lens, const int *done, int R, const int *block_table, long long table_stride,
                  int max_blocks, int *free_blocks, const int *free_count, int num_blocks, int page_size,
                  int *lens_out, int *free_count_out, void *stream) {
    if (R < 0 || max_blocks < 0 || num_blocks < 0 || page_size < 1) return FA_ERR_INVALID_ARG;
    if (table_stride != 0 && table_stride < max_blocks) return FA_ERR_INVALID_ARG;   // 0: one row for all
    if (std::max({R, num_blocks}) > kMostItems) return FA_ERR_INVALID_ARG;
    if ((long long)max_blocks * page_size > 0x7fffffffLL) return FA_ERR_INVALID_ARG;
    const size_t lens_b = size_t(R) * 4, tab_b = max_blocks > 0 ? table_bytes(R, table_stride, max_blocks) : 0;
    const size_t free_b = size_t(num_blocks) * 4;
    if (free_count == nullptr || free_count_out == nullptr) return FA_ERR_INVALID_ARG;
    if (R > 0 && (lens == nullptr || done == nullptr || lens_out == nullptr)) return FA_ERR_INVALID_ARG;
    if ((tab_b > 0 && block_table == nullptr) || (free_b > 0 && free_blocks == nullptr)) return FA_ERR_INVALID_ARG;
    const Span in[] = {{lens, lens_b, 4}, {done, lens_b, 4}, {block_table, tab_b, 4}, {free_count, 4, 4}};
    const Span out[] = {{free_blocks, free_b, 4}, {lens_out, lens_b, 4}, {free_count_out, 4, 4}};
    int rc = check_layout(in, 4, out, 3, [&](int i, int o) {
        return (i == 0 && o == 1 && lens == lens_out) || (i == 3 && o == 2 && free_count == free_count_out);
    });
    if (rc != FA_OK) return rc;
    DeviceState *dev = nullptr;
    int dev_id = -1;
    if ((rc = current_device(&dev, &dev_id)) != FA_OK) return rc;
    SpanRanges seen;
    if ((rc = check_spans(&seen, in, 4, dev_id)) != FA_OK || (rc = check_spans(&seen, out, 3, dev_id)) != FA_OK) return rc;
    ReleaseParams p{};
    p.lens = lens;
    p.done = done;
    p.table = block_table;
    p.table_stride = table_stride;
    p.free_blocks = free_blocks;
    p.free_count = free_count;
    p.free_count_out = free_count_out;
    p.lens_out = lens_out;
    p.status = dev->status_ptr;
    p.R = R;
    p.max_blocks = max_blocks;
    p.num_blocks = num_blocks;
    p.page = page_size;
    // the blocks that come back are not known here: at most the pool, and what the table can hold
    const long long items = std::min<long long>(num_blocks, (long long)R * max_blocks);
    return launch_cluster(fa_kv_release_kernel, p, std::max<long long>(R, items), R, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
