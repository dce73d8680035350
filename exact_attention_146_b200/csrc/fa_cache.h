// fa_cache.h -- host-side argument checks of the paged-cache entry points: the cache's layout,
// and rows of a strided [T, heads, d] array.  Internal to the library.
#pragma once

#include <algorithm>
#include <cstddef>
#include <cstdint>

#include "fa.h"
#include "fa_host.h"

namespace fa_host {

// Sites of FA_ERR_PAGED_RANGE in the device status word (bits 8..15).
enum PagedSite : int {
    kSiteLengths = 41, kSiteTokens = 42, kSiteBlocks = 43, kSiteFreeId = 44, kSiteTableId = 45, kSiteSlot = 46
};

#ifdef __CUDACC__
__device__ __forceinline__ void report_range(int *status, int site, long long who) {
    const int w = who < 0 ? 0 : (who > 0x7FFF ? 0x7FFF : int(who));
    atomicCAS(status, 0, int(FA_ERR_PAGED_RANGE) | (site << 8) | (w << 16));
}
#endif

// T rows of `width` elements, `stride` elements apart.
struct Rows {
    const void *p;
    long long stride;
    int width;
};

inline bool same_rows(const Rows &a, const Rows &b) { return a.p == b.p && a.stride == b.stride; }

// Whether any row of a shares memory with a row of b (T rows each, es bytes an element).  Rows
// of equal stride may lie between each other's (slices of one fused projection): then the offset
// of b's rows against a's, modulo the stride, decides.  With other strides the whole extents do.
inline bool rows_overlap(const Rows &a, const Rows &b, int T, int es) {
    if (T <= 0 || a.width == 0 || b.width == 0 || a.p == nullptr || b.p == nullptr) return false;
    const size_t na = (size_t(T - 1) * size_t(a.stride) + size_t(a.width)) * size_t(es);
    const size_t nb = (size_t(T - 1) * size_t(b.stride) + size_t(b.width)) * size_t(es);
    if (!overlaps(a.p, na, b.p, nb)) return false;
    if (a.stride != b.stride) return true;
    const uintptr_t pa = reinterpret_cast<uintptr_t>(a.p), pb = reinterpret_cast<uintptr_t>(b.p);
    const uintptr_t step = uintptr_t(a.stride) * uintptr_t(es);
    const uintptr_t off = pb >= pa ? (pb - pa) % step : (step - (pa - pb) % step) % step;   // b's row after a's
    return off < uintptr_t(a.width) * es || off + uintptr_t(b.width) * es > step;
}

// The strides of axes of one entry mean nothing: they become d, which every rule allows.
inline fa_paged_cache tidy_cache(const fa_paged_cache &given) {
    fa_paged_cache c = given;
    if (c.num_blocks <= 1) c.block_stride = c.d;
    if (c.page_size <= 1) c.slot_stride = c.d;
    if (c.Hkv <= 1) c.head_stride = c.d;
    return c;
}

// Bytes from the cache's base to the end of its last element (k and v alike).
inline size_t cache_bytes(const fa_paged_cache *c) {
    if (c->num_blocks == 0) return 0;
    return (size_t(c->num_blocks - 1) * size_t(c->block_stride) + size_t(c->page_size - 1) * size_t(c->slot_stride) +
            size_t(c->Hkv - 1) * size_t(c->head_stride) + size_t(c->d)) * 2;
}

inline int valid_cache(const fa_paged_cache *c) {
    if (c->num_blocks < 0 || c->page_size < 1 || c->Hkv < 1 || c->Hkv > 65535) return FA_ERR_INVALID_ARG;
    if (fa_tile_config(c->d, nullptr, nullptr, nullptr, nullptr) != FA_OK) return FA_ERR_UNSUPPORTED_HEAD_DIM;
    if (c->block_stride % 8 != 0 || c->slot_stride % 8 != 0 || c->head_stride % 8 != 0) return FA_ERR_INVALID_ARG;
    // axes from the innermost out: each stride spans all that lies inside it
    struct Axis { long long stride, n; } ax[3] = {{c->block_stride, c->num_blocks}, {c->slot_stride, c->page_size},
                                                  {c->head_stride, c->Hkv}};
    std::sort(ax, ax + 3, [](const Axis &a, const Axis &b) { return a.stride < b.stride; });
    long long extent = c->d;
    constexpr long long kMost = 1LL << 39;   // elements: 2^40 bytes, the tensor map's limit of a stride
    for (const Axis &a : ax) {
        if (a.n <= 1) continue;
        if (a.stride < extent || a.stride >= kMost) return FA_ERR_INVALID_ARG;
        extent += a.stride * (a.n - 1);
        if (extent >= (1LL << 46)) return FA_ERR_INVALID_ARG;
    }
    return FA_OK;
}

// k and v may be interleaved (slices of one [block, 2, ...] array): the same strides, v's base
// inside k's extent.  Then the smallest stride gap decides whether any row is shared.
inline bool caches_overlap(const fa_paged_cache *c) {
    const size_t n = cache_bytes(c);
    if (!overlaps(c->k, n, c->v, n)) return false;
    const uintptr_t a = reinterpret_cast<uintptr_t>(c->k), b = reinterpret_cast<uintptr_t>(c->v);
    const long long off = (long long)((b > a ? b - a : a - b) / 2);   // elements between the bases
    if ((b > a ? b - a : a - b) % 2 != 0) return true;
    // The rows of one array lie in a gap of some axis of the other's, and stay clear of the next
    // index of every axis outside that one.
    struct Axis { long long stride, n; } ax[3] = {{c->block_stride, c->num_blocks}, {c->slot_stride, c->page_size},
                                                  {c->head_stride, c->Hkv}};
    std::sort(ax, ax + 3, [](const Axis &x, const Axis &y) { return x.stride < y.stride; });
    long long extent = c->d;
    bool apart = false;
    for (const Axis &x : ax) {
        if (x.n <= 1) continue;
        apart = off + extent <= x.stride && (apart || off >= extent);
        extent += x.stride * (x.n - 1);
    }
    return !apart;
}

}  // namespace fa_host
