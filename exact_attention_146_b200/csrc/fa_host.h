// fa_host.h -- host-side helpers shared by the translation units of libfa.so (defined in
// fa_fwd.cu): per-device state and probing, pointer checks, TMA tensor-map encoding and a
// zero-fill launch.  Internal to the library; not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>
#include <mutex>

#include <cuda.h>
#include <cuda_runtime.h>

#include "fa.h"

namespace fa_host {

// Forward instantiations with per-device launch state: slots 0-6 bf16 and 8-14 fp16 (one per
// head dim), 15, 17 and 18 the FP8 ones (d = 128, 64, 256), 16 the failure-path test build.
// (The backward keeps its own state in fa_bwd.cu.)
constexpr int kNumCfgSlots = 19;
constexpr int kFp8Slot = 15;
constexpr int kFaultSlot = 16;
constexpr int kFp8Slot64 = 17;
constexpr int kFp8Slot256 = 18;

constexpr int kMaxDevices = 64;
constexpr int kMaxSplits = 256;

struct DeviceState {
    bool probed = false;
    bool supported = false;
    int num_sms = 0;
    int *status_ptr = nullptr;
    bool smem_attr_set[kNumCfgSlots] = {};
    int regs_ok[kNumCfgSlots] = {};   // 0 unknown, 1 verified, -1 mismatch
};

extern std::mutex g_mutex;   // guards the per-device state and lazily found addresses

// The current device's state, probed once (sm_100 or not, SM count, status word address).
int current_device(DeviceState **out, int *dev_out);
// `bytes` starting at `p` must be device (or managed) memory of device `dev`, inside one allocation.
int check_device_range(const void *p, size_t bytes, int dev);
bool overlaps(const void *a, size_t na, const void *b, size_t nb);

// One array of an entry point: where it starts, its bytes (0: empty, not looked at), its alignment.
struct Span {
    const void *p;
    size_t bytes;
    uintptr_t align;
};
// Host-only checks of an entry point's arrays: alignment, and that no output overlaps an input or
// another output.  same(i, o): input i and output o may be the same array (an in-place update).
template <class Same>
int check_layout(const Span *in, int n_in, const Span *out, int n_out, Same same) {
    for (int i = 0; i < n_in; ++i)
        if (in[i].bytes > 0 && reinterpret_cast<uintptr_t>(in[i].p) % in[i].align != 0) return FA_ERR_MISALIGNED;
    for (int o = 0; o < n_out; ++o)
        if (out[o].bytes > 0 && reinterpret_cast<uintptr_t>(out[o].p) % out[o].align != 0) return FA_ERR_MISALIGNED;
    for (int o = 0; o < n_out; ++o) {
        for (int i = 0; i < n_in; ++i)
            if (overlaps(out[o].p, out[o].bytes, in[i].p, in[i].bytes) && !same(i, o)) return FA_ERR_OVERLAP;
        for (int u = 0; u < o; ++u)
            if (overlaps(out[o].p, out[o].bytes, out[u].p, out[u].bytes)) return FA_ERR_OVERLAP;
    }
    return FA_OK;
}
// The allocations that one call's arrays have been found in.
struct SpanRanges {
    static constexpr int kMax = 16;
    int n = 0;
    uintptr_t lo[kMax], hi[kMax];
};
// check_device_range of every array that is not empty.
int check_spans(SpanRanges *seen, const Span *s, int n, int dev);

// 4-D view of a strided tensor: (d, dims) with `strides` elements, box (cw, box).
int encode_view(CUtensorMap *m, const void *base, int d, const long long (&dims)[3], const long long (&strides)[3],
                int cw, const int (&box)[3], int elem, int line = 256);
// 4-D view (d, H, N, B) of a [B, N, H, d] tensor, box (cw, heads, rows, 1); elem: 0 bf16,
// 1 fp16, 2 E4M3 bytes.
int encode_bnhd(CUtensorMap *m, const void *base, int d, int H, int N, int B, int cw, int rows, int heads = 1,
                int elem = 0);
// Zero `bytes` (a multiple of 16) at dst and set n_lse floats at lse (if not NULL) to -inf.
int zero_fill(void *dst, size_t bytes, float *lse, size_t n_lse, int num_sms, cudaStream_t st);

}  // namespace fa_host
