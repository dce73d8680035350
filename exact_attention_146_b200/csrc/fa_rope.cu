// fa_rope.cu -- rotary position embedding with one to four position axes (fa_rope, and fa_rope_append,
// which also writes the rotated keys and the values into a paged cache; declared in include/fa.h).
//
// Pair i of a head turns by the angle pos[axis_i][t] * inv_freq_i:
//     (a, b) -> (a cos - b sin, b cos + a sin),   pairs (i, i + rot/2), or (2i, 2i + 1) interleaved;
// the gradient is the same turn by the opposite angle (`inverse`).
//
// The angle is formed in fp64 as a number of whole turns, position x (inv_freq / 2 pi), whose
// fractional part goes to sincospif in fp32: at position 2^20 an fp32 product would be off by up to
// 0.06 radians, here the error is that of rounding half a turn to fp32 (2^-25).  The rot/2 angles of
// a token are computed once per CTA, into shared memory, and used by all its heads.
//
// Bound by memory: every value is read once and written once, 16 bytes a thread at a time.  A CTA
// takes TOK tokens and all heads; a thread keeps its (head, 16 values) over the TOK tokens, so the
// index arithmetic is done once and 2 TOK loads are in flight together.  The block has as many threads
// as there are such units (or an even share of them), and the first loads are on their way while the
// angles are computed.  Measured (B200, in a CUDA graph): 16384 tokens of 32 + 8 heads of 128, forward and gradient,
// 124 us (5.4 TB/s); 4 tokens a CTA (2: 141 us, 3: 150, 8: 183).
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_cache.h"
#include "fa_host.h"

namespace {

using namespace fa_host;

constexpr int kRopeThreads = 512;   // at most
constexpr int kRopeTokens = 4;      // tokens a CTA, where there are many
constexpr int kMaxPairs = 128;   // rot_dim <= 256
constexpr int kMaxAxes = 4;

struct RopeParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out, *k_out;             // k_out: rows (fa_rope) or nullptr (fa_rope_append)
    uint16_t *k_cache, *v_cache;         // fa_rope_append
    const int *positions;                // [axes][pos_stride]
    const long long *slots;              // fa_rope_append: [T], negative: the row is left out
    int *status;
    long long q_stride, qo_stride, k_stride, ko_stride, v_stride, pos_stride;   // elements per token (axis)
    long long block_stride, slot_stride, head_stride, num_slots;
    int T, Hq, Hkv, d, rot, page, interleaved;
    float sin_sign;
    double turns[kMaxPairs];             // inv_freq / 2 pi
    unsigned char axis[kMaxPairs];
};

template <bool F16>
__device__ __forceinline__ float2 unpack(uint32_t w) {
    if constexpr (F16) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    else return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
}

template <bool F16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
    if constexpr (F16) {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}

template <bool F16>
__device__ __forceinline__ float widen(uint16_t x) {
    if constexpr (F16) return __half2float(__ushort_as_half(x));
    else return __bfloat162float(__ushort_as_bfloat16(x));
}

template <bool F16>
__device__ __forceinline__ uint16_t narrow(float x) {
    if constexpr (F16) return __half_as_ushort(__float2half_rn(x));
    else return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// Shared set-up of both kernels: which of the CTA's tokens are there, where their cache rows are
// (elements; -1: left out), and their angles.
template <int TOK>
__device__ __forceinline__ void stage_tokens(const RopeParams &p, long long t0, long long (&row)[TOK], float2 *angles) {
    const int tid = int(threadIdx.x), half = p.rot / 2;
    if (tid < TOK) {
        const long long t = t0 + tid;
        long long at = t < p.T ? 0 : -1;
        if (at == 0 && p.slots != nullptr) {
            const long long slot = p.slots[t];
            if (slot < 0) {
                at = -1;
            } else if (slot >= p.num_slots) {
                at = -1;
                report_range(p.status, kSiteSlot, t);
            } else {
                at = (slot / p.page) * p.block_stride + (slot % p.page) * p.slot_stride;
            }
        }
        row[tid] = at;
    }
    // Token fastest: a warp's lanes then share few pairs (the parameters are read one address at a time).
#pragma unroll 1
    for (int w = tid; w < TOK * half; w += int(blockDim.x)) {
        const int i = w / TOK, tok = w % TOK;
        const long long t = t0 + tok;
        if (t < p.T) {
            double turn = double(p.positions[p.axis[i] * p.pos_stride + t]) * p.turns[i];
            turn -= rint(turn);
            float s, c;
            sincospif(2.f * float(turn), &s, &c);
            angles[tok * (half + 1) + i] = make_float2(c, p.sin_sign * s);   // (padded: the lanes' tokens in other banks)
        }
    }
    __syncthreads();
}

// One head's rows for this CTA: source and destination of the unit's head at token t0.
struct Lane {
    const uint16_t *src;
    uint16_t *dst;            // rows: + tok * dst_stride; cache: + row[tok]
    long long src_stride, dst_stride;
    bool cache, turn;
};

__device__ __forceinline__ Lane head_lane(const RopeParams &p, int h, long long t0) {
    Lane l;
    if (h < p.Hq) {
        l = {p.q + t0 * p.q_stride + (long long)h * p.d, p.q_out + t0 * p.qo_stride + (long long)h * p.d, p.q_stride,
             p.qo_stride, false, true};
    } else if (h < p.Hq + p.Hkv) {
        const long long kh = h - p.Hq;
        l.src = p.k + t0 * p.k_stride + kh * p.d;
        l.src_stride = p.k_stride;
        l.cache = p.k_out == nullptr;
        l.dst = l.cache ? p.k_cache + kh * p.head_stride : p.k_out + t0 * p.ko_stride + kh * p.d;
        l.dst_stride = p.ko_stride;
        l.turn = true;
    } else {
        const long long vh = h - p.Hq - p.Hkv;
        l = {p.v + t0 * p.v_stride + vh * p.d, p.v_cache + vh * p.head_stride, p.v_stride, 0, true, false};
    }
    return l;
}

// N words of a row, one vector.
template <int N>
__device__ __forceinline__ void load_words(uint32_t (&x)[N], const uint16_t *src) {
    if constexpr (N == 4) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(src));
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else {
        const uint2 v = __ldcs(reinterpret_cast<const uint2 *>(src));
        x[0] = v.x, x[1] = v.y;
    }
}
template <int N>
__device__ __forceinline__ void store_words(uint16_t *dst, const uint32_t (&x)[N]) {
    if constexpr (N == 4) *reinterpret_cast<uint4 *>(dst) = make_uint4(x[0], x[1], x[2], x[3]);
    else *reinterpret_cast<uint2 *>(dst) = make_uint2(x[0], x[1]);
}

// Vector path: every row 16-byte aligned, and rot a multiple of 2 W (W = 8, or 4 where rot / 2 is an odd
// number of fours).  A unit is 2 W values of one head: for the rotated part W pairs (two runs of W
// values rot/2 apart, or one run of 2 W interleaved), else 2 W values that are copied.
template <bool F16, int TOK, int W>
__global__ void __launch_bounds__(kRopeThreads, 2) fa_rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr int N = W / 2;   // words a run
    extern __shared__ float2 angles[];
    __shared__ long long row[TOK];
    const long long t0 = (long long)blockIdx.x * TOK;
    const int half = p.rot / 2, per_head = p.d / (2 * W);
    const int heads = p.Hq + p.Hkv + (p.v_cache != nullptr ? p.Hkv : 0), units = heads * per_head;
    const int here = int(min((long long)TOK, p.T - t0));   // tokens of this CTA
    bool staged = false;
    for (int u = int(threadIdx.x); u < units || !staged; u += int(blockDim.x)) {
        const int h = u / per_head, i = u - h * per_head;
        Lane l{};
        if (u < units) l = head_lane(p, h, t0);
        const bool turn = l.turn && 2 * W * i < p.rot;
        const bool split = turn && p.interleaved == 0;
        const int e0 = split ? W * i : 2 * W * i, e1 = split ? half + W * i : 2 * W * i + W;
        const int a0 = W * i;   // first pair of the unit
        uint32_t x[TOK][2][N];
#pragma unroll
        for (int tok = 0; tok < TOK; ++tok) {
            if (u < units && tok < here) {
                load_words<N>(x[tok][0], l.src + tok * l.src_stride + e0);
                load_words<N>(x[tok][1], l.src + tok * l.src_stride + e1);
            }
        }
        if (!staged) {   // (every thread comes here once: in its first round, with a unit or without)
            stage_tokens<TOK>(p, t0, row, angles);
            staged = true;
        }
        if (u >= units) break;
#pragma unroll
        for (int tok = 0; tok < TOK; ++tok) {
            if (row[tok] < 0) continue;
            uint32_t (&a)[N] = x[tok][0], (&b)[N] = x[tok][1];
            if (turn) {
                const float2 *cs = angles + tok * (half + 1) + a0;
#pragma unroll
                for (int w = 0; w < N; ++w) {
                    const float2 lo = unpack<F16>(a[w]), hi = unpack<F16>(b[w]);
                    if (split) {
                        const float2 r0 = cs[2 * w], r1 = cs[2 * w + 1];
                        a[w] = pack<F16>(lo.x * r0.x - hi.x * r0.y, lo.y * r1.x - hi.y * r1.y);
                        b[w] = pack<F16>(hi.x * r0.x + lo.x * r0.y, hi.y * r1.x + lo.y * r1.y);
                    } else {
                        const float2 r0 = cs[w], r1 = cs[N + w];
                        a[w] = pack<F16>(lo.x * r0.x - lo.y * r0.y, lo.y * r0.x + lo.x * r0.y);
                        b[w] = pack<F16>(hi.x * r1.x - hi.y * r1.y, hi.y * r1.x + hi.x * r1.y);
                    }
                }
            }
            uint16_t *dst = l.dst + (l.cache ? row[tok] : tok * l.dst_stride);
            store_words<N>(dst + e0, a);
            store_words<N>(dst + e1, b);
        }
    }
}

// Any even rot <= d and any alignment: a unit is one pair, or one value that is copied.
template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) fa_rope_any_kernel(const __grid_constant__ RopeParams p) {
    extern __shared__ float2 angles[];
    __shared__ long long row[1];
    const long long t0 = blockIdx.x;
    stage_tokens<1>(p, t0, row, angles);
    if (row[0] < 0) return;
    const int half = p.rot / 2;
    const int heads = p.Hq + p.Hkv + (p.v_cache != nullptr ? p.Hkv : 0);
    const int per_head = half + (p.d - p.rot);   // pairs, then single values
    for (int u = int(threadIdx.x); u < heads * per_head; u += int(blockDim.x)) {
        const int h = u / per_head, i = u - h * per_head;
        const Lane l = head_lane(p, h, t0);
        uint16_t *dst = l.dst + (l.cache ? row[0] : 0);
        if (i < half) {
            const int e0 = p.interleaved ? 2 * i : i, e1 = p.interleaved ? 2 * i + 1 : i + half;
            const uint16_t xa = l.src[e0], xb = l.src[e1];
            uint16_t ya = xa, yb = xb;
            if (l.turn) {
                const float a = widen<F16>(xa), b = widen<F16>(xb);
                const float2 r = angles[i];
                ya = narrow<F16>(a * r.x - b * r.y);
                yb = narrow<F16>(b * r.x + a * r.y);
            }
            dst[e0] = ya;
            dst[e1] = yb;
        } else {
            const int e = p.rot + (i - half);
            dst[e] = l.src[e];
        }
    }
}

template <bool F16, int W>
void launch_vec(const RopeParams &p, int num_sms, unsigned threads, size_t per_token, cudaStream_t st) {
    if (p.T <= 4 * num_sms) {
        fa_rope_kernel<F16, 1, W><<<unsigned(p.T), threads, per_token, st>>>(p);
    } else {
        constexpr int TOK = kRopeTokens;
        fa_rope_kernel<F16, TOK, W><<<unsigned((p.T + TOK - 1) / TOK), threads, TOK * per_token, st>>>(p);
    }
}

template <bool F16>
int launch(const RopeParams &p, bool vec, int num_sms, cudaStream_t st) {
    const size_t per_token = size_t(p.rot / 2 + 1) * sizeof(float2);
    const int heads = p.Hq + p.Hkv + (p.v_cache != nullptr ? p.Hkv : 0), width = p.rot % 16 == 0 ? 8 : 4;
    vec = vec && p.rot % 8 == 0;
    const int units = vec ? heads * (p.d / (2 * width)) : heads * (p.d - p.rot / 2), rounds = (units + kRopeThreads - 1) / kRopeThreads;
    const unsigned threads = unsigned(((units + rounds - 1) / rounds + 31) / 32 * 32);
    if (!vec) fa_rope_any_kernel<F16><<<unsigned(p.T), threads, per_token, st>>>(p);
    else if (width == 8) launch_vec<F16, 8>(p, num_sms, threads, per_token, st);
    else launch_vec<F16, 4>(p, num_sms, threads, per_token, st);
    return cudaGetLastError() == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

// Rows [T, H, d] with `stride` elements from token to token: 0 bytes if there are none.
size_t rows_bytes(int T, int H, int d, long long stride) {
    return T == 0 || H == 0 ? 0 : (size_t(T - 1) * size_t(stride) + size_t(H) * size_t(d)) * 2;
}

bool valid_spec(const fa_rope_spec *s, int d) {
    if (s->rot_dim < 0 || s->rot_dim % 2 != 0 || s->rot_dim > d || s->num_axes < 1 || s->num_axes > kMaxAxes) return false;
    if (s->interleaved != 0 && s->interleaved != 1) return false;
    if (s->rot_dim > 0 && s->inv_freq == nullptr) return false;
    for (int i = 0; i < s->rot_dim / 2; ++i) {
        if (!std::isfinite(s->inv_freq[i])) return false;
        if (s->axis != nullptr && (s->axis[i] < 0 || s->axis[i] >= s->num_axes)) return false;
    }
    return true;
}

void fill_spec(RopeParams *p, const fa_rope_spec *s, int inverse) {
    p->rot = s->rot_dim;
    p->interleaved = s->interleaved;
    p->sin_sign = inverse ? -1.f : 1.f;
    for (int i = 0; i < s->rot_dim / 2; ++i) {
        p->turns[i] = s->inv_freq[i] * 0.15915494309189533577;   // 1 / 2 pi
        p->axis[i] = static_cast<unsigned char>(s->axis != nullptr ? s->axis[i] : 0);
    }
}

bool head_dim_ok(int d) { return fa_tile_config(d, nullptr, nullptr, nullptr, nullptr) == FA_OK; }

bool vec_rows(const void *p, long long stride) { return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride % 8 == 0; }

int rope(const void *q, long long q_stride, void *q_out, long long qo_stride, int Hq, const void *k, long long k_stride,
         void *k_out, long long ko_stride, int Hkv, int T, int d, const int *positions, long long pos_stride,
         const fa_rope_spec *spec, int inverse, bool f16, void *stream) {
    if (T < 0 || Hq < 0 || Hkv < 0 || spec == nullptr || (inverse != 0 && inverse != 1)) return FA_ERR_INVALID_ARG;
    if (!head_dim_ok(d)) return FA_ERR_UNSUPPORTED_HEAD_DIM;
    if (!valid_spec(spec, d)) return FA_ERR_INVALID_ARG;
    if (T == 0 || Hq + Hkv == 0) return FA_OK;
    if (Hq > 0 && (q == nullptr || q_out == nullptr || q_stride < (long long)Hq * d || qo_stride < (long long)Hq * d))
        return FA_ERR_INVALID_ARG;
    if (Hkv > 0 && (k == nullptr || k_out == nullptr || k_stride < (long long)Hkv * d || ko_stride < (long long)Hkv * d))
        return FA_ERR_INVALID_ARG;
    if (positions == nullptr || (pos_stride != 0 && pos_stride < T) || Hq > 65535 || Hkv > 65535) return FA_ERR_INVALID_ARG;
    const size_t pos_b = (size_t(spec->num_axes - 1) * size_t(pos_stride) + size_t(T)) * 4;
    const Span in[] = {{q, rows_bytes(T, Hq, d, q_stride), 2}, {k, rows_bytes(T, Hkv, d, k_stride), 2}, {positions, pos_b, 4}};
    const Span out[] = {{q_out, rows_bytes(T, Hq, d, qo_stride), 2}, {k_out, rows_bytes(T, Hkv, d, ko_stride), 2}};
    // In place: each value is read and written by one thread, so exactly the same rows may be
    // given.  Slices of one fused projection interleave q's and k's rows without sharing any.
    int rc = check_layout(in, 3, out, 0, [](int, int) { return false; });
    if (rc != FA_OK) return rc;
    for (const Span &o : out)
        if (o.bytes > 0 && reinterpret_cast<uintptr_t>(o.p) % o.align != 0) return FA_ERR_MISALIGNED;
    const Rows rq{q, q_stride, Hq * d}, rk{k, k_stride, Hkv * d}, rqo{q_out, qo_stride, Hq * d}, rko{k_out, ko_stride, Hkv * d};
    if (Hq > 0 && !same_rows(rq, rqo) && rows_overlap(rqo, rq, T, 2)) return FA_ERR_OVERLAP;
    if (Hkv > 0 && !same_rows(rk, rko) && rows_overlap(rko, rk, T, 2)) return FA_ERR_OVERLAP;
    if (Hq > 0 && Hkv > 0 && (rows_overlap(rqo, rk, T, 2) || rows_overlap(rko, rq, T, 2) || rows_overlap(rqo, rko, T, 2)))
        return FA_ERR_OVERLAP;
    for (const Span &o : out)
        if (overlaps(o.p, o.bytes, positions, pos_b)) return FA_ERR_OVERLAP;
    DeviceState *dev = nullptr;
    int dev_id = -1;
    if ((rc = current_device(&dev, &dev_id)) != FA_OK) return rc;
    SpanRanges seen;
    if ((rc = check_spans(&seen, in, 3, dev_id)) != FA_OK || (rc = check_spans(&seen, out, 2, dev_id)) != FA_OK) return rc;
    RopeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_out = static_cast<uint16_t *>(k_out);
    p.positions = positions;
    p.status = dev->status_ptr;
    p.q_stride = q_stride;
    p.qo_stride = qo_stride;
    p.k_stride = k_stride;
    p.ko_stride = ko_stride;
    p.pos_stride = pos_stride;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.d = d;
    p.page = 1;
    fill_spec(&p, spec, inverse);
    const bool vec = (Hq == 0 || (vec_rows(q, q_stride) && vec_rows(q_out, qo_stride))) &&
                     (Hkv == 0 || (vec_rows(k, k_stride) && vec_rows(k_out, ko_stride)));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return f16 ? launch<true>(p, vec, dev->num_sms, st) : launch<false>(p, vec, dev->num_sms, st);
}

int rope_append(const void *q, long long q_stride, void *q_out, long long qo_stride, int Hq, const void *k,
                long long k_stride, const void *v, long long v_stride, int T, const int *positions, long long pos_stride,
                const fa_rope_spec *spec, const fa_paged_cache *given, const long long *slots, bool f16, void *stream) {
    if (T < 0 || Hq < 0 || spec == nullptr || given == nullptr) return FA_ERR_INVALID_ARG;
    const fa_paged_cache tidy = tidy_cache(*given), *cache = &tidy;
    const int rc0 = valid_cache(cache);
    if (rc0 != FA_OK) return rc0;
    const int d = cache->d, Hkv = cache->Hkv;
    if (!valid_spec(spec, d)) return FA_ERR_INVALID_ARG;
    if (T == 0) return FA_OK;
    if (Hq > 0 && (q == nullptr || q_out == nullptr || q_stride < (long long)Hq * d || qo_stride < (long long)Hq * d))
        return FA_ERR_INVALID_ARG;
    if (k == nullptr || v == nullptr || k_stride < (long long)Hkv * d || v_stride < (long long)Hkv * d) return FA_ERR_INVALID_ARG;
    if (slots == nullptr || positions == nullptr || (pos_stride != 0 && pos_stride < T) || Hq > 65535 || Hkv > 65535) return FA_ERR_INVALID_ARG;
    const size_t pos_b = (size_t(spec->num_axes - 1) * size_t(pos_stride) + size_t(T)) * 4;
    const size_t cache_b = cache_bytes(cache);
    if (cache_b > 0 && (cache->k == nullptr || cache->v == nullptr)) return FA_ERR_INVALID_ARG;
    const Span in[] = {{q, rows_bytes(T, Hq, d, q_stride), 2}, {k, rows_bytes(T, Hkv, d, k_stride), 2},
                       {v, rows_bytes(T, Hkv, d, v_stride), 2}, {positions, pos_b, 4}, {slots, size_t(T) * 8, 8}};
    const Span out[] = {{q_out, rows_bytes(T, Hq, d, qo_stride), 2}, {cache->k, cache_b, 16}, {cache->v, cache_b, 16}};
    const Rows rq{q, q_stride, Hq * d}, rqo{q_out, qo_stride, Hq * d};
    const Rows rk{k, k_stride, Hkv * d}, rv{v, v_stride, Hkv * d};
    int rc = check_layout(in, 5, out, 1, [&](int i, int) {   // q_out: q itself, or rows between those of k and v
        if (i == 0) return same_rows(rq, rqo) || !rows_overlap(rqo, rq, T, 2);
        return (i == 1 && !rows_overlap(rqo, rk, T, 2)) || (i == 2 && !rows_overlap(rqo, rv, T, 2));
    });
    if (rc != FA_OK) return rc;
    for (int o = 1; o < 3; ++o) {
        if (out[o].bytes > 0 && reinterpret_cast<uintptr_t>(out[o].p) % out[o].align != 0) return FA_ERR_MISALIGNED;
        for (const Span &s : in)
            if (overlaps(out[o].p, out[o].bytes, s.p, s.bytes)) return FA_ERR_OVERLAP;
        if (overlaps(out[o].p, out[o].bytes, q_out, out[0].bytes)) return FA_ERR_OVERLAP;
    }
    if (caches_overlap(cache)) return FA_ERR_OVERLAP;
    DeviceState *dev = nullptr;
    int dev_id = -1;
    if ((rc = current_device(&dev, &dev_id)) != FA_OK) return rc;
    SpanRanges seen;
    if ((rc = check_spans(&seen, in, 5, dev_id)) != FA_OK || (rc = check_spans(&seen, out, 3, dev_id)) != FA_OK) return rc;
    RopeParams p{};
    p.q = static_cast<const uint16_t *>(q);
    p.k = static_cast<const uint16_t *>(k);
    p.v = static_cast<const uint16_t *>(v);
    p.q_out = static_cast<uint16_t *>(q_out);
    p.k_cache = static_cast<uint16_t *>(cache->k);
    p.v_cache = static_cast<uint16_t *>(cache->v);
    p.positions = positions;
    p.slots = slots;
    p.status = dev->status_ptr;
    p.q_stride = q_stride;
    p.qo_stride = qo_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.pos_stride = pos_stride;
    p.block_stride = cache->block_stride;
    p.slot_stride = cache->slot_stride;
    p.head_stride = cache->head_stride;
    p.num_slots = (long long)cache->num_blocks * cache->page_size;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.d = d;
    p.page = cache->page_size;
    fill_spec(&p, spec, 0);
    const bool vec = (Hq == 0 || (vec_rows(q, q_stride) && vec_rows(q_out, qo_stride))) &&
                     vec_rows(k, k_stride) && vec_rows(v, v_stride);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    return f16 ? launch<true>(p, vec, dev->num_sms, st) : launch<false>(p, vec, dev->num_sms, st);
}

}  // namespace

extern "C" {

int fa_rope(const void *q, long long q_stride, void *q_out, long long qo_stride, int Hq, const void *k,
            long long k_stride, void *k_out, long long ko_stride, int Hkv, int T, int d, const int *positions,
            long long pos_stride, const fa_rope_spec *spec, int inverse, void *stream) {
    return rope(q, q_stride, q_out, qo_stride, Hq, k, k_stride, k_out, ko_stride, Hkv, T, d, positions, pos_stride,
                spec, inverse, false, stream);
}

int fa_rope_f16(const void *q, long long q_stride, void *q_out, long long qo_stride, int Hq, const void *k,
                long long k_stride, void *k_out, long long ko_stride, int Hkv, int T, int d, const int *positions,
                long long pos_stride, const fa_rope_spec *spec, int inverse, void *stream) {
    return rope(q, q_stride, q_out, qo_stride, Hq, k, k_stride, k_out, ko_stride, Hkv, T, d, positions, pos_stride,
                spec, inverse, true, stream);
}

int fa_rope_append(const void *q, long long q_stride, void *q_out, long long qo_stride, int Hq, const void *k,
                   long long k_stride, const void *v, long long v_stride, int T, const int *positions,
                   long long pos_stride, const fa_rope_spec *spec, const fa_paged_cache *cache,
                   const long long *slots, void *stream) {
    return rope_append(q, q_stride, q_out, qo_stride, Hq, k, k_stride, v, v_stride, T, positions, pos_stride, spec,
                       cache, slots, false, stream);
}

int fa_rope_append_f16(const void *q, long long q_stride, void *q_out, long long qo_stride, int Hq, const void *k,
                       long long k_stride, const void *v, long long v_stride, int T, const int *positions,
                       long long pos_stride, const fa_rope_spec *spec, const fa_paged_cache *cache,
                       const long long *slots, void *stream) {
    return rope_append(q, q_stride, q_out, qo_stride, Hq, k, k_stride, v, v_stride, T, positions, pos_stride, spec,
                       cache, slots, true, stream);
}

}  // extern "C"
