// The 8-bit KV cache: shared argument block, and the kernels that quantise rows as they are written and
// read them back.
//
// Values are e4m3 codes with one scale for each block of `scale_block` consecutive slots of a page, for
// K and V and each kv head on their own: x ~ s * code. s is the smallest power of two with
// amax <= 448 s, so code = rn(x / s) has a relative error of at most 2^-4 down to 2^-6 s and an
// absolute one of 2^-10 s below. Powers of two make growing a scale harmless: when a later row of a
// block needs a larger s, code * old/new is exact but where it falls below 2^-6 (a subnormal code).
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"

namespace sdv {

// Division of 0 <= n < 2^31 by a fixed d >= 1 as a multiplication: floor(n m / 2^(31 + l)) with
// l = ceil(log2 d), m = floor(2^(31 + l) / d) + 1 < 2^32. m d exceeds 2^(31 + l) by at most d <= 2^l, so the
// quotient is off by less than n / 2^31 / d < 1 / d: never across a whole number.
struct FastDiv {
    uint32_t m;
    int shift;
    static FastDiv of(uint32_t d) {
        int l = 0;
        while ((1ull << l) < d) ++l;
        return {static_cast<uint32_t>((1ull << (31 + l)) / d + 1), 31 + l};
    }
    __device__ __forceinline__ int div(int n) const {
        return static_cast<int>(static_cast<unsigned long long>(static_cast<uint32_t>(n)) * m >> shift);
    }
};

struct QCacheArgs {
    uint8_t *codes;   // the layer's [n_pages][2][nkv][page_size][D]
    float *scales;    // the layer's [n_pages][2][nkv][page_size / scale_block]
    int *status;
    const int *page_table, *row_off, *base;
    int pages_per_seq, page_size, n_pages, scale_block, nkv, B, max_span, max_rows, max_context;
    int blocks;                           // scale blocks of a page
    FastDiv by_page, by_block, by_heads;  // page_size, scale_block, 2 nkv
};

// One sequence's span: rows r0 .. r0 + S - 1 at positions p0 .. p0 + S - 1. S = 0 where it is empty or
// refused (then `code` says why and the span's own rows, if they lie in the call's rows, are `rows`).
struct QSpan {
    int r0, S, p0, rows, code;
};
__device__ __forceinline__ QSpan qcache_span(const QCacheArgs &a, int b) {
    QSpan s;
    s.r0 = a.row_off[b];
    s.S = a.row_off[b + 1] - s.r0;
    s.p0 = a.base[b];
    s.rows = 0;
    s.code = SDV_OK;
    if (s.S == 0) return s;
    if (s.S < 0 || s.r0 < 0 || s.S > a.max_rows || s.r0 > a.max_rows - s.S) {
        s.code = SDV_ERR_ARG;
    } else if (s.S > a.max_span) {
        s.code = SDV_ERR_ARG;
        s.rows = s.S;
    } else if (s.p0 < 0 || s.p0 > a.max_context - s.S) {
        s.code = SDV_ERR_CAPACITY;
        s.rows = s.S;
    }
    if (s.code != SDV_OK) s.S = 0;
    return s;
}

// Page of a sequence's page-table slot, or -1 (and the status word) where its id is not in the pool.
__device__ __forceinline__ int qcache_page(const QCacheArgs &a, int b, int slot) {
    const int page = a.page_table[static_cast<size_t>(b) * a.pages_per_seq + slot];
    if (page >= 0 && page < a.n_pages) return page;
    set_status(a.status, SDV_ERR_CAPACITY);
    return -1;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ bf16 from_f32<bf16>(float x) { return __float2bfloat16(x); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half(x); }

// Eight values of a row as they lie in memory, from a row that is 16-byte aligned or (VEC false) not.
template <typename T>
struct Raw8 {
    uint4 u[sizeof(T) / 2];
    __device__ __forceinline__ float at(int k) const { return to_f32(reinterpret_cast<const T *>(u)[k]); }
    // The larger of `m` and the values' magnitudes; not below infinity where one of them is not finite. Magnitudes of a
    // type order like their bits, and so above infinity do NaNs.
    __device__ __forceinline__ uint32_t top(uint32_t m) const {
        const uint32_t *w = reinterpret_cast<const uint32_t *>(u);
#pragma unroll
        for (int k = 0; k < static_cast<int>(sizeof(u)) / 4; ++k) {
            if constexpr (sizeof(T) == 4)
                m = max(m, w[k] & 0x7fffffffu);
            else
                m = __vmaxu2(m, w[k] & 0x7fff7fffu);
        }
        return m;
    }
    static __device__ __forceinline__ float top_value(uint32_t m) {
        if constexpr (sizeof(T) == 4) return __uint_as_float(m);
        const unsigned short h = static_cast<unsigned short>(max(m & 0xffffu, m >> 16));
        if constexpr (sizeof(T) == 2) return to_f32(*reinterpret_cast<const T *>(&h));
        return 0.f;
    }
};
template <typename T, bool VEC>
__device__ __forceinline__ Raw8<T> load_raw8(const T *src) {
    Raw8<T> r;
    if constexpr (VEC) {
#pragma unroll
        for (int w = 0; w < static_cast<int>(sizeof(T)) / 2; ++w) r.u[w] = __ldg(reinterpret_cast<const uint4 *>(src) + w);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) reinterpret_cast<T *>(r.u)[k] = src[k];
    }
    return r;
}
// Two fp32 values as e4m3 codes (round to nearest even, clamped to +-448): lo in bits 0-7.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 e4m3x2_f32(uint32_t c) {
    const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c), __NV_E4M3);
    return __half22float2(__half2(h));
}

// The smallest power of two s >= 2^-126 with amax <= 448 s (448 = 1.75 * 2^8), for a finite amax >= 0.
__device__ __forceinline__ float e4m3_scale(float amax) {
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 127 - ((u & 0x7fffffu) <= 0x600000u ? 8 : 7);
    return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}

constexpr int kQWriteThreads = 256;
constexpr int kQHold = 8;  // rows a lane holds between finding the scale and rounding: 16 rows a block at D = 128

// A warp quantises one block: (sequence, block of its span, K or V, kv head). Lanes hold eight values
// each, 32 / (D / 8) rows at a time; the first kQHold of a lane's rows stay in registers, those of longer
// blocks are read twice. A block that the span starts inside keeps its scale or a larger one, and its rows
// below the span are rounded again by the ratio of the two. Warps of a CTA take K and V of neighbouring
// heads, whose rows lie side by side.
// Bound by memory: two bytes in and one out a value (bf16). A lane's eight loads before the first use carry it: 16
// prompts of up to 4,096 tokens (8 heads of 128, 302 MB) take 49.1 us, 6.15 TB/s of the 6.77 that a copy reaches; 128
// rows of a verify step take 2.5 us, a launch and three dependent loads (span, page, scale).
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kQWriteThreads, VEC && sizeof(T) == 2 ? 4 : 2) qcache_write_kernel(QCacheArgs a, const T *k, const T *v,
                                                                      long long k_stride, long long v_stride) {
    pdl_wait();
    pdl_trigger();
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const int item = blockIdx.x * (kQWriteThreads / 32) + threadIdx.x / 32;
    const int b = blockIdx.y, lane = threadIdx.x % 32;
    const int blk = a.by_heads.div(item), kvh = item - blk * 2 * a.nkv, kv = kvh >= a.nkv, h = kvh - kv * a.nkv;
    const QSpan s = qcache_span(a, b);
    if (s.S == 0) {
        if (s.code != SDV_OK && item == 0 && lane == 0) set_status(a.status, s.code);
        return;
    }
    const int tok0 = (a.by_block.div(s.p0) + blk) * a.scale_block;
    if (tok0 >= s.p0 + s.S) return;
    const int lo = max(tok0, s.p0), hi = min(tok0 + a.scale_block, s.p0 + s.S);
    const int col = lane % LPR * 8, sub = lane / LPR;
    const long long stride = kv ? v_stride : k_stride;
    const T *src = (kv ? v : k) + (s.r0 + (lo + sub - s.p0)) * stride + h * D + col;
    Raw8<T> x[kQHold];
#pragma unroll
    for (int n = 0; n < kQHold; ++n)
        if (lo + sub + n * RPI < hi) x[n] = load_raw8<T, VEC>(src + n * RPI * stride);
    const int slots = a.by_page.div(tok0), slot0 = tok0 - slots * a.page_size, page = qcache_page(a, b, slots);
    if (page < 0) return;
    const size_t ph = (static_cast<size_t>(page) * 2 + kv) * a.nkv + h;
    uint8_t *dst = a.codes + (ph * a.page_size + slot0) * D;  // the block's first slot
    float *scale = a.scales + ph * a.blocks + a.by_block.div(slot0);
    const float was = lo > tok0 ? *scale : 0.f;
    uint32_t m = 0;
#pragma unroll
    for (int n = 0; n < kQHold; ++n)
        if (lo + sub + n * RPI < hi) m = x[n].top(m);
    for (int t = lo + sub + kQHold * RPI; t < hi; t += RPI) m = load_raw8<T, VEC>(src + (t - lo - sub) * stride).top(m);
    float amax = Raw8<T>::top_value(m);
    if (__any_sync(0xffffffffu, !(amax < INFINITY))) {  // values that are not finite do not count
        amax = 0.f;
        for (int t = lo + sub; t < hi; t += RPI) {
            const Raw8<T> r = load_raw8<T, VEC>(src + (t - lo - sub) * stride);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(r.at(j)) < INFINITY ? fabsf(r.at(j)) : 0.f);
        }
        if (lane == 0) set_status(a.status, SDV_ERR_DEVICE);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float now = e4m3_scale(amax);
    if (lo > tok0) {
        const float old = was > 0.f && was < INFINITY ? was : 0.f;  // 0: never written, nothing below the span counts
        now = fmaxf(now, old);
        const float ratio = old / now;
        if (ratio != 1.f)
            for (int t = tok0 + sub; t < lo; t += RPI) {
                uint2 *c = reinterpret_cast<uint2 *>(dst + (t - tok0) * D + col);
                const uint2 w = *c;
                uint32_t r[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = e4m3x2_f32(r[j]);
                    r[j] = e4m3x2(f.x * ratio, f.y * ratio);
                }
                *c = make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
            }
    }
    const float inv = 1.f / now;  // exact: a power of two from 2^-127 to 2^126
    auto put = [&](int t, const Raw8<T> &r) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float f = r.at(2 * j), g = r.at(2 * j + 1);
            w[j] = e4m3x2(f == f ? f * inv : 0.f, g == g ? g * inv : 0.f);
        }
        *reinterpret_cast<uint2 *>(dst + (t - tok0) * D + col) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
    };
#pragma unroll
    for (int n = 0; n < kQHold; ++n)
        if (lo + sub + n * RPI < hi) put(lo + sub + n * RPI, x[n]);
    for (int t = lo + sub + kQHold * RPI; t < hi; t += RPI) put(t, load_raw8<T, VEC>(src + (t - lo - sub) * stride));
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = now;
}

// Blocks of 1, 2, 4 or 8 tokens: a warp takes a window of kQHold * (32 / (D / 8)) tokens (16 at D = 128),
// whole blocks of it, so that a lane still has kQHold rows under way (one block a warp wrote 65,536 rows of one
// token a block in 8 times the time). Each row finds its page; the rows of a block agree on its maximum by
// shuffles and, past a warp's width of rows, across the rows a lane holds. The same prompts with a scale a token: 110 us,
// bound by the per-row work (a page, a scale and a store of eight bytes a lane; 184 bytes spilled); fp32 rows in blocks of 4: 148 us
// (82 in blocks of 16).
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kQWriteThreads, VEC && sizeof(T) == 2 ? 3 : 2) qcache_write_small_kernel(
    QCacheArgs a, const T *k, const T *v, long long k_stride, long long v_stride) {
    pdl_wait();
    pdl_trigger();
    constexpr int LPR = D / 8, RPI = 32 / LPR, WIN = kQHold * RPI;
    const int item = blockIdx.x * (kQWriteThreads / 32) + threadIdx.x / 32;
    const int b = blockIdx.y, lane = threadIdx.x % 32;
    const int win = a.by_heads.div(item), kvh = item - win * 2 * a.nkv, kv = kvh >= a.nkv, h = kvh - kv * a.nkv;
    const QSpan s = qcache_span(a, b);
    if (s.S == 0) {
        if (s.code != SDV_OK && item == 0 && lane == 0) set_status(a.status, s.code);
        return;
    }
    const int t0 = (s.p0 / WIN + win) * WIN, sb = a.scale_block;
    if (t0 >= s.p0 + s.S) return;
    const int lo = max(t0, s.p0), hi = min(t0 + WIN, s.p0 + s.S), live0 = lo & ~(sb - 1);  // sb is a power of two
    const int col = lane % LPR * 8, sub = lane / LPR;
    const long long stride = kv ? v_stride : k_stride;
    const T *src = (kv ? v : k) + h * D + col;
    Raw8<T> x[kQHold];
    uint8_t *dst[kQHold];
    float *scale[kQHold], was[kQHold];
#pragma unroll
    for (int n = 0; n < kQHold; ++n) {
        const int t = t0 + sub + n * RPI;
        if (t >= lo && t < hi) x[n] = load_raw8<T, VEC>(src + (s.r0 + (t - s.p0)) * stride);
    }
#pragma unroll
    for (int n = 0; n < kQHold; ++n) {
        const int t = t0 + sub + n * RPI;
        dst[n] = nullptr;
        was[n] = 0.f;
        scale[n] = nullptr;
        if (t >= live0 && t < hi) {
            const int at = a.by_page.div(t), slot = t - at * a.page_size, page = qcache_page(a, b, at);
            if (page >= 0) {
                const size_t ph = (static_cast<size_t>(page) * 2 + kv) * a.nkv + h;
                dst[n] = a.codes + (ph * a.page_size + slot) * D + col;
                scale[n] = a.scales + ph * a.blocks + a.by_block.div(slot);
                if (live0 < lo && (t & ~(sb - 1)) == live0) was[n] = *scale[n];
            }
        }
    }
    float peak[kQHold];
#pragma unroll
    for (int n = 0; n < kQHold; ++n) {
        const int t = t0 + sub + n * RPI;
        const bool mine = t >= lo && t < hi;
        float m = mine ? Raw8<T>::top_value(x[n].top(0)) : 0.f;
        if (mine && !(m < INFINITY)) {  // values that are not finite do not count
            m = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(x[n].at(j)) < INFINITY ? fabsf(x[n].at(j)) : 0.f);
            set_status(a.status, SDV_ERR_DEVICE);
        }
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll
        for (int r = 1; r < RPI; r <<= 1)
            if (r < sb) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, r * LPR));
        peak[n] = m;
    }
#pragma unroll
    for (int g = 2; g <= kQHold / 2; g <<= 1)  // blocks that go on in the next rows of a lane
        if (sb >= g * RPI) {
#pragma unroll
            for (int n = 0; n < kQHold; n += g) {
                const float m = fmaxf(peak[n], peak[n + g / 2]);
#pragma unroll
                for (int j = 0; j < g; ++j) peak[n + j] = m;
            }
        }
    __syncwarp();  // the old scales are read
#pragma unroll
    for (int n = 0; n < kQHold; ++n) {
        const int t = t0 + sub + n * RPI;
        if (!dst[n]) continue;
        const float old = was[n] > 0.f && was[n] < INFINITY ? was[n] : 0.f;
        const float now = fmaxf(e4m3_scale(peak[n]), old);
        uint32_t w[4];
        if (t >= lo) {
            const float inv = 1.f / now;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float f = x[n].at(2 * j), g = x[n].at(2 * j + 1);
                w[j] = e4m3x2(f == f ? f * inv : 0.f, g == g ? g * inv : 0.f);
            }
        } else {  // a row below the span in the block that it starts inside
            const float ratio = old / now;
            if (ratio == 1.f) continue;
            const uint2 c = *reinterpret_cast<const uint2 *>(dst[n]);
            const uint32_t r[4] = {c.x & 0xffffu, c.x >> 16, c.y & 0xffffu, c.y >> 16};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = e4m3x2_f32(r[j]);
                w[j] = e4m3x2(f.x * ratio, f.y * ratio);
            }
        }
        *reinterpret_cast<uint2 *>(dst[n]) = make_uint2(w[0] | w[1] << 16, w[2] | w[3] << 16);
        if (t >= lo && col == 0 && (t == lo || (t & (sb - 1)) == 0)) *scale[n] = now;
    }
}

constexpr int kQReadThreads = 256;
constexpr int kQReadRows = 4;  // rows a thread reads, so that many loads are under way

// Eight codes of a row a thread and kQReadRows rows: code * scale (exact in fp32 but where it leaves
// fp32's range), rounded once. Grid (K|V x heads, span rows in groups, sequences): neighbouring CTAs fill
// neighbouring parts of the same output rows. Bound by memory, two thirds of it writes: the prompts above come back in
// 48.1 us, 6.3 TB/s; 509 rows as fp32 in 3.2 us.
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kQReadThreads) qcache_read_kernel(QCacheArgs a, T *k, T *v, long long k_stride,
                                                                    long long v_stride) {
    pdl_wait();
    pdl_trigger();
    constexpr int LPR = D / 8, RPB = kQReadThreads / LPR;
    const int b = blockIdx.z, kv = blockIdx.x >= a.nkv, h = blockIdx.x - kv * a.nkv;
    const QSpan s = qcache_span(a, b);
    if (s.S == 0) {
        if (s.code != SDV_OK && blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) set_status(a.status, s.code);
        return;
    }
    const int i0 = blockIdx.y * RPB * kQReadRows + threadIdx.x / LPR, col = threadIdx.x % LPR * 8;
    if (i0 >= s.S) return;
    uint2 w[kQReadRows];
    float sc[kQReadRows];
#pragma unroll
    for (int n = 0; n < kQReadRows; ++n) {
        const int i = i0 + n * RPB, p = s.p0 + i;
        w[n] = make_uint2(0, 0);
        sc[n] = 0.f;
        if (i < s.S) {
            const int at = a.by_page.div(p), slot = p - at * a.page_size, page = qcache_page(a, b, at);
            if (page >= 0) {
                const size_t ph = (static_cast<size_t>(page) * 2 + kv) * a.nkv + h;
                w[n] = *reinterpret_cast<const uint2 *>(a.codes + (ph * a.page_size + slot) * D + col);
                sc[n] = a.scales[ph * a.blocks + a.by_block.div(slot)];
            }
        }
    }
    T *dst = (kv ? v : k) + s.r0 * (kv ? v_stride : k_stride) + h * D + col;
    const long long stride = kv ? v_stride : k_stride;
#pragma unroll
    for (int n = 0; n < kQReadRows; ++n) {
        const int i = i0 + n * RPB;
        if (i >= s.S) break;
        const uint32_t r[4] = {w[n].x & 0xffffu, w[n].x >> 16, w[n].y & 0xffffu, w[n].y >> 16};
        alignas(16) T y[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = e4m3x2_f32(r[j]);
            y[2 * j] = from_f32<T>(f.x * sc[n]);
            y[2 * j + 1] = from_f32<T>(f.y * sc[n]);
        }
        if constexpr (VEC) {
#pragma unroll
            for (int u = 0; u < static_cast<int>(sizeof(T)) / 2; ++u)
                reinterpret_cast<uint4 *>(dst + i * stride)[u] = reinterpret_cast<const uint4 *>(y)[u];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) dst[i * stride + j] = y[j];
        }
    }
}

}  // namespace sdv
