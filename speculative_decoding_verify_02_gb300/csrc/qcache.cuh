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
    __device__ __forceinline__ int mod(int n, int d) const { return n - div(n) * d; }
};

struct QCacheArgs {
    uint8_t *codes;   // the layer's [n_pages][2][nkv][page_size][D]
    float *scales;    // the layer's [n_pages][2][nkv][page_size / scale_block]
    int *status;
    const int *page_table, *row_off, *base;
    int pages_per_seq, page_size, n_pages, scale_block, nkv, B, max_span, max_rows, max_context;
    FastDiv by_page, by_block;  // page_size and scale_block
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

// Eight values of a row in registers, from a row that is 16-byte aligned or (VEC false) not.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T *src, float (&x)[8]) {
    if constexpr (VEC) {
        constexpr int W = sizeof(T) * 8 / 16;
        uint4 u[W];
#pragma unroll
        for (int w = 0; w < W; ++w) u[w] = __ldg(reinterpret_cast<const uint4 *>(src) + w);
        const T *t = reinterpret_cast<const T *>(u);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = to_f32(t[k]);
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = to_f32(src[k]);
    }
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

// A warp quantises one block: (sequence, block of its span, K or V, kv head). Lanes hold eight values
// each, 32 / (D / 8) rows at a time. A block that the span starts inside keeps its scale or a larger
// one, and its rows below the span are rounded again by the ratio of the two.
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kQWriteThreads) qcache_write_kernel(QCacheArgs a, const T *k, const T *v,
                                                                      long long k_stride, long long v_stride) {
    pdl_trigger();
    pdl_wait();
    constexpr int LPR = D / 8, RPI = 32 / LPR;
    const int item = blockIdx.x * (kQWriteThreads / 32) + threadIdx.x / 32;
    const int b = blockIdx.y, lane = threadIdx.x % 32;
    const int kv = item % (2 * a.nkv) / a.nkv, h = item % a.nkv;
    const QSpan s = qcache_span(a, b);
    if (s.S == 0) {
        if (s.code != SDV_OK && item == 0 && lane == 0) set_status(a.status, s.code);
        return;
    }
    const int tok0 = (s.p0 / a.scale_block + item / (2 * a.nkv)) * a.scale_block;
    if (tok0 >= s.p0 + s.S) return;
    const int lo = max(tok0, s.p0), hi = min(tok0 + a.scale_block, s.p0 + s.S);
    const int page = qcache_page(a, b, tok0 / a.page_size);
    if (page < 0) return;
    const size_t ph = (static_cast<size_t>(page) * 2 + kv) * a.nkv + h;
    uint8_t *dst = a.codes + (ph * a.page_size + tok0 % a.page_size) * D;  // the block's first slot
    float *scale = a.scales + ph * (a.page_size / a.scale_block) + tok0 % a.page_size / a.scale_block;
    const int col = lane % LPR * 8, sub = lane / LPR;
    const T *src = (kv ? v + (s.r0 - s.p0) * v_stride : k + (s.r0 - s.p0) * k_stride) + h * D + col;
    const long long stride = kv ? v_stride : k_stride;
    float amax = 0.f;
    bool bad = false;
    for (int t = lo + sub; t < hi; t += RPI) {
        float x[8];
        load8<T, VEC>(src + t * stride, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float m = fabsf(x[j]);
            if (m < INFINITY) amax = fmaxf(amax, m);
            else bad = true;
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (bad) set_status(a.status, SDV_ERR_DEVICE);
    float now = e4m3_scale(amax);
    if (lo > tok0) {
        float old = *scale;
        if (!(old > 0.f && old < INFINITY)) old = 0.f;  // never written: nothing below the span counts
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
    const float inv = 1.f / now;  // exact: a power of two from 2^-120 to 2^126
    for (int t = lo + sub; t < hi; t += RPI) {
        float x[8];
        load8<T, VEC>(src + t * stride, x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = x[j] == x[j] ? x[j] * inv : 0.f;
        *reinterpret_cast<uint2 *>(dst + (t - tok0) * D + col) =
            make_uint2(e4m3x2(x[0], x[1]) | e4m3x2(x[2], x[3]) << 16, e4m3x2(x[4], x[5]) | e4m3x2(x[6], x[7]) << 16);
    }
    __syncwarp();  // every lane has read the old scale
    if (lane == 0) *scale = now;
}

constexpr int kQReadThreads = 256;

// Eight codes a thread: code * scale (exact in fp32 but where it leaves fp32's range), rounded once.
// Grid (span rows in groups, sequences, K|V x heads).
template <typename T, int D, bool VEC>
__global__ void __launch_bounds__(kQReadThreads) qcache_read_kernel(QCacheArgs a, T *k, T *v, long long k_stride,
                                                                    long long v_stride) {
    pdl_trigger();
    pdl_wait();
    constexpr int LPR = D / 8, RPB = kQReadThreads / LPR;
    const int b = blockIdx.y, kv = blockIdx.z / a.nkv, h = blockIdx.z % a.nkv;
    const QSpan s = qcache_span(a, b);
    if (s.S == 0) {
        if (s.code != SDV_OK && blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) set_status(a.status, s.code);
        return;
    }
    const int i = blockIdx.x * RPB + threadIdx.x / LPR, col = threadIdx.x % LPR * 8;
    if (i >= s.S) return;
    const int p = s.p0 + i, page = qcache_page(a, b, p / a.page_size), slot = p % a.page_size;
    float x[8];
    if (page >= 0) {
        const size_t ph = (static_cast<size_t>(page) * 2 + kv) * a.nkv + h;
        const uint2 w = *reinterpret_cast<const uint2 *>(a.codes + (ph * a.page_size + slot) * D + col);
        const float sc = a.scales[ph * (a.page_size / a.scale_block) + slot / a.scale_block];
        const uint32_t r[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float2 f = e4m3x2_f32(r[j]);
            x[2 * j] = f.x * sc;
            x[2 * j + 1] = f.y * sc;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = 0.f;
    }
    T *dst = (kv ? v + (s.r0 + i) * v_stride : k + (s.r0 + i) * k_stride) + h * D + col;
    alignas(16) T y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = from_f32<T>(x[j]);
    if constexpr (VEC) {
#pragma unroll
        for (int w = 0; w < static_cast<int>(sizeof(T)) / 2; ++w)
            reinterpret_cast<uint4 *>(dst)[w] = reinterpret_cast<const uint4 *>(y)[w];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) dst[j] = y[j];
    }
}

}  // namespace sdv
