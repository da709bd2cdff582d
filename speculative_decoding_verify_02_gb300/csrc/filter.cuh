// Filtered sampling: a row's tokens cut to its top-k, top-p and min-p set, and a draw from it by given random numbers.
//
// Tokens are ordered by logit, equal ones by index: a 64-bit key each, and a kept set is the keys at or above one of them.
// With w = 2^-((m - x) log2(e) / T), m the row's largest logit, top-p keeps token i iff the weights before it sum to less than
// p of the top-k set's. The row stays in the shared memory of a cluster of CTAs. Each thread's largest logit is known from the
// search for the row's: k of those, or as many as weigh p of the total, are a bound that the border does not pass. (For k up to
// 256 the largest of each eight threads will do, which are few enough for every CTA to have them all: 8 rows 12.4 us, 12.8 by a
// histogram that the CTAs add up.) Where no
// more than kFilterList tokens lie above it, as in most rows of a language model, they go to one CTA, which sorts them and cuts
// and draws by itself. Where more do, a histogram of all tokens over (m - x) / T shows the border's bin, sums over the bin's
// edges confirm it, and its tokens alone are compared with one another.
//
// Whether a token is kept is decided as exact arithmetic would: sums of fp32 weights hold to 2^-17 of the total each
// (kFilterNear); a border nearer than that is decided on weights of 2^-37 (weight_exact), to 2^-36 of the total. Sums are
// integers, units of 2^-44, whose order does not matter; 64-bit floats stay out of the way of most rows: this part does them at
// 1/64 of fp32's rate, and the first kernel, which used them for sums and settings, took 75,000 clocks a row where it is 26,000 now.
#pragma once

#include <float.h>

#include "accept_sampled.cuh"

namespace sdv {

constexpr int kFilterThreads = 512;
constexpr int kFilterBins = 1024;
constexpr int kFilterFew = 256;                  // tokens that are compared with one another
constexpr float kFilterRange = 40.f;             // log2 of the weights that the histogram's bins cover
constexpr int kFilterCluster = 8;                // CTAs of a row
constexpr int kFilterGroups = kFilterCluster * kFilterThreads / 8;
constexpr int kFilterList = 2048;                // tokens that one CTA sorts; a row of no more is one CTA's
constexpr int kFilterMost = 49152;               // tokens of a CTA at most (192 KB)
// How far a sum of fp32 weights and p times another may lie from each other's exact values, over the total: an exponent
// t = (m - x) log2(e) / T takes three roundings, 2.1 t 2^-24 after ln 2, and t averages log2 of the vocabulary at most over the
// weights (19: 40 2^-24); ex2 is off by 4 2^-24, a thread's sum of up to 96 terms by 96 2^-24. 140 2^-24 each, 2^-15.9 both.
constexpr int kFilterNear = 15;  // 2^-15

// 2^(58 - j / 64)
__device__ const unsigned long long kFilterTable[64] = {
    0x400000000000000ull, 0x3f4f83033d21b06ull, 0x3ea0ecb6dc8a80dull, 0x3df437dcc2b44efull,
    0x3d495f454921b31ull, 0x3ca05dcf167fec5ull, 0x3bf92e66f736bd7ull, 0x3b53cc07b6650aeull,
    0x3ab031b9f7490e5ull, 0x3a0e5a940f12f72ull, 0x396e41b9df20d23ull, 0x38cfe25cafa2969ull,
    0x383337bb0aa5384ull, 0x37983d209783a45ull, 0x36feede5f6bc8ddull, 0x366745709e2bf5full,
    0x35d13f32b5a75acull, 0x353cd6aaf3fb7e8ull, 0x34aa07647c4ab91ull, 0x3418ccf6bbcac96ull,
    0x3389230547e1204ull, 0x32fb053fbc9c9f1ull, 0x326e6f619b8bc9full, 0x31e35d322aee6c5ull,
    0x3159ca845541b6bull, 0x30d1b3368925d90ull, 0x304b1332999c251ull, 0x2fc5e66d9e9cc42ull,
    0x2f4228e7d6030dbull, 0x2ebfd6ac84cf918ull, 0x2e3eebd1d8bee7cull, 0x2dbf6478ca345deull,
    0x2d413cccfe77992ull, 0x2cc47104aa44492ull, 0x2c48fd6074ab096ull, 0x2bcede2b5a4290eull,
    0x2b560fba90a852bull, 0x2ade8e6d6a4fb4dull, 0x2a6856ad3a9f03cull, 0x29f364ed3a594d6ull,
    0x297fb5aa6c544e4ull, 0x290d456b8279a02ull, 0x289c10c0c3125a0ull, 0x282c1443ee5c53full,
    0x27bd4c982468447ull, 0x274fb669cb3feddull, 0x26e34e6e7553955ull, 0x26781164c82dfeaull,
    0x260dfc14636e2a6ull, 0x25a50b4dc806168ull, 0x253d3bea3fbdc26ull, 0x24d68acbc4f9ba5ull,
    0x2470f4dceac470dull, 0x240c7710c519ac7ull, 0x23a90e62d17354full, 0x2346b7d6df96ea8ull,
    0x22e57078faa2f5cull, 0x2285355d525bbf6ull, 0x222603a024b6a15ull, 0x21c7d865a7a3440ull,
    0x216ab0d9f3121ecull, 0x210e8a30eb37901ull, 0x20b361a62b0ae87ull, 0x2059347cef00c1eull,
};

struct FilterArgs {
    int *status;
    const int *row_off;
    const float *logits, *temperature, *top_p, *min_p, *noise;
    const int *top_k;
    long long logits_stride, noise_stride, out_stride;  // floats between rows
    float *out;      // filter: the kept logits, -inf elsewhere
    int *tokens;     // sample: a token a row
    int *n_kept;     // or null
    int B, vocab, max_span, rows_cap, chunk;  // chunk: tokens of a CTA
};

__device__ __forceinline__ float filter_ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int BYTES>
__device__ __forceinline__ void filter_copy(float *dst, const float *src) {
    if constexpr (BYTES == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// ------------------------------------------------------------------ clusters
__device__ __forceinline__ unsigned long long ld_dsmem_u64(uint32_t addr) {
    unsigned long long v;
    asm volatile("ld.shared::cluster.u64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_dsmem_u32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_dsmem_u16(uint32_t addr) {
    unsigned short v;
    asm volatile("ld.shared::cluster.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void st_dsmem_u64(uint32_t addr, unsigned long long v) {
    asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t add_dsmem_u32(uint32_t addr, uint32_t v) {
    uint32_t old;
    asm volatile("atom.shared::cluster.add.u32 %0, [%1], %2;" : "=r"(old) : "r"(addr), "r"(v) : "memory");
    return old;
}

struct FilterSums {
    unsigned long long a, b;              // summed
    unsigned long long hi, lo;            // the largest, the smallest
};
struct FilterShared {
    uint32_t hist[kFilterBins], total[kFilterBins];  // of this CTA, of the row
    FilterSums warp[kFilterThreads / 32], part[2][kFilterCluster];
    unsigned long long list[kFilterList];            // CTA 0's: keys, or the border's tokens' keys and then their weights
    uint16_t pick[kFilterList];                      // tokens of this CTA for the list, places in its chunk
    float group[kFilterGroups];                      // of the row: the largest logit of each eight threads
    unsigned long long cut, scan_e[kFilterThreads / 32];
    unsigned long long target, table[64];     // table: kFilterTable's
    uint32_t n_cand, n_pick, scan[kFilterThreads / 32], warp_sum[kFilterThreads / 32], ambiguous, kept;
    float scan_w[kFilterThreads / 32], about, about_all;
    int found[3], seq, fails;
};

__device__ __forceinline__ unsigned long long filter_key(float x, int v) {  // -0 and 0 are equal
    return static_cast<unsigned long long>(orderable(x + 0.f)) << 32 | static_cast<uint32_t>(~v);
}

__device__ __forceinline__ float filter_value(uint32_t key) {
    return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// A row's constants.
struct FilterRow {
    float m, c_hi, c_lo, scale, T;  // the maximum, log2(e) / T in two parts, bins a logit
};
__device__ __forceinline__ float filter_weight(const FilterRow &r, float x) {
    if (x == r.m) return 1.f;
    const float t = (r.m - x) * r.c_hi;
    return t < 150.f ? filter_ex2(-t) : 0.f;
}
// v 2^-bits, rounded
__device__ __forceinline__ unsigned long long filter_round(unsigned long long v, int bits) {
    return bits ? (v >> bits) + (v >> (bits - 1) & 1) : v;
}
// The weight as an integer times 2^-58, to 2^-37: the exponent in two fp32 parts, 2^-n/64 from a table and the rest, below
// 2^-7, by the series of e^z in two parts.
__device__ __forceinline__ unsigned long long weight_exact(const FilterRow &r, float x, const unsigned long long *table) {
    if (x == r.m) return 1ull << 58;
    const float s = r.m - x, bb = s - r.m, e = (r.m - (s - bb)) - (x + bb);  // s + e = m - x
    const float p = s * r.c_hi;
    if (!(p < 60.f)) return 0;
    const float q = fmaf(s, r.c_hi, -p) + (s * r.c_lo + e * r.c_hi);         // p + q = (m - x) c
    const int n = __float2int_rn(p * 64.f);
    const float f = p - static_cast<float>(n) * 0.015625f;                   // exact
    constexpr float L = -0.693147182f, L_lo = 1.90465421e-9f;                // L + L_lo = -ln 2
    const float u = f * L, u_lo = fmaf(f, L, -u) + (f * L_lo + q * L);       // z = u + u_lo
    const float g0 = u * u * (0.5f + u * (0.16666667f + u * 0.041666668f));  // e^u - 1 = u + g0
    const float g = g0 + fmaf(u_lo, u + g0, u_lo);                           // e^z - 1 = u + g; u u_lo is up to 2^-26 (p near 25)
    const unsigned long long t58 = table[n & 63];
    const uint32_t t_hi = static_cast<uint32_t>(t58 >> 35), t_lo = static_cast<uint32_t>(t58 >> 3);  // 24 bits, 32 more
    const float tf = __uint2float_rn(t_hi) * 0x1p-23f, tl = __uint2float_rn(t_lo) * 0x1p-55f;
    const float a = tf * u, b = fmaf(tf, u, -a) + (tf * g + tl * u);         // t (e^z - 1)
    // as integers by 32-bit conversions, 64-bit ones being as slow as 64-bit floats: |a| < 2^-7, |b| < 2^-15
    const float a37 = a * 0x1p37f;
    const int a_hi = __float2int_rn(a37), a_lo = __float2int_rn((a37 - __int2float_rn(a_hi)) * 0x1p21f), b46 = __float2int_rn(b * 0x1p45f);
    const long long w = static_cast<long long>(t58) + (static_cast<long long>(a_hi) << 21) + a_lo + (static_cast<long long>(b46) << 13);
    return filter_round(static_cast<unsigned long long>(w), n >> 6);
}

// Which of the four a reduction takes along.
constexpr int kSumA = 1, kSumB = 2, kHi = 4, kLo = 8;
template <int F>
__device__ __forceinline__ void filter_join(FilterSums &s, const FilterSums &o) {
    if constexpr (F & kSumA) s.a += o.a;
    if constexpr (F & kSumB) s.b += o.b;
    if constexpr (F & kHi) s.hi = o.hi > s.hi ? o.hi : s.hi;
    if constexpr (F & kLo) s.lo = o.lo < s.lo ? o.lo : s.lo;
}
// Over the row, by every thread of every CTA, who all get the result. `shift`: the sums lose that many bits on the way, half once a
// warp's are added up and the rest once a CTA's are, which keeps theirs from overflowing.
template <int F>
__device__ __forceinline__ FilterSums filter_reduce(FilterShared &sh, FilterSums s, int ctas, int rank, int turn, int shift = 0) {
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    constexpr int W = kFilterThreads / 32;
    auto across = [&](int from) {
#pragma unroll
        for (int o = from; o > 0; o >>= 1) {
            FilterSums t{};
            if constexpr (F & kSumA) t.a = __shfl_xor_sync(0xffffffffu, s.a, o);
            if constexpr (F & kSumB) t.b = __shfl_xor_sync(0xffffffffu, s.b, o);
            if constexpr (F & kHi) t.hi = __shfl_xor_sync(0xffffffffu, s.hi, o);
            if constexpr (F & kLo) t.lo = __shfl_xor_sync(0xffffffffu, s.lo, o);
            filter_join<F>(s, t);
        }
    };
    across(16);
    const int late = shift / 2;
    s.a = filter_round(s.a, shift - late);
    s.b = filter_round(s.b, shift - late);
    if (lane == 0) sh.warp[warp] = s;
    __syncthreads();
    FilterSums (&part)[kFilterCluster] = sh.part[turn & 1];
    if (warp == 0) {  // this CTA's to every CTA
        s = sh.warp[lane % W];
        across(W / 2);
        s.a = filter_round(s.a, late);
        s.b = filter_round(s.b, late);
        if (lane < ctas) {
            const uint32_t to = mapa_shared(smem_u32(&part[rank]), lane);
            if constexpr (F & kSumA) st_dsmem_u64(to, s.a);
            if constexpr (F & kSumB) st_dsmem_u64(to + 8, s.b);
            if constexpr (F & kHi) st_dsmem_u64(to + 16, s.hi);
            if constexpr (F & kLo) st_dsmem_u64(to + 24, s.lo);
        }
    }
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    s = part[0];
    for (int r = 1; r < ctas; ++r) filter_join<F>(s, part[r]);
    return s;
}
__device__ __forceinline__ void filter_sync(int ctas) {
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
}

// CTA 0's list in order, the largest key first: key[u] of a thread is the list's tid + u threads, `top` the largest of all.
// Each goes to its bin between the largest logit and the list's smallest, and to its place among the bin's, which are a few;
// bins are even over the square of the distance, as logits crowd at the list's end.
// Where some bin holds more than kFilterFew (nearly all logits equal, or one far above the others) a bitonic network sorts.
// 890 of a row's tokens take 5,700 clocks, by the network 22,000: 55 passes through shared memory, a barrier behind each.
__device__ __forceinline__ void filter_sort(FilterShared &sh, const unsigned long long *key, int n, unsigned long long top) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    constexpr int PER = kFilterList / kFilterThreads;
    for (int i = tid; i < kFilterBins; i += kFilterThreads) sh.hist[i] = 0;
    uint32_t least = 0xffffffffu;
#pragma unroll
    for (int u = 0; u < PER; ++u)
        if (tid + u * kFilterThreads < n) least = min(least, static_cast<uint32_t>(key[u] >> 32));
    least = __reduce_min_sync(0xffffffffu, least);
    if (lane == 0) sh.scan[warp] = least;
    __syncthreads();
    for (int i = 0; i < kFilterThreads / 32; ++i) least = min(least, sh.scan[i]);
    const float m = filter_value(static_cast<uint32_t>(top >> 32)), range = m - filter_value(least);
    const float scale = 1.f / range;  // no number where range is infinite or zero: bin 0
    int bin[PER], at[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        if (tid + u * kFilterThreads >= n) continue;
        const float t = (m - filter_value(static_cast<uint32_t>(key[u] >> 32))) * scale;  // monotone, rounded or not
        bin[u] = t > 0.f ? static_cast<int>(fminf(kFilterBins * (t * t), kFilterBins - 1.f)) : 0;
        at[u] = static_cast<int>(atomicAdd(&sh.hist[bin[u]], 1u));
    }
    __syncthreads();
    const uint32_t n0 = sh.hist[2 * tid], n1 = sh.hist[2 * tid + 1];
    uint32_t sum = n0 + n1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
    }
    if (lane == 31) sh.warp_sum[warp] = sum;
    const bool network = __syncthreads_or(max(n0, n1) > kFilterFew);
    for (int i = 0; i < warp; ++i) sum += sh.warp_sum[i];
    sh.total[2 * tid] = sum - n1 - n0;
    sh.total[2 * tid + 1] = sum - n1;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u)
        if (tid + u * kFilterThreads < n) sh.list[sh.total[bin[u]] + at[u]] = key[u];
    if (network) {
        int size = 32;
        while (size < n) size *= 2;
        for (int i = n + tid; i < size; i += kFilterThreads) sh.list[i] = 0;
        __syncthreads();
        for (int k = 2; k <= size; k *= 2)
            for (int j = k / 2; j > 0; j /= 2) {
                for (int i = tid; i < size / 2; i += kFilterThreads) {
                    const int p = 2 * i - (i & (j - 1)), q = p + j;
                    const unsigned long long u = sh.list[p], v = sh.list[q];
                    if ((u < v) == ((p & k) == 0)) sh.list[p] = v, sh.list[q] = u;
                }
                __syncthreads();
            }
        return;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u) {
        if (tid + u * kFilterThreads >= n) continue;
        const int first = static_cast<int>(sh.total[bin[u]]), end = first + static_cast<int>(sh.hist[bin[u]]);
        at[u] = first;
#pragma unroll 8
        for (int i = first; i < end; ++i) at[u] += sh.list[i] > key[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < PER; ++u)
        if (tid + u * kFilterThreads < n) sh.list[at[u]] = key[u];
    __syncthreads();
}

// What a search looks for: the last token with fewer than `k` before it and, if by_mass, less than `target` of weight before it.
struct FilterGoal {
    bool by_mass;
    int k;
    float p;
    unsigned long long target, total;  // target = p total, rounded up: a sum is below it iff it is below p total
    float off;                         // what the histogram takes the total for less what it is
    unsigned long long set;            // the mass's tokens: keys at or above it
};
constexpr float kFilterUnit = 0x1p-44f;
// p v for 0 < p < 1, rounded up
__device__ __forceinline__ unsigned long long filter_share(float p, unsigned long long v) {
    const uint32_t u = __float_as_uint(p), e = u >> 23;
    const unsigned long long m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
    const int s = 150 - static_cast<int>(e ? e : 1);  // p = m 2^-s, 24 <= s
    const unsigned long long hi = __umul64hi(v, m), lo = v * m;
    if (s >= 64) return s - 64 >= 64 ? (hi | lo) != 0 : (hi >> (s - 64)) + (((hi & ((1ull << (s - 64)) - 1)) | lo) != 0);
    return (hi << (64 - s) | lo >> s) + ((lo & ((1ull << s) - 1)) != 0);
}

template <bool SAMPLE>
__global__ void __launch_bounds__(kFilterThreads, 2) filter_kernel(const __grid_constant__ FilterArgs a) {
    extern __shared__ __align__(16) float x_s[];
    __shared__ FilterShared sh;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32, row = blockIdx.y, ctas = gridDim.x, rank = blockIdx.x;
    const int v0 = rank * a.chunk, n = max(0, min(a.chunk, a.vocab - v0)), n4 = (n + 3) / 4;
    if (ctas > 1) cluster_arrive();  // others' shared memory is there once they have started
    if (tid < 64) sh.table[tid] = kFilterTable[tid];
    if (tid == 0) sh.seq = -1, sh.n_cand = sh.n_pick = 0;
    pdl_wait();
    pdl_trigger();
    // the row's logits are asked for before its sequence is known; four at a time in every pass, -inf behind the last
    const float *src = a.logits + row * a.logits_stride + v0;
    if ((reinterpret_cast<uintptr_t>(src) & 15) == 0) {
        for (int i = tid * 4; i + 3 < n; i += kFilterThreads * 4) filter_copy<16>(x_s + i, src + i);
        for (int i = (n & ~3) + tid; i < n; i += kFilterThreads) filter_copy<4>(x_s + i, src + i);
    } else {
        for (int i = tid; i < n; i += kFilterThreads) filter_copy<4>(x_s + i, src + i);
    }
    if (tid < 4 && n + tid < 4 * n4) x_s[n + tid] = -INFINITY;
    __syncthreads();
    if (tid < a.B) {  // B <= 256 threads
        const int r0 = a.row_off[tid], S = a.row_off[tid + 1] - r0;
        const bool ok = S > 0 && S <= a.max_span && r0 >= 0 && r0 <= a.rows_cap - S;
        if (ok && row >= r0 && row < r0 + S) sh.seq = tid;
        if (!ok && S != 0 && row == 0 && rank == 0) set_status(a.status, SDV_ERR_ARG);
    }
    for (int i = tid; i < kFilterBins; i += kFilterThreads) sh.hist[i] = sh.total[i] = 0;
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();
    const int b = sh.seq;
    if (ctas > 1) cluster_wait();
    if (b < 0) return;  // a row of no span: every CTA of the cluster leaves
    const float T = a.temperature[b];
    const float top_p = a.top_p ? a.top_p[b] : 2.f, min_p = a.min_p ? a.min_p[b] : 0.f;
    const int top_k = a.top_k ? a.top_k[b] : 0;
    const bool by_groups = ctas == kFilterCluster && top_k > 0 && top_k <= min(kFilterThreads, a.chunk / 4) / 16 * kFilterCluster;
    int turn = 0;
    const unsigned long long none = ~0ull;
    float4 *x4 = reinterpret_cast<float4 *>(x_s);
    auto each = [&](auto f) {  // f(logit, place in the chunk) of this thread's tokens above -inf
        for (int i = tid; i < n4; i += kFilterThreads) {
            const float4 x = x4[i];
            if (x.x > -INFINITY) f(x.x, 4 * i);
            if (x.y > -INFINITY) f(x.y, 4 * i + 1);
            if (x.z > -INFINITY) f(x.z, 4 * i + 2);
            if (x.w > -INFINITY) f(x.w, 4 * i + 3);
        }
    };
    // ---- the maximum, and the tokens above -inf
    FilterRow r;
    int valid;
    unsigned long long top;  // the first token
    float m = -INFINITY;     // this thread's largest
    {
        int count = 0, first = 0;
        for (int i = tid; i < n4; i += kFilterThreads) {
            float4 x = x4[i];
            const bool ok = x.x > -INFINITY && x.y > -INFINITY && x.z > -INFINITY && x.w > -INFINITY;
            if (!ok) {  // NaN counts as -inf
                x.x = x.x > -INFINITY ? x.x : -INFINITY, x.y = x.y > -INFINITY ? x.y : -INFINITY;
                x.z = x.z > -INFINITY ? x.z : -INFINITY, x.w = x.w > -INFINITY ? x.w : -INFINITY;
                x4[i] = x;
                count -= (x.x == -INFINITY) + (x.y == -INFINITY) + (x.z == -INFINITY) + (x.w == -INFINITY);
            }
            count += 4;
            const float four = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w));
            if (four > m) {  // a thread's indexes ascend
                m = four;
                first = v0 + 4 * i + (x.x == m ? 0 : x.y == m ? 1 : x.z == m ? 2 : 3);
            }
        }
        if (by_groups) {  // the largest of each eight threads, for every CTA
            float most = m;
#pragma unroll
            for (int o = 1; o < 8; o *= 2) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, o));
            st_dsmem_u32(mapa_shared(smem_u32(&sh.group[(rank * (kFilterThreads / 32) + warp) * 4 + lane / 8]), lane % 8), __float_as_uint(most));
        }
        FilterSums s = {static_cast<unsigned long long>(count), 0, count ? filter_key(m, first) : 0ull, none};
        s = filter_reduce<kSumA | kHi>(sh, s, ctas, rank, turn++);
        valid = static_cast<int>(s.a);
        top = s.hi;
        r.m = filter_value(static_cast<uint32_t>(s.hi >> 32));
    }
    unsigned long long cut = 0;  // the kept set: keys at or above it
    int kept = valid;
    float *out = SAMPLE ? nullptr : a.out + row * a.out_stride + v0;
    const bool vec = !SAMPLE && (reinterpret_cast<uintptr_t>(out) & 15) == 0;
    auto fill = [&](float *to, int n) {
        const float4 nil = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY);
        if (vec) {
            for (int i = tid; i < n / 4; i += kFilterThreads) reinterpret_cast<float4 *>(to)[i] = nil;
            if (tid < n % 4) to[(n & ~3) + tid] = -INFINITY;
        } else {
            for (int i = tid; i < n; i += kFilterThreads) to[i] = -INFINITY;
        }
    };
    if (valid == 0) {  // nothing to keep
        if constexpr (!SAMPLE) fill(out, n);
        if (rank == 0 && tid == 0) {
            if (SAMPLE) a.tokens[row] = 0;
            if (a.n_kept) a.n_kept[row] = 0;
            set_status(a.status, SDV_ERR_DEVICE);
        }
        if (ctas > 1) cluster_sync();
        return;
    }
    r.T = T;
    {  // the quotient and its remainder's
        constexpr float L = 1.44269502f, L_lo = 1.92596303e-8f;  // L + L_lo = log2(e)
        r.c_hi = L / T;
        r.c_lo = (fmaf(-r.c_hi, T, L) + L_lo) / T;
    }
    r.scale = r.c_hi * (kFilterBins / kFilterRange);
    if (!(T > 0.f) || min_p > 1.f || top_p <= 0.f || valid == 1) cut = top, kept = 1;  // the first token alone
    const bool want_k = kept > 1 && top_k > 0 && top_k < valid, want_p = kept > 1 && top_p > 0.f && top_p < 1.f;
    const bool want_m = kept > 1 && min_p > 0.f;
    // w >= min_p: exponents are compared, (m - x) log2(e) / T with -log2(min_p), and in 64 bits where fp32 could not tell
    const float weakest = want_m ? -log2f(min_p) : INFINITY;
    auto strong = [&](float x) {
        if (!want_m || x == r.m) return true;
        const float t = (r.m - x) * r.c_hi, near = (fabsf(t) + weakest + 1.f) * 0x1p-20f;
        if (!(fabsf(t - weakest) <= near)) return t < weakest;
        return static_cast<double>(x) - static_cast<double>(r.m) >= static_cast<double>(T) * log(static_cast<double>(min_p));
    };
    auto place_of = [&](float x) { return x == r.m ? 0.f : (r.m - x) * r.scale; };  // on the line of bins
    auto bin_of = [&](float x) {
        const float t = place_of(x);
        return t < kFilterBins - 1 ? static_cast<int>(t) : kFilterBins - 1;
    };
    auto middle_weight = [](int i) { return filter_ex2(-(i + .5f) * (kFilterRange / kFilterBins)); };
    bool precise = false, listed = false;  // listed: the kept tokens are CTA 0's first ones, in order

    if (want_k || want_p) {
        // this CTA's histogram -> the row's, in every CTA
        auto add_up = [&]() {
            filter_sync(ctas);
            const int share = kFilterBins / ctas;
            for (int i = tid; i < share; i += kFilterThreads) {
                const int bin = rank * share + i;
                uint32_t part[kFilterCluster], sum = 0;
#pragma unroll
                for (int q = 0; q < kFilterCluster; ++q) part[q] = q < ctas ? ld_dsmem_u32(mapa_shared(smem_u32(&sh.hist[bin]), q)) : 0;
#pragma unroll
                for (int q = 0; q < kFilterCluster; ++q) sum += part[q];
                for (int q = 0; q < ctas; ++q) st_dsmem_u32(mapa_shared(smem_u32(&sh.total[bin]), q), sum);
            }
            filter_sync(ctas);
        };
        // The first bin in [first, last] at which the tokens so far reach `k`, or about `mass` of weight (bin i's tokens weigh
        // about weight(i) each; mass < 0: all but -mass), else the last: found[0]; tokens before it: found[1], in it: found[2],
        // weight before it: about, of all: about_all.
        auto find_bin = [&](bool by_mass, int k, float mass, int first, int last, auto weight) {
            const uint32_t n0 = sh.total[2 * tid], n1 = sh.total[2 * tid + 1];
            __syncthreads();
            if (tid == 0) sh.found[0] = last;
            uint32_t count = n0 + n1;
            const float w0 = by_mass ? n0 * weight(2 * tid) : 0.f, w1 = by_mass ? n1 * weight(2 * tid + 1) : 0.f;
            float w = w0 + w1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t c2 = __shfl_up_sync(0xffffffffu, count, o);
                const float w2 = __shfl_up_sync(0xffffffffu, w, o);
                if (lane >= o) count += c2, w += w2;
            }
            if (lane == 31) sh.scan[warp] = count, sh.scan_w[warp] = w;
            __syncthreads();
            float w_all = 0.f;
#pragma unroll
            for (int i = 0; i < kFilterThreads / 32; ++i) {
                w_all += sh.scan_w[i];
                if (i < warp) count += sh.scan[i], w += sh.scan_w[i];
            }
            if (mass < 0.f) mass += w_all;
            const uint32_t c0 = count - n1;
            auto reaches = [&](uint32_t cnt, float ms) { return by_mass ? ms >= mass : cnt >= static_cast<uint32_t>(k); };
            const int here = reaches(c0, w - w1) ? 2 * tid : reaches(count, w) ? 2 * tid + 1 : kFilterBins;
            if (here < kFilterBins) atomicMin(&sh.found[0], max(here, first));
            __syncthreads();
            const int j = sh.found[0];
            if (j / 2 == tid) {
                sh.found[1] = static_cast<int>(j & 1 ? c0 : c0 - n0);
                sh.found[2] = static_cast<int>(j & 1 ? n1 : n0);
                sh.about = w - w1 - (j & 1 ? 0.f : w0), sh.about_all = w_all;
            }
            __syncthreads();
        };
        // Exact sums: a token's weight is rounded to 2^-57, a thread's sum to 2^-51, a warp's to 2^-47 and a CTA's to 2^-44. That is
        // off by 2^-38.5 at most, of 2^18.6 tokens; by tokens cut at 2^-51, all the same way where they are equal, it would be 2^-33.
        // Weight of the tokens for which in0 and in1 hold, and the keys for which in1 holds but not in0: smallest and largest.
        auto sums = [&](auto in0, auto in1) {
            FilterSums s = {0, 0, 0ull, none};
            float f0 = 0.f, f1 = 0.f;
            unsigned long long e0 = 0, e1 = 0;
            each([&](float x, int i) {
                if (!in1(x, i)) return;
                const bool both = in0(x, i);
                if (precise) {
                    const unsigned long long w = filter_round(weight_exact(r, x, sh.table), 1);  // a thread adds up to 96
                    e1 += w;
                    if (both) e0 += w;
                } else {
                    const float w = filter_weight(r, x);
                    f1 += w;
                    if (both) f0 += w;
                }
                if (!both) {
                    const unsigned long long k = filter_key(x, v0 + i);
                    s.hi = k > s.hi ? k : s.hi;
                    s.lo = k < s.lo ? k : s.lo;
                }
            });
            s.a = precise ? filter_round(e0, 6) : __float2ull_rn(f0 * 0x1p51f);
            s.b = precise ? filter_round(e1, 6) : __float2ull_rn(f1 * 0x1p51f);
            return filter_reduce<kSumA | kSumB | kHi | kLo>(sh, s, ctas, rank, turn++, 7);
        };
        auto set_total = [&](FilterGoal &g) {
            g.total = sums([&](float, int) { return true; }, [&](float x, int i) { return filter_key(x, v0 + i) >= g.set; }).a;
            g.target = filter_share(g.p, g.total);
        };
        auto close = [&](unsigned long long sum, const FilterGoal &g) {
            return (sum > g.target ? sum - g.target : g.target - sum) <= g.total >> kFilterNear;
        };
        // The key of the goal's last token; kept: tokens down to it.
        auto search = [&](FilterGoal g, int &kept_out) -> unsigned long long {
            // ---- a bin of the histogram over (m - x) / T: by weight a guess, confirmed by the sums over its edges or made
            // again from how far the sum before it is from the guess's
            int first = 0, last = kFilterBins - 1, above, count;
            unsigned long long A = 0;
            float guess = g.target * kFilterUnit + g.off;
            unsigned long long hi = 0, lo = none;
            for (int tries = 0;; ++tries) {
                const int half = (first + last) / 2;  // guesses that do not settle
                find_bin(g.by_mass, g.k, guess, tries < 4 ? first : half, tries < 4 ? last : half, middle_weight);
                const int j = sh.found[0];
                above = sh.found[1], count = sh.found[2];
                const float about = sh.about;
                for (;;) {
                    const FilterSums s = sums([&](float x, int) { return bin_of(x) < j; }, [&](float x, int) { return bin_of(x) <= j; });
                    A = s.a, hi = s.hi, lo = s.lo;
                    if (g.by_mass && !precise && (close(A, g) || close(s.b, g))) {
                        precise = true;
                        set_total(g);
                        continue;
                    }
                    if (g.by_mass && A >= g.target)
                        last = j - 1;
                    else if (g.by_mass && s.b < g.target)
                        first = j + 1;
                    else
                        last = -1;
                    break;
                }
                if (first > last) break;
                guess = fmaxf(0.f, static_cast<float>(static_cast<long long>(g.target - A)) * kFilterUnit + about);
            }
            // ---- while there are many tokens, a bin of the histogram over their keys' logits
            while (count > kFilterFew) {
                const uint32_t k_hi = static_cast<uint32_t>(hi >> 32), k_lo = static_cast<uint32_t>(lo >> 32);
                if (k_hi == k_lo) break;
                int shift = 0;
                while ((k_hi - k_lo) >> shift >= kFilterBins) ++shift;
                __syncthreads();
                for (int i = tid; i < kFilterBins; i += kFilterThreads) sh.hist[i] = 0;
                __syncthreads();
                each([&](float x, int) {
                    const uint32_t k = orderable(x + 0.f);
                    if (k <= k_hi && k >= k_lo) atomicAdd(&sh.hist[(k_hi - k) >> shift], 1u);
                });
                add_up();
                find_bin(g.by_mass, g.k - above, static_cast<float>(static_cast<long long>(g.target - A)) * kFilterUnit, 0, kFilterBins - 1,
                         [&](int i) { return filter_weight(r, filter_value(k_hi - (static_cast<uint32_t>(i) << shift))); });
                const int bin = sh.found[0], before = sh.found[1], inside = sh.found[2];
                const uint32_t h = k_hi - (static_cast<uint32_t>(bin) << shift), width = 1u << shift;
                const uint32_t l = h - k_lo >= width ? h - width + 1 : k_lo;
                FilterSums s;
                bool anew = false;  // once sums are exact, what lies before these tokens is summed up again, too
                for (;;) {
                    const unsigned long long over = anew ? hi : static_cast<unsigned long long>(h) << 32 | 0xffffffffu;
                    s = sums([&](float x, int i) { return filter_key(x, v0 + i) > over; }, [&](float x, int) { return orderable(x + 0.f) >= l; });
                    if (anew) {
                        anew = false;
                        A = s.a;
                    } else if (g.by_mass && !precise && (close(s.a, g) || close(s.b, g))) {
                        precise = anew = true;
                        set_total(g);
                    } else {
                        break;
                    }
                }
                if (g.by_mass && s.a >= g.target && before > 0) {  // above this bin
                    lo = static_cast<unsigned long long>(h + 1) << 32;
                    count = before;
                } else if (g.by_mass && s.b < g.target && before + inside < count) {  // below it
                    hi = static_cast<unsigned long long>(l - 1) << 32 | 0xffffffffu;
                    above += before + inside;
                    count -= before + inside;
                    A = s.b;
                } else {
                    hi = s.hi, lo = s.lo;
                    above += before;
                    count = inside;
                    A = s.a;
                }
            }
            if (count > kFilterFew) {
                // ---- many equal logits: the first of them by index
                const uint32_t k = static_cast<uint32_t>(hi >> 32);
                const float x = filter_value(k);
                int want = min(count, g.k - above);
                if (g.by_mass) {
                    if (!precise) {
                        precise = true;
                        set_total(g);
                        A = sums([&](float y, int) { return orderable(y + 0.f) > k; }, [&](float y, int) { return orderable(y + 0.f) > k; }).a;
                    }
                    // the first of them with weight enough before it: 2^-58 is 2^-14 of the sums' unit
                    const unsigned long long w = weight_exact(r, x, sh.table), lack = g.target > A ? g.target - A : 0;
                    const double need = ceil(static_cast<double>(lack) * 0x1p14 / static_cast<double>(w));
                    if (w > 0 && need < want) want = max(1, static_cast<int>(need));
                }
                // tokens in order: CTAs, then threads, a run of the chunk each
                const int run = (n + kFilterThreads - 1) / kFilterThreads, i0 = min(n, tid * run), i1 = min(n, i0 + run);
                int mine = 0;
                for (int i = i0; i < i1; ++i) mine += x_s[i] == x;
                int sum = mine;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int v = __shfl_up_sync(0xffffffffu, sum, o);
                    if (lane >= o) sum += v;
                }
                __syncthreads();
                if (lane == 31) sh.scan[warp] = sum;
                __syncthreads();
                int before = sum - mine, all = 0;
                for (int i = 0; i < kFilterThreads / 32; ++i) {
                    if (i < warp) before += sh.scan[i];
                    all += sh.scan[i];
                }
                if (tid == 0) sh.kept = all;
                filter_sync(ctas);
                for (int q = 0; q < rank; ++q) before += ld_dsmem_u32(mapa_shared(smem_u32(&sh.kept), q));
                filter_sync(ctas);
                if (before < want && before + mine >= want) {
                    int i = i0, seen = before;
                    for (; i < i1; ++i)
                        if (x_s[i] == x && ++seen == want) break;
                    for (int q = 0; q < ctas; ++q) st_dsmem_u64(mapa_shared(smem_u32(&sh.cut), q), filter_key(x, v0 + i));
                }
                filter_sync(ctas);
                kept_out = above + want;
                const unsigned long long found = sh.cut;
                __syncthreads();
                return found;
            }
            // ---- the border's tokens, to the first CTA
            const uint32_t counter = mapa_shared(smem_u32(&sh.n_cand), 0);
            each([&](float x, int i) {
                const unsigned long long k = filter_key(x, v0 + i);
                if (k <= hi && k >= lo) {
                    const uint32_t at = add_dsmem_u32(counter, 1);
                    if (at < kFilterFew) {
                        st_dsmem_u64(mapa_shared(smem_u32(&sh.list[at]), 0), k);
                        st_dsmem_u64(mapa_shared(smem_u32(&sh.list[kFilterFew + at]), 0), g.by_mass ? weight_exact(r, x, sh.table) >> 8 : 0ull);
                    }
                }
            });
            filter_sync(ctas);
            for (;;) {
                if (rank == 0) {
                    const int m = min(static_cast<int>(sh.n_cand), kFilterFew);
                    if (tid == 0) sh.ambiguous = 0, sh.kept = 0;
                    __syncthreads();
                    if (tid < m) {
                        const unsigned long long mine = sh.list[tid];
                        unsigned long long before = 0;
                        int place = above;
                        for (int q = 0; q < m; ++q) {
                            const bool earlier = sh.list[q] > mine;
                            before += earlier ? sh.list[kFilterFew + q] : 0ull;
                            place += earlier;
                        }
                        bool keep = place < g.k;
                        if (g.by_mass) {
                            const unsigned long long mass = A + (before >> 6);
                            if (!precise && close(mass, g)) sh.ambiguous = 1;
                            keep = keep && mass < g.target;
                        }
                        if (keep || place == 0) atomicMax(&sh.kept, static_cast<uint32_t>(place + 1));
                    }
                    __syncthreads();
                    const int last = max(static_cast<int>(sh.kept), above + 1);  // at least the first of them
                    if (tid < m) {
                        int place = above;
                        const unsigned long long mine = sh.list[tid];
                        for (int q = 0; q < m; ++q) place += sh.list[q] > mine;
                        if (place + 1 == last) {
                            for (int q = 0; q < ctas; ++q) {
                                st_dsmem_u64(mapa_shared(smem_u32(&sh.cut), q), mine);
                                st_dsmem_u32(mapa_shared(smem_u32(&sh.kept), q), last);
                                st_dsmem_u32(mapa_shared(smem_u32(&sh.ambiguous), q), sh.ambiguous);
                            }
                        }
                    }
                }
                filter_sync(ctas);
                const bool again = g.by_mass && !precise && sh.ambiguous;
                const unsigned long long found = sh.cut;
                kept_out = static_cast<int>(sh.kept);
                filter_sync(ctas);
                if (!again) {
                    if (rank == 0 && tid == 0) sh.n_cand = 0;
                    return found;
                }
                precise = true;
                set_total(g);
                A = sums([&](float x, int i) { return filter_key(x, v0 + i) > hi; }, [&](float x, int i) { return filter_key(x, v0 + i) > hi; }).a;
            }
        };

        // all tokens' histogram and the total; the last bin's tokens are those that the others leave
        auto count_bins = [&]() {
            float f = 0.f;
            __syncthreads();
            for (int i = tid; i < kFilterBins; i += kFilterThreads) sh.hist[i] = 0;
            __syncthreads();
            each([&](float x, int) {
                const float t = place_of(x);
                if (t < kFilterBins - 1) atomicAdd(&sh.hist[static_cast<int>(t)], 1u);
            });
            add_up();
            const int others = static_cast<int>(sh.total[2 * tid] + (tid == kFilterThreads - 1 ? 0 : sh.total[2 * tid + 1]));
            const int sum = __reduce_add_sync(0xffffffffu, others);
            if (lane == 0) sh.scan[warp] = sum;
            __syncthreads();
            int all = 0;
            for (int w = 0; w < kFilterThreads / 32; ++w) all += sh.scan[w];
            if (tid == 0) sh.total[kFilterBins - 1] = valid - all;
            __syncthreads();
            float off = 0.f;
            for (int i = 0; i < 2; ++i) off += sh.total[2 * tid + i] * middle_weight(2 * tid + i);
            off = warp_sum(off);
            if (lane == 0) sh.scan_w[warp] = off;
            __syncthreads();
            for (int w = 0; w < kFilterThreads / 32; ++w) f += sh.scan_w[w];
            return f;
        };
        FilterGoal g = {false, want_k ? top_k : valid, top_p, 0, 0, 0.f, 0ull};
        auto sum_up = [&]() {
            float f = 0.f;
            each([&](float x, int) { f += filter_weight(r, x); });
            FilterSums s = {__float2ull_rn(f * 0x1p51f), 0, 0ull, none};
            g.total = filter_reduce<kSumA>(sh, s, ctas, rank, turn++, 7).a;
            g.target = filter_share(g.p, g.total);
        };
        // ---- few tokens: those above the bound that the threads' largest give. Of weight, a bin's tokens count as its
        // lightest would, and the total's error as missing.
        const bool all = valid <= kFilterList;
        if (!want_k) sum_up();
        if (!all) {
            for (bool groups = by_groups && want_k;; groups = false) {  // few groups with a token: the threads' after all
                if (groups) {  // few enough for every CTA to count by itself
                    const float most = sh.group[tid];
                    if (most > -INFINITY) atomicAdd(&sh.total[bin_of(most)], 1u);
                    __syncthreads();
                } else {
                    if (m > -INFINITY) atomicAdd(&sh.hist[bin_of(m)], 1u);
                    add_up();
                }
                find_bin(!want_k, g.k, g.target * (kFilterUnit * 1.0001f), 0, kFilterBins - 1, [](int i) { return i < kFilterBins - 1 ? filter_ex2(-(i + 1) * (kFilterRange / kFilterBins)) : 0.f; });
                if (!groups || sh.found[0] < kFilterBins - 1) break;
            }
        }
        const int last = all ? 0 : sh.found[0];
        if (last < kFilterBins - 1) {
            // the bins' end as a logit, a little below: a few tokens more do no harm
            const float width = (last + 1) / r.scale, least = all ? -FLT_MAX : r.m - (width + (fabsf(r.m) + width) * 0x1p-20f);
            auto pick = [&](float x, int i) {
                if (!(x >= least) || x == -INFINITY) return;
                const uint32_t at = atomicAdd(&sh.n_pick, 1u);
                if (at < kFilterList) sh.pick[at] = static_cast<uint16_t>(i);
            };
#pragma unroll 4
            for (int i = tid; i < n4; i += kFilterThreads) {
                const float4 x = x4[i];
                if (fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)) >= least) pick(x.x, 4 * i), pick(x.y, 4 * i + 1), pick(x.z, 4 * i + 2), pick(x.w, 4 * i + 3);
            }
            filter_sync(ctas);
            int in_list = 0;
            unsigned long long key[kFilterList / kFilterThreads];
            if (rank == 0) {  // fetches everybody's
                int from[kFilterCluster + 1];
                from[0] = 0;
#pragma unroll
                for (int q = 0; q < kFilterCluster; ++q)
                    from[q + 1] = from[q] + (q < ctas ? static_cast<int>(ld_dsmem_u32(mapa_shared(smem_u32(&sh.n_pick), q))) : 0);
                in_list = from[kFilterCluster];
#pragma unroll
                for (int u = 0; u < kFilterList / kFilterThreads; ++u) {
                    const int i = tid + u * kFilterThreads;
                    key[u] = 0;
                    if (i >= in_list || in_list > kFilterList) continue;
                    int q = 0, first = 0;
#pragma unroll
                    for (int w = 1; w < kFilterCluster; ++w)
                        if (i >= from[w]) q = w, first = from[w];
                    const uint32_t at = ld_dsmem_u16(mapa_shared(smem_u32(&sh.pick[i - first]), q));
                    const float x = __uint_as_float(ld_dsmem_u32(mapa_shared(smem_u32(x_s + at), q)));
                    key[u] = filter_key(x, q * a.chunk + static_cast<int>(at));
                }
            }
            // what is kept will be few: -inf everywhere, by the others while CTA 0 decides
            if constexpr (!SAMPLE) {
                if (ctas == 1) fill(out, n);
                if (rank > 0) {
                    fill(out, n);
                    const int part = (a.chunk / 4 + ctas - 2) / (ctas - 1) * 4, first = (rank - 1) * part;  // of CTA 0's whole chunk
                    fill(out - v0 + first, max(0, min(part, a.chunk - first)));
                }
            }
            const bool fits = in_list > 0 && in_list <= kFilterList;
            if (rank == 0 && fits) filter_sort(sh, key, in_list, top);
            for (;;) {
                if (rank == 0 && !fits) {
                    if (tid < ctas) st_dsmem_u32(mapa_shared(smem_u32(&sh.ambiguous), tid), 2);
                } else if (rank == 0) {
                    // weights before each token, in order: exact
                    constexpr int PER = kFilterList / kFilterThreads;
                    const int per = (in_list + kFilterThreads - 1) / kFilterThreads;
                    unsigned long long w[PER], sum = 0;
#pragma unroll
                    for (int u = 0; u < PER; ++u) {
                        const int i = tid * per + u;
                        w[u] = want_p && u < per && i < in_list ? weight_exact(r, filter_value(static_cast<uint32_t>(sh.list[i] >> 32)), sh.table) >> 7 : 0ull;
                        sum += w[u];
                    }
                    unsigned long long before = sum;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const unsigned long long v = __shfl_up_sync(0xffffffffu, before, o);
                        if (lane >= o) before += v;
                    }
                    if (lane == 31) sh.scan_e[warp] = before;
                    if (tid == 0) sh.fails = in_list, sh.ambiguous = 0, sh.target = g.target;
                    __syncthreads();
                    before -= sum;
                    for (int i = 0; i < warp; ++i) before += sh.scan_e[i];
                    if (want_k) {  // the top-k set's weight
                        unsigned long long upto = before;
#pragma unroll
                        for (int u = 0; u < PER; ++u) {
                            upto += w[u];
                            if (want_p && u < per && tid * per + u == g.k - 1) sh.target = filter_share(g.p, upto >> 7);
                        }
                        __syncthreads();
                    }
                    const unsigned long long target = sh.target;
                    int fails = in_list;  // this thread's first token that is not kept
#pragma unroll
                    for (int u = 0; u < PER; ++u) {
                        const int i = tid * per + u;
                        if (u < per && i < in_list) {
                            const unsigned long long mass = before >> 7;
                            if (want_p && !want_k && !precise && close(mass, g)) sh.ambiguous = 1;
                            if (i >= g.k || (want_p && !(mass < target)) || !strong(filter_value(static_cast<uint32_t>(sh.list[i] >> 32))))
                                fails = min(fails, max(i, 1));
                            before += w[u];
                        }
                    }
                    fails = __reduce_min_sync(0xffffffffu, fails);
                    if (lane == 0 && fails < in_list) atomicMin(&sh.fails, fails);
                    __syncthreads();
                    // the list ends before the border: the search below
                    if (tid == 0 && sh.fails == in_list && in_list < min(valid, g.k)) sh.ambiguous |= 2;
                    __syncthreads();
                    if (tid < ctas) {
                        st_dsmem_u64(mapa_shared(smem_u32(&sh.cut), tid), sh.list[sh.fails - 1]);
                        st_dsmem_u32(mapa_shared(smem_u32(&sh.kept), tid), sh.fails);
                        if (tid > 0) st_dsmem_u32(mapa_shared(smem_u32(&sh.ambiguous), tid), sh.ambiguous);
                    }
                }
                filter_sync(ctas);
                const uint32_t state = sh.ambiguous;
                cut = sh.cut, kept = static_cast<int>(sh.kept);
                listed = !(state & 2);
                if (!(state & 1)) break;
                filter_sync(ctas);  // all have read it
                precise = true;
                set_total(g);
            }
            if (!listed) cut = 0, kept = valid;
        }
        if (!listed) {
            const float about = count_bins();
            if (want_p && !want_k) g.off = about - g.total * kFilterUnit;
            FilterGoal h = g;
            if (want_k) cut = search(h, kept);
            if (want_p && kept > 1) {
                if (want_k) {  // the row's histogram again: a search may have used its place
                    count_bins();
                    h.set = cut;
                    set_total(h);
                }
                h.by_mass = true;
                cut = search(h, kept);
            }
        }
    }
    // ---- what is kept
    if constexpr (!SAMPLE) {
        int count = 0;
        // keys as floats: the cut's logit, and of equal ones those up to its token
        const float cut_x = cut ? filter_value(static_cast<uint32_t>(cut >> 32)) : -INFINITY;
        const int cut_i = cut ? static_cast<int>(~static_cast<uint32_t>(cut)) - v0 : -1;
        auto write = [&](auto keep) {
#pragma unroll 4
            for (int i = tid; i < n4; i += kFilterThreads) {
                float4 x = x4[i];
                x.x = keep(x.x, 4 * i) ? x.x : -INFINITY, x.y = keep(x.y, 4 * i + 1) ? x.y : -INFINITY;
                x.z = keep(x.z, 4 * i + 2) ? x.z : -INFINITY, x.w = keep(x.w, 4 * i + 3) ? x.w : -INFINITY;
                if (vec && 4 * i + 3 < n) {
                    *reinterpret_cast<float4 *>(out + 4 * i) = x;
                } else {
                    out[4 * i] = x.x;
                    if (4 * i + 1 < n) out[4 * i + 1] = x.y;
                    if (4 * i + 2 < n) out[4 * i + 2] = x.z;
                    if (4 * i + 3 < n) out[4 * i + 3] = x.w;
                }
            }
        };
        if (listed) {  // -inf is there already
            for (int i = tid; i < static_cast<int>(sh.n_pick); i += kFilterThreads) {
                const int at = sh.pick[i];
                const float x = x_s[at];
                if (x > cut_x || (x == cut_x && at <= cut_i)) out[at] = x;
            }
        } else if (want_m)
            write([&](float x, int i) {
                const bool yes = (x > cut_x || (x == cut_x && i <= cut_i)) && strong(x);
                count += yes;
                return yes;
            });
        else
            write([&](float x, int i) { return x > cut_x || (x == cut_x && i <= cut_i); });
        if (a.n_kept) {
            if (want_m && !listed) {
                FilterSums s = {static_cast<unsigned long long>(count), 0, 0ull, none};
                kept = static_cast<int>(filter_reduce<kSumA>(sh, s, ctas, rank, turn++).a);
            }
            if (rank == 0 && tid == 0) a.n_kept[row] = kept;
        }
    } else {
        // the race: w / noise, the two largest of a thread; 2^-14 apart they are decided, if fp32 holds them. Of a list CTA 0 alone
        // runs it.
        const float *noise = a.noise + row * a.noise_stride;
        const int racers = listed ? 1 : ctas;
        if (!listed || rank == 0) {
            auto runners = [&](auto f) {  // f(logit, token)
                if (listed) {
                    for (int i = tid; i < kept; i += kFilterThreads)
                        f(filter_value(static_cast<uint32_t>(sh.list[i] >> 32)), static_cast<int>(~static_cast<uint32_t>(sh.list[i])));
                } else if (kept == 1) {
                    const int at = static_cast<int>(~static_cast<uint32_t>(cut)) - v0;
                    if (tid == 0 && at >= 0 && at < n) f(x_s[at], v0 + at);
                } else {
                    each([&](float x, int i) {
                        if ((cut == 0 || filter_key(x, v0 + i) >= cut) && strong(x)) f(x, v0 + i);
                    });
                }
            };
            // infinite where a quotient could pass fp32's range; elsewhere a weight that was flushed to zero scores below 2^-86
            auto score = [&](float x, int v) {
                const float e = noise[v];
                return e > 0.f && e < 0x1p-40f ? INFINITY : filter_weight(r, x) * __frcp_rn(e);
            };
            float s1 = -1.f, s2 = -1.f;
            int at = 0, count = 0;
            runners([&](float x, int v) {
                const float s = score(x, v);
                ++count;
                if (s > s1 || (s == s1 && v < at))
                    s2 = s1, s1 = s, at = v;
                else
                    s2 = fmaxf(s2, s);
            });
            FilterSums s = {static_cast<unsigned long long>(count), 0,
                            s1 >= 0.f ? static_cast<unsigned long long>(__float_as_uint(s1)) << 32 | static_cast<uint32_t>(~at) : 0ull, none};
            s = filter_reduce<kSumA | kHi>(sh, s, racers, rank, turn++);
            kept = static_cast<int>(s.a);
            unsigned long long won = s.hi ? s.hi : top;  // no noise above zero
            const float best = __uint_as_float(static_cast<uint32_t>(s.hi >> 32));
            const float near = best < INFINITY && best > 0x1p-60f ? best * (1.f - 0x1p-14f) : 0.f;  // else all
            FilterSums t = {(s1 >= near && s1 >= 0.f ? 1ull : 0ull) + (s2 >= near && s2 >= 0.f ? 1ull : 0ull), 0, 0ull, none};
            t = filter_reduce<kSumA>(sh, t, racers, rank, turn++);
            if (t.a > 1) {  // near ones again, in 64 bits
                double top_score = -1.;
                int who = 0;
                runners([&](float x, int v) {
                    if (score(x, v) >= near) {
                        const double w = x == r.m ? 1. : exp((static_cast<double>(x) - static_cast<double>(r.m)) / static_cast<double>(T));
                        const double exact = w / static_cast<double>(noise[v]);
                        if (exact > top_score || (exact == top_score && v < who)) top_score = exact, who = v;
                    }
                });
                FilterSums u = {0, 0, top_score >= 0. ? static_cast<unsigned long long>(__double_as_longlong(top_score)) : 0ull, none};
                const unsigned long long mine = u.hi;
                u = filter_reduce<kHi>(sh, u, racers, rank, turn++);
                FilterSums f = {0, 0, 0ull, top_score >= 0. && mine == u.hi ? static_cast<unsigned long long>(who) : none};
                f = filter_reduce<kLo>(sh, f, racers, rank, turn++);
                won = static_cast<uint32_t>(~static_cast<uint32_t>(f.lo));
            }
            if (rank == 0 && tid == 0) {
                a.tokens[row] = static_cast<int>(~static_cast<uint32_t>(won));
                if (a.n_kept) a.n_kept[row] = kept;
            }
        }
    }
    if (ctas > 1) cluster_sync();  // nobody leaves while its shared memory may be read
}

}  // namespace sdv
