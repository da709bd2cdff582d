// Attention over the 8-bit cache.
#pragma once

#include "qcache.cuh"

namespace sdv {

struct QAttnArgs {
    QCacheArgs c;
    const void *q;
    void *out;
    long long q_stride, out_stride;  // elements between rows
    int nq, window;                  // window: positions a row sees, its own the last (0: all)
    float scale_log2;                // log2(e) / sqrt(D)
};

constexpr int kQSimpleThreads = 128;

// One CTA per (span row, q head, sequence): its warps take 32 keys at a time, a lane one key, with a
// running maximum and sum a warp, joined at the end.
template <typename T, int D>
__global__ void __launch_bounds__(kQSimpleThreads) qcache_attn_simple_kernel(QAttnArgs a) {
    pdl_trigger();
    pdl_wait();
    const QCacheArgs &c = a.c;
    const int i = blockIdx.x, hq = blockIdx.y, b = blockIdx.z, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const QSpan s = qcache_span(c, b);
    T *out = static_cast<T *>(a.out);
    if (s.S == 0) {
        if (s.code != SDV_OK && i == 0 && hq == 0 && tid == 0) set_status(c.status, s.code);
        for (int r = i; r < s.rows; r += gridDim.x)  // refused: NaN rather than stale memory
            for (int d = tid; d < D; d += kQSimpleThreads)
                out[(s.r0 + r) * a.out_stride + hq * D + d] = from_f32<T>(NAN);
        return;
    }
    if (i >= s.S) return;
    __shared__ float q_s[D], o_s[4][D], m_s[4], l_s[4];
    const T *q = static_cast<const T *>(a.q) + (s.r0 + i) * a.q_stride + hq * D;
    for (int d = tid; d < D; d += kQSimpleThreads) q_s[d] = to_f32(q[d]) * a.scale_log2;
    __syncthreads();
    const int pos = s.p0 + i, h = hq / (a.nq / c.nkv), first = a.window > 0 ? max(0, pos - a.window + 1) : 0;
    const int nblk = c.page_size / c.scale_block;
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d) o[d] = 0.f;
    for (int t0 = first + warp * 32; t0 <= pos; t0 += 128) {
        const int t = t0 + lane;
        float sc = -INFINITY, vs = 0.f;
        size_t vrow = 0;
        if (t <= pos) {
            const int page = qcache_page(c, b, t / c.page_size), slot = t % c.page_size;
            sc = 0.f;
            if (page >= 0) {
                const size_t ph = (static_cast<size_t>(page) * 2) * c.nkv + h;
                const uint2 *kc = reinterpret_cast<const uint2 *>(c.codes + (ph * c.page_size + slot) * D);
                for (int d = 0; d < D / 8; ++d) {
                    const uint2 w = kc[d];
                    const uint32_t r[4] = {w.x & 0xffffu, w.x >> 16, w.y & 0xffffu, w.y >> 16};
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = e4m3x2_f32(r[j]);
                        sc = fmaf(f.x, q_s[8 * d + 2 * j], fmaf(f.y, q_s[8 * d + 2 * j + 1], sc));
                    }
                }
                sc *= c.scales[ph * nblk + slot / c.scale_block];
                vs = c.scales[(ph + c.nkv) * nblk + slot / c.scale_block];
                vrow = ((ph + c.nkv) * c.page_size + slot) * D;
            }
        }
        float mn = sc;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) mn = fmaxf(mn, __shfl_xor_sync(0xffffffffu, mn, x));
        mn = fmaxf(mn, m);
        const float alpha = exp2f(m - mn), p = exp2f(sc - mn);
        m = mn;
        l = l * alpha + warp_sum(p);
#pragma unroll
        for (int d = 0; d < D / 32; ++d) o[d] *= alpha;
        for (int j = 0; j < 32; ++j) {
            const float pv = __shfl_sync(0xffffffffu, p, j) * __shfl_sync(0xffffffffu, vs, j);
            const size_t row = __shfl_sync(0xffffffffu, vrow, j);
            if (pv == 0.f) continue;
#pragma unroll
            for (int d = 0; d < D / 32; ++d) {
                const uint32_t code = c.codes[row + d * 32 + lane];
                o[d] = fmaf(pv, e4m3x2_f32(code).x, o[d]);
            }
        }
    }
    if (lane == 0) m_s[warp] = m, l_s[warp] = l;
#pragma unroll
    for (int d = 0; d < D / 32; ++d) o_s[warp][d * 32 + lane] = o[d];
    __syncthreads();
    const float mx = fmaxf(fmaxf(m_s[0], m_s[1]), fmaxf(m_s[2], m_s[3]));
    for (int d = tid; d < D; d += kQSimpleThreads) {
        float num = 0.f, den = 0.f;
        for (int w = 0; w < 4; ++w) {
            const float f = exp2f(m_s[w] - mx);
            num += f * o_s[w][d];
            den += f * l_s[w];
        }
        out[(s.r0 + i) * a.out_stride + hq * D + d] = from_f32<T>(num / den);
    }
}

}  // namespace sdv
