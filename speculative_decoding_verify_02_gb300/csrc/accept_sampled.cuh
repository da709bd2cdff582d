// Sampled acceptance: drafted tokens verified against the target's probabilities from given random
// numbers (the rejection rule of speculative sampling), two kernels.
//
// With p_r = softmax(logits_r / T) and q_r the distribution draft d (token of row r + 1) was drawn
// from, d is accepted iff u_r q_r(d) < p_r(d). The first row whose draft is not accepted commits a
// token drawn from max(p - q, 0) (normalised), the last row of a fully accepted span one from p; the
// committed tokens are then distributed as the target's own samples. A draw from weights w is
// argmax_v w_v / e_v with e exponential noise: the scores' maximum falls on v with probability
// w_v / sum w (competing exponentials), no sum over the vocabulary is needed, and the two best scores
// differ by a factor of order one, so float32 weights decide it as exact ones would (a cumulative sum
// over 150,000 weights has borders closer than its own rounding).
#pragma once

#include "common.cuh"
#include "small.cuh"

namespace sdv {

constexpr int kAcceptThreads = 256;
constexpr int kAcceptPer = 16;                               // logits a thread holds
constexpr int kAcceptChunk = kAcceptThreads * kAcceptPer;    // logits of one statistics CTA
constexpr int kDrawThreads = 512;
constexpr int kDrawCluster = 8;                              // CTAs that share a sequence's draw
constexpr int kAcceptMaxSpan = 128;

struct AcceptSampledArgs {
    DevState s;
    const int *tokens, *row_off;
    const float *logits, *temperature, *uniform, *noise, *probs;
    long long logits_stride, noise_stride, probs_stride;  // floats between rows
    int B, max_span, max_commit, vocab, n_chunks, rows_cap, adaptive, k_max;
    float2 *part;  // [rows_cap][n_chunks]: (max, sum) of a chunk, or (max, index of the max) of a greedy row
    int *n_accept, *committed, *n_commit, *new_len;
};

// First row and length of sequence b's span; length 0 where the span is empty or not usable.
__device__ __forceinline__ int2 accept_span(const AcceptSampledArgs &p, int b) {
    const int r0 = p.row_off[b], S = p.row_off[b + 1] - r0;
    const bool ok = S > 0 && S <= p.max_span && r0 >= 0 && r0 + S <= p.rows_cap;
    return make_int2(r0, ok ? S : 0);
}

// Weight of logit x against the row's maximum m: exp((x - m) / T) with c = log2(e) / T. NaN and -inf
// weigh nothing; the maximum weighs one whatever it is (an infinite maximum shares the row).
__device__ __forceinline__ float logit_weight(float x, float m, float c) {
    if (x == m) return 1.f;
    return x > -INFINITY && x < m ? exp2f((x - m) * c) : 0.f;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}
__device__ __forceinline__ unsigned long long warp_max_u64(unsigned long long v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const unsigned long long w = __shfl_xor_sync(0xffffffffu, v, o);
        v = w > v ? w : v;
    }
    return v;
}

// Statistics of one chunk of one row: grid (chunks, B * max_span).
__global__ void __launch_bounds__(kAcceptThreads) accept_stats_kernel(AcceptSampledArgs p) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.y / p.max_span, i = blockIdx.y % p.max_span;
    const int2 sp = accept_span(p, b);
    if (i >= sp.y) return;
    const int r = sp.x + i;
    const float T = p.temperature[b];
    const float *row = p.logits + r * p.logits_stride;
    const int v0 = blockIdx.x * kAcceptChunk, tid = threadIdx.x;
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0 && v0 + kAcceptChunk <= p.vocab;
    float x[kAcceptPer];
#pragma unroll
    for (int j = 0; j < kAcceptPer / 4; ++j) {
        const int v = v0 + (j * kAcceptThreads + tid) * 4;
        if (vec) {
            const float4 f = *reinterpret_cast<const float4 *>(row + v);
            x[4 * j] = f.x, x[4 * j + 1] = f.y, x[4 * j + 2] = f.z, x[4 * j + 3] = f.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * j + k] = v + k < p.vocab ? row[v + k] : -INFINITY;
        }
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kAcceptPer; ++j) m = fmaxf(m, x[j]);  // fmaxf passes over NaN
    __shared__ float red_m[kAcceptThreads / 32], red_l[kAcceptThreads / 32];
    __shared__ int best;
    const int warp = tid / 32, lane = tid % 32;
    m = warp_max(m);
    if (lane == 0) red_m[warp] = m;
    if (tid == 0) best = 0x7fffffff;
    __syncthreads();
    m = red_m[0];
#pragma unroll
    for (int w = 1; w < kAcceptThreads / 32; ++w) m = fmaxf(m, red_m[w]);
    float2 *out = p.part + static_cast<size_t>(r) * p.n_chunks + blockIdx.x;
    if (!(T > 0.f)) {  // greedy row: the lowest index of the maximum
        if (m > -INFINITY) {
#pragma unroll
            for (int j = 0; j < kAcceptPer; ++j)
                if (x[j] == m) atomicMin(&best, v0 + ((j / 4) * kAcceptThreads + tid) * 4 + (j & 3));
        }
        __syncthreads();
        if (tid == 0) *out = make_float2(m, __int_as_float(best));
        return;
    }
    const float c = 1.4426950408889634f / T;
    float l = 0.f;
    if (m > -INFINITY) {
#pragma unroll
        for (int j = 0; j < kAcceptPer; ++j) l += logit_weight(x[j], m, c);
    }
    l = warp_sum(l);
    if (lane == 0) red_l[warp] = l;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kAcceptThreads / 32; ++w) l += red_l[w];
        *out = make_float2(m, l);
    }
}

// One cluster per sequence: the accepted prefix (each CTA finds it from the chunk statistics), the
// race over the vocabulary split over the CTAs, and the outputs and loop state as accept_kernel
// writes them.
__global__ void __launch_bounds__(kDrawThreads) accept_draw_kernel(AcceptSampledArgs p) {
    pdl_trigger();
    pdl_wait();
    const int b = blockIdx.x / kDrawCluster;
    const uint32_t rank = cluster_ctarank();
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int2 sp = accept_span(p, b);
    const int r0 = sp.x, S = sp.y;
    if (S == 0) {  // the whole cluster leaves together
        if (rank == 0 && tid == 0) {
            if (p.row_off[b + 1] != r0) set_status(p.s.status, SDV_ERR_ARG);
            p.n_accept[b] = -1;
            p.n_commit[b] = 0;
            p.new_len[b] = -1;
        }
        return;
    }
    __shared__ float row_m[kAcceptMaxSpan], row_l[kAcceptMaxSpan];
    __shared__ int row_best[kAcceptMaxSpan], row_ok[kAcceptMaxSpan], m_s;
    __shared__ unsigned long long keys[2][kDrawThreads / 32], cta_key[2];
    const float T = p.temperature[b];
    const bool greedy = !(T > 0.f);
    const float c = 1.4426950408889634f / T;
    for (int i = warp; i < S; i += kDrawThreads / 32) {
        const int r = r0 + i;
        const float2 *part = p.part + static_cast<size_t>(r) * p.n_chunks;
        float m = -INFINITY, l = 0.f;
        int best = 0x7fffffff;
        for (int k = lane; k < p.n_chunks; k += 32) m = fmaxf(m, part[k].x);
        m = warp_max(m);
        for (int k = lane; k < p.n_chunks; k += 32) {
            const float2 t = part[k];
            if (greedy) {
                if (t.x == m) best = min(best, __float_as_int(t.y));
            } else {
                l += t.y * logit_weight(t.x, m, c);
            }
        }
        l = warp_sum(l);
        best = __reduce_min_sync(0xffffffffu, best);
        if (lane == 0) {
            row_m[i] = m;
            row_l[i] = l;
            row_best[i] = best;
            int ok = 0;
            if (i + 1 < S && m > -INFINITY) {
                const int d = p.tokens[r + 1];
                if (d >= 0 && d < p.vocab) {
                    const float q = p.probs ? p.probs[r * p.probs_stride + d] : 1.f;
                    // the draft's own weight in 64 bits: one value a row, and the one that decides
                    const float x = p.logits[r * p.logits_stride + d];
                    double pd;
                    if (greedy)
                        pd = d == best ? 1.0 : 0.0;
                    else if (x == m)
                        pd = 1.0 / l;
                    else
                        pd = x > -INFINITY && x < m
                                 ? exp((static_cast<double>(x) - static_cast<double>(m)) / static_cast<double>(T)) / l
                                 : 0.0;
                    ok = static_cast<double>(p.uniform[r]) * static_cast<double>(q) < pd;
                }
            }
            row_ok[i] = ok;
        }
    }
    __syncthreads();
    if (tid == 0) {
        int m = 0;
        while (m < S - 1 && row_ok[m]) ++m;
        m_s = m;
    }
    __syncthreads();
    const int m = m_s, r = r0 + m;
    const bool rejected = m < S - 1;
    const float xm = row_m[m];
    int token = 0;
    if (greedy) {
        token = xm > -INFINITY ? row_best[m] : 0;
    } else {
        const float inv_l = 1.f / row_l[m];
        const float *x = p.logits + r * p.logits_stride, *e = p.noise + b * p.noise_stride;
        const float *q = rejected && p.probs ? p.probs + r * p.probs_stride : nullptr;
        const int drop = rejected && !p.probs ? p.tokens[r + 1] : -1;  // a certain draft leaves no weight
        // best score over max(p - q, 0), and over p in case nothing is left of it
        float s0 = -1.f, s1 = -1.f;
        int i0 = 0, i1 = 0;
        auto consider = [&](int v, float xv, float qv, float ev) {
            const float pv = logit_weight(xv, xm, c) * inv_l;
            const float w = v == drop ? 0.f : pv - qv;
            const float t0 = w > 0.f ? w / ev : -1.f, t1 = pv > 0.f ? pv / ev : -1.f;
            if (t0 > s0) s0 = t0, i0 = v;
            if (t1 > s1) s1 = t1, i1 = v;
        };
        const bool vec = ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(e) |
                           reinterpret_cast<uintptr_t>(q)) & 15) == 0;
        const int nvec = vec ? p.vocab / 4 : 0;
        for (int k = rank * kDrawThreads + tid; k < nvec; k += kDrawCluster * kDrawThreads) {
            const float4 xv = reinterpret_cast<const float4 *>(x)[k], ev = reinterpret_cast<const float4 *>(e)[k];
            const float4 qv = q ? reinterpret_cast<const float4 *>(q)[k] : make_float4(0.f, 0.f, 0.f, 0.f);
            consider(4 * k, xv.x, qv.x, ev.x);
            consider(4 * k + 1, xv.y, qv.y, ev.y);
            consider(4 * k + 2, xv.z, qv.z, ev.z);
            consider(4 * k + 3, xv.w, qv.w, ev.w);
        }
        for (int v = 4 * nvec + rank * kDrawThreads + tid; v < p.vocab; v += kDrawCluster * kDrawThreads)
            consider(v, x[v], q ? q[v] : 0.f, e[v]);
        // scores are >= 0, so their bits order them; the complement of the index breaks ties low
        auto pack = [](float s, int v) {
            return s < 0.f ? 0ull
                           : (static_cast<unsigned long long>(__float_as_uint(s)) << 32 | static_cast<uint32_t>(~v));
        };
        const unsigned long long k0 = warp_max_u64(pack(s0, i0)), k1 = warp_max_u64(pack(s1, i1));
        if (lane == 0) keys[0][warp] = k0, keys[1][warp] = k1;
        __syncthreads();
        if (warp < 2) {
            const unsigned long long k = warp_max_u64(lane < kDrawThreads / 32 ? keys[warp][lane] : 0ull);
            if (lane == 0) cta_key[warp] = k;
        }
        cluster_sync();
        if (rank == 0 && warp == 0) {
            unsigned long long k[2];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                k[t] = 0;
                if (lane < kDrawCluster) {
                    const float2 f = ld_dsmem_f2(mapa_shared(smem_u32(&cta_key[t]), lane));
                    k[t] = static_cast<unsigned long long>(__float_as_uint(f.y)) << 32 | __float_as_uint(f.x);
                }
                k[t] = warp_max_u64(k[t]);
            }
            const unsigned long long won = k[0] ? k[0] : k[1];
            token = won ? static_cast<int>(~static_cast<uint32_t>(won)) : 0;
        }
        cluster_sync();  // no CTA leaves while its key may still be read
    }
    if (rank != 0 || warp != 0) return;
    for (int i = lane; i < m; i += 32) p.committed[static_cast<size_t>(b) * p.max_commit + i] = p.tokens[r0 + 1 + i];
    if (lane != 0) return;
    if (xm == -INFINITY) set_status(p.s.status, SDV_ERR_DEVICE);  // a row without a logit to draw
    for (int i = 0; i <= m && i + 1 < S; ++i) {
        const int d = p.tokens[r0 + 1 + i];
        if (d < 0 || d >= p.vocab) set_status(p.s.status, SDV_ERR_DEVICE);
    }
    p.committed[static_cast<size_t>(b) * p.max_commit + m] = token;
    p.n_accept[b] = m;
    p.n_commit[b] = m + 1;
    p.new_len[b] = p.s.seq_len[b] - S + m + 1;
    // loop state: next current token, tokens generated, adaptive draft length
    const int k = S - 1;
    p.s.cur_tok[b] = token;
    p.s.generated[b] += m + 1;
    if (p.adaptive && k > 0) p.s.kcur[b] = (m == k) ? min(p.s.kcur[b] + 2, p.k_max) : max(p.s.kcur[b] - 1, 1);
}

}  // namespace sdv
