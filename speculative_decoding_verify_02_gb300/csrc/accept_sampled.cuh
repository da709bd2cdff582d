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
constexpr int kAcceptMaxSpan = 128;

struct AcceptSampledArgs {
    DevState s;
    const int *tokens, *row_off;
    const float *logits, *temperature, *uniform, *noise, *probs;
    long long logits_stride, noise_stride, probs_stride;  // floats between rows
    int B, max_span, max_commit, vocab, n_chunks, rows_cap, adaptive, k_max;
    float2 *part;  // [rows_cap][n_chunks]: (max, sum) of a chunk, or (max, index of the max) of a greedy row
    unsigned long long *keys;  // [max_batch][2]: best score so far, over max(p - q, 0) and over p
    int *arrived;              // [max_batch]: chunks that have put in theirs
    int *n_accept, *committed, *n_commit, *new_len;
};

// First row and length of sequence b's span; length 0 where the span is empty or not usable.
__device__ __forceinline__ int2 accept_span(const AcceptSampledArgs &p, int b) {
    const int r0 = p.row_off[b], S = p.row_off[b + 1] - r0;
    const bool ok = S > 0 && S <= p.max_span && r0 >= 0 && r0 <= p.rows_cap - S;  // S is small: no overflow
    return make_int2(r0, ok ? S : 0);
}

// Weight of logit x against the row's maximum m: exp((x - m) / T) with c = log2(e) / T. NaN and -inf
// weigh nothing; the maximum weighs one whatever it is (an infinite maximum shares the row). A row without a logit,
// m = -inf, is the caller's to leave out (asked here, for every logit, it costs 8 rows 2 us of 12.4).
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

// Sixteen values a thread of a chunk of a row: four groups of four, coalesced, `fill` past the vocabulary.
__device__ __forceinline__ void load_chunk(const float *row, int v0, int vocab, float fill, float (&x)[kAcceptPer]) {
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15) == 0 && v0 + kAcceptChunk <= vocab;
#pragma unroll
    for (int j = 0; j < kAcceptPer / 4; ++j) {
        const int v = v0 + (j * kAcceptThreads + threadIdx.x) * 4;
        if (vec) {
            const float4 f = *reinterpret_cast<const float4 *>(row + v);
            x[4 * j] = f.x, x[4 * j + 1] = f.y, x[4 * j + 2] = f.z, x[4 * j + 3] = f.w;
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) x[4 * j + k] = v + k < vocab ? row[v + k] : fill;
        }
    }
}
// Vocabulary index of value j of this thread.
__device__ __forceinline__ int chunk_index(int v0, int j) {
    return v0 + ((j / 4) * kAcceptThreads + threadIdx.x) * 4 + (j & 3);
}

// Statistics of one chunk of one row: grid (chunks, rows). The row's logits are asked for before its
// sequence is known: 128 rows of 151,936 (78 MB) keep 4 waves of CTAs busy, and every latency in a CTA's chain counts
// in each. Bound by memory: those in 19.5 us, 4.0 TB/s (CTAs that stay and ask for their next chunk ahead: 23.5 us).
__global__ void __launch_bounds__(kAcceptThreads) accept_stats_kernel(AcceptSampledArgs p) {
    pdl_wait();
    pdl_trigger();
    const int r = blockIdx.y, v0 = blockIdx.x * kAcceptChunk, tid = threadIdx.x;
    float x[kAcceptPer];
    load_chunk(p.logits + r * p.logits_stride, v0, p.vocab, -INFINITY, x);
    __shared__ int seq_s;
    if (tid == 0) seq_s = -1;
    __syncthreads();
    if (tid < p.B) {  // B <= 256 threads
        const int2 sp = accept_span(p, tid);
        if (r >= sp.x && r < sp.x + sp.y) seq_s = tid;
    }
    __syncthreads();
    const int b = seq_s;
    if (b < 0) return;  // a row of no span
    const float T = p.temperature[b];
    if (blockIdx.x == 0 && r == p.row_off[b] && tid < 2) {  // for the draw that follows
        p.keys[2 * b + tid] = 0;
        if (tid == 0) p.arrived[b] = 0;
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
                if (x[j] == m) atomicMin(&best, chunk_index(v0, j));
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

__device__ __forceinline__ double logit_weight64(float x, float m, float T) {
    if (!(x > -INFINITY)) return 0.;
    return x == m ? 1. : exp((static_cast<double>(x) - static_cast<double>(m)) / static_cast<double>(T));
}
// u q < w(x) / l in 64 bits, by a whole warp. The row's float sum l decides where it can: its weights are off by
// 2.3 a 2^-24 (a = (m - x) / T log2 e; the roundings of x - m, log2 e / T and their product) and two exp2f's
// 4 2^-24, a averages log2 of the vocabulary at most over the weights, and at most 34 + n_chunks / 32 additions follow one
// another: below (90 + n_chunks) 2^-24 altogether for n_chunks * 4,096 logits. Nearer than that to the border, at most one draft in
// 2^16, the row is summed again: 1.2 ms for 151,936 logits, bound by 64-bit products.
__device__ __forceinline__ bool accept_near(const float *row, int vocab, int n_chunks, float x, float m, float l, float T, float u,
                                         float q) {
    const double uq = static_cast<double>(u) * static_cast<double>(q), w = logit_weight64(x, m, T), lw = uq * l;
    if (!(w > 0.) || fabs(lw - w) > (90 + n_chunks) * 0x1p-24 * w) return lw < w;
    double sum = 0.;
    for (int v = threadIdx.x % 32; v < vocab; v += 32) sum += logit_weight64(row[v], m, T);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return uq * sum < w;
}

// The accepted prefix of a sequence (every CTA finds it from the chunk statistics), the race over one
// chunk of the vocabulary at its last row, and, in the CTA that comes last, the outputs and loop state as
// accept_kernel writes them. Grid (chunks, B). The best key is the same in any order of arrival. One sequence of
// eight rows, both kernels: 10.4 us, a chain of launches and dependent reads; 16 with drafter probabilities: 30.4 us.
__global__ void __launch_bounds__(kAcceptThreads, 4) accept_draw_kernel(AcceptSampledArgs p) {
    pdl_wait();
    pdl_trigger();
    constexpr int NW = kAcceptThreads / 32;
    const int b = blockIdx.y, v0 = blockIdx.x * kAcceptChunk, tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int2 sp = accept_span(p, b);
    const int r0 = sp.x, S = sp.y;
    if (S == 0) {
        if (blockIdx.x == 0 && tid == 0) {
            if (p.row_off[b + 1] != r0) set_status(p.s.status, SDV_ERR_ARG);
            p.n_accept[b] = -1;
            p.n_commit[b] = 0;
            p.new_len[b] = -1;
        }
        return;
    }
    __shared__ float row_m[kAcceptMaxSpan], row_l[kAcceptMaxSpan];
    __shared__ int row_best[kAcceptMaxSpan], row_ok[kAcceptMaxSpan], m_s, last_s;
    __shared__ unsigned long long keys[2][NW];
    const float T = p.temperature[b];
    const bool greedy = !(T > 0.f);
    if (greedy && blockIdx.x > 0) return;  // the statistics hold the answer
    const float c = 1.4426950408889634f / T;
    // what the last CTA will need, asked for early
    const int length = p.s.seq_len[b], done = p.s.generated[b], kcur = p.s.kcur[b];
    float e[kAcceptPer];
    if (!greedy) load_chunk(p.noise + b * p.noise_stride, v0, p.vocab, 1.f, e);
    for (int i = warp; i < S; i += NW) {
        const int r = r0 + i, d = i + 1 < S ? p.tokens[r + 1] : -1;
        const bool draft = d >= 0 && d < p.vocab;
        // asked for ahead of the sums
        const float q = draft && p.probs ? p.probs[r * p.probs_stride + d] : 1.f, u = p.uniform[r];
        const float x = draft ? p.logits[r * p.logits_stride + d] : 0.f;
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
        bool ok = false;
        if (draft && m > -INFINITY) {
            if (greedy) {
                ok = d == best && u * q < 1.f;
            } else {
                const float uq = u * q, pd = logit_weight(x, m, c) / l;
                ok = uq < pd;
                // the draft's own weight is off by 2.3 (m - x) / T log2 e + 4 of 2^-24, its exponent below 150, and the
                // sum as said at accept_near: together below 512 + n_chunks. Where p is no normal number: 2^-140
                if (fabsf(uq - pd) <= (512 + p.n_chunks) * 0x1p-24f * pd + 0x1p-140f)
                    ok = accept_near(p.logits + r * p.logits_stride, p.vocab, p.n_chunks, x, m, l, T, u, q);
            }
        }
        if (lane == 0) {
            row_m[i] = m;
            row_l[i] = l;
            row_best[i] = best;
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
    if (!(xm > -INFINITY)) {  // no logit to draw: token 0, from one CTA
        if (blockIdx.x > 0) return;
    } else if (greedy) {
        token = row_best[m];
    } else {
        const float inv_l = 1.f / row_l[m];
        const int drop = rejected && !p.probs ? p.tokens[r + 1] : -1;  // a certain draft leaves no weight
        float x[kAcceptPer], q[kAcceptPer];
        load_chunk(p.logits + r * p.logits_stride, v0, p.vocab, -INFINITY, x);
        if (rejected && p.probs) {
            load_chunk(p.probs + r * p.probs_stride, v0, p.vocab, 0.f, q);
        } else {
#pragma unroll
            for (int j = 0; j < kAcceptPer; ++j) q[j] = 0.f;
        }
        // best score over max(p - q, 0), and over p in case nothing is left of it; a thread's indexes ascend
        float s0 = -1.f, s1 = -1.f;
        int i0 = 0, i1 = 0;
#pragma unroll
        for (int j = 0; j < kAcceptPer; ++j) {
            const int v = chunk_index(v0, j);
            const float pv = logit_weight(x[j], xm, c) * inv_l, w = v == drop ? 0.f : pv - q[j];
            const float inv = __frcp_rn(e[j]), t0 = w > 0.f ? w * inv : -1.f, t1 = pv > 0.f ? pv * inv : -1.f;
            if (t0 > s0) s0 = t0, i0 = v;
            if (t1 > s1) s1 = t1, i1 = v;
        }
        // scores are >= 0, so their bits order them; the complement of the index breaks ties low
        auto pack = [](float s, int v) {
            return s < 0.f ? 0ull
                           : (static_cast<unsigned long long>(__float_as_uint(s)) << 32 | static_cast<uint32_t>(~v));
        };
        const unsigned long long k0 = warp_max_u64(pack(s0, i0)), k1 = warp_max_u64(pack(s1, i1));
        if (lane == 0) keys[0][warp] = k0, keys[1][warp] = k1;
        __syncthreads();
        if (tid == 0) {
            unsigned long long best[2] = {0, 0};
#pragma unroll
            for (int w = 0; w < NW; ++w)
#pragma unroll
                for (int t = 0; t < 2; ++t) best[t] = keys[t][w] > best[t] ? keys[t][w] : best[t];
            if (best[0]) atomicMax(&p.keys[2 * b], best[0]);
            if (best[1]) atomicMax(&p.keys[2 * b + 1], best[1]);
            __threadfence();
            last_s = atomicAdd(&p.arrived[b], 1) == p.n_chunks - 1;
            if (last_s) {
                __threadfence();
                const unsigned long long a0 = atomicMax(&p.keys[2 * b], 0ull), a1 = atomicMax(&p.keys[2 * b + 1], 0ull);
                const unsigned long long won = a0 ? a0 : a1;
                m_s = won ? static_cast<int>(~static_cast<uint32_t>(won)) : 0;
            }
        }
        __syncthreads();
        if (!last_s) return;
        token = m_s;
    }
    if (warp != 0) return;
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
    p.new_len[b] = length - S + m + 1;
    // loop state: next current token, tokens generated, adaptive draft length
    const int k = S - 1;
    p.s.cur_tok[b] = token;
    p.s.generated[b] = done + m + 1;
    if (p.adaptive && k > 0) p.s.kcur[b] = (m == k) ? min(kcur + 2, p.k_max) : max(kcur - 1, 1);
}

}  // namespace sdv
