// Attention over the 8-bit cache on the fp8 tensor cores.
//
// For one kv head, ROWS query rows (span row x head of the group) against 128 keys at a time:
//     S^T [128 keys x rows] = K . Q^T          (A = the K codes as they lie in the cache, B = Q)
//     O^T [dims x rows]     = V^T . P^T        (A = the V codes read along the other axis, B = P)
// so K and V enter the tensor cores as the bytes they are, a key (then a dim) to a TMEM lane, and the few query rows of
// a verify step are the narrow operand: an MMA of 128 lanes and 32 of depth costs 46 clocks for any width up to 64, 56
// at 96, 64 at 128 (measured), 400 for the eight of a chunk of 32 rows, against the 1,370 that its 32 KB take at this
// SM's share of HBM.
//
// The 16-bit operand of each product is split into e4m3 planes laid side by side along the width:
//   q = 2^-e (q0 + 2^-5 q1 + 2^-10 q2), e from the tile's largest |q|: two planes hold a bf16's eight
//       bits exactly, three an fp16's eleven (what lies 2^-20 below the largest rounds away);
//   p = x0 + 2^-6 x1 + 2^-11 x2, x = 64 p in (0, 128]: p is rounded to fp16's eleven bits and the planes hold
//       them down to 2^-26 (two planes lost the tail under one large p: 2% off at p = 2^-16).
// The planes' products are added in fp32 afterwards.
//
// A key's V scale is not applied to V: it joins the exponent. With s_t the score in log2 units and
// w_t = s_t + log2 vs_t, x_t = 2^(w_t - M) multiplies the bare codes, M being a row's running maximum of w,
// and the sum l takes 2^(s_t - M); o / l is the result, precise relative to the largest contribution
// however far the scales lie apart. M follows the maximum only when that has grown by more than one
// (hence x up to 2 . 64), so the accumulators are rarely rescaled. A scale below 2^-90 (a block of zeros has
// 2^-126) counts as 2^-90 for M, or the sum of its keys' 2^(s_t - M) would leave fp32's range: where all of a row's
// keys have such scales, its result (below 2^-81) is off by 2^-100 at most.
//
// What bounds it (GB300, 32 q heads on 8 kv heads of 128, bf16): with spans of eight rows a CTA's chain, not the
// bytes: a chunk is two commits, two TMEM reads and 25 to 27 instructions a score, and a unit costs 6,000 to 8,000 clocks more
// for its queries, first maximum and results. In caches whose limit is the call's longest sequence (the parts follow the limit:
// up to 1.5 times as long in larger ones): 32,768 keys in 24.6 us (2.7 TB/s; loads alone reach 6.5), 16 sequences of
// 512 to 4,096 keys in 35.7 us; 848 keys in 8.2 us, one chunk and the joining of seven parts in a cluster (9.0 with a
// merge kernel, and 1.5 us of host more). Long spans read the keys out of L2 once
// a tile and are bound by issue and latency of the softmax: 128 rows at 32,768 keys in 193 us, 2,900 clocks a chunk of
// 64 x 128 scores, half of the issue slots used (tensor pipe 18%).
#pragma once

#include "qcache.cuh"

namespace sdv {

struct QAttnArgs {
    QCacheArgs c;
    const void *q;
    void *out;
    long long q_stride, out_stride;  // elements between rows
    int nq, window;                  // window: positions a row sees, its own the last (0: all)
    int units;                       // B x splits x nkv x tiles
    int *counter;                    // units taken beyond the first of each CTA, CTAs done; both zero between calls
    int splits;                      // parts a sequence's keys are cut into at most
    int cluster;                     // a tile's parts are the CTAs of a cluster, which join them
    int tiles;                       // row tiles of a span of max_span rows
    int grp;                         // q heads a kv head
    int q_vec;                       // q rows are 16-byte aligned
    FastDiv by_tiles, by_kv, by_splits, by_grp, by_nq;
    float scale_log2;                // log2(e) / sqrt(D)
    float *part_o;                   // [sequence][span row][q head][splits][D]
    int box_rows;                    // pool rows of a TMA box; 0: pages that no box fits, copied in 16-byte pieces
    int pool_rows;                   // rows of the layer's pool: a box there reads zeros
    float2 *part_ml;                 // [sequence][span row][q head][splits]: (M, l)
};

constexpr int kQKeys = 128;     // keys of a chunk
constexpr int kQJoin = 8;          // parts that a cluster joins (its portable size), or one warp a row
constexpr float kQLeast = -90.f;   // log2 of a V scale as M counts it, at least
constexpr float kQNoRef = -1e30f;  // a row's M before it has seen a key: below any w, and w - M is no NaN
template <typename T, int D_, int ROWS_>
struct QTile {
    static constexpr int D = D_, ROWS = ROWS_;
    static constexpr int PQ = sizeof(T) == 2 && !__is_same(T, __half) ? 2 : 3;  // planes of q
    static constexpr int PP = 3;                                                  // planes of p
    static constexpr int CW = 16, WG = ROWS / CW;                                 // columns of a softmax warpgroup
    static constexpr int NQ = PQ * ROWS, NP = PP * ROWS;                          // widths of the two products
    static constexpr int CTAS = ROWS == 64 ? 1 : 2, STAGES = ROWS == 64 ? 4 : 2;  // CTAs an SM, chunks in a CTA's memory
    static constexpr int W = ROWS == 32 ? 128 : 64, P_ATOMS = (NP + W - 1) / W;   // bytes of a key's P line, lines a key
    static constexpr int TILE = kQKeys * D;                                       // bytes of a K or V chunk
    static constexpr int Q_BYTES = (NQ * D + 1023) / 1024 * 1024, P_BYTES = kQKeys * W * P_ATOMS;
    static constexpr int SMEM = 1024 + STAGES * 2 * TILE + Q_BYTES + P_BYTES;
    static constexpr int SCALES = 2 * STAGES;  // chunks of scales: loads run STAGES ahead of the scores, those two of softmax
    static constexpr int TMEM = 512 / CTAS;
    static constexpr int NSB = 2 * NQ + NP <= TMEM ? 2 : 1;                       // S^T of the next chunk beside this one's
    static constexpr int O_COL = (NSB * NQ + 31) / 32 * 32;                       // TMEM column of O^T
    static constexpr int COLS = O_COL + NP <= 128 ? 128 : O_COL + NP <= 256 ? 256 : 512;
    // O^T of a unit's chunks grows in TMEM and is taken over where a reference moves, or every chunk's is added up in
    // registers: the long units of long spans move theirs rarely (128 rows at 32K: 193 us against 209), short ones lose
    // (848 keys x 8 rows: 8.5 against 8.3 us, 16 sequences 37.1 against 36.6).
    static constexpr bool GROWS = ROWS == 64;
    static constexpr int THREADS = WG * 128 + 64;  // softmax warps, the load warp, the MMA warp
    static_assert(ROWS == 16 || ROWS == 32 || ROWS == 64, "tile rows");
    static_assert(COLS <= TMEM && O_COL + NP <= COLS, "TMEM columns");
    static_assert(NQ % 16 == 0 && NP % 16 == 0, "MMA widths");
    static_assert(CTAS * (SMEM + 6400 + (SCALES - 4) * 1024 + 1024) <= 228 * 1024, "CTAs per SM");
};

// ------------------------------------------------------------------ PTX
// D[tmem] (+)= A . B^T, kind::f8f6f4 (e4m3 operands, fp32 accumulate), one CTA.
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor: fp32 D, e4m3 A and B; mn: both operands run along M / N in memory.
__host__ __device__ constexpr uint32_t idesc_e4m3(int M, int N, bool mn) {
    return (1u << 4) | (mn ? 3u << 15 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
// Matrix descriptor over lines of `width` bytes (64 or 128) with that width's swizzle, eight lines to an
// atom; `beside` bytes on lie the atoms that continue the lines (0: the same atom again, so that the 64
// dims of V at D = 64 fill both halves of the 128 lanes, of which the upper is not read).
__device__ __forceinline__ uint64_t line_desc(uint32_t addr, int width, uint32_t beside = 0) {
    return static_cast<uint64_t>((addr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(beside >> 4) << 16 | static_cast<uint64_t>(8 * width >> 4) << 32 |
           static_cast<uint64_t>(1) << 46 | static_cast<uint64_t>(width == 128 ? 2 : 4) << 61;
}
// Byte offset of (line, byte) under that swizzle, in a buffer aligned to 1024 bytes.
__device__ __forceinline__ uint32_t line_offset(uint32_t line, uint32_t byte, int width) {
    const uint32_t off = line * width + byte;
    return off ^ ((off >> 7 & (width == 128 ? 7 : 3)) << 4);
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
// Arrive on `bar` once all of this thread's earlier cp.async have landed (counted at init).
__device__ __forceinline__ void cp_async_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// A box of pool rows into shared memory, completion counted on `bar`.
__device__ __forceinline__ void load_box(uint32_t dst, const CUtensorMap *tm, uint64_t *bar, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(0), "r"(row)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// mbar_wait with a limit of its own.
__device__ __forceinline__ bool mbar_wait_for(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer() - t0 > limit_ns) return false;
    return true;
}
// Whether the phase of the given parity is over, without waiting.
__device__ __forceinline__ bool mbar_done(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float redux_max(float x) {
    float y;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}
// Barrier of `threads` threads that also tells each whether any of them brought true.
__device__ __forceinline__ bool bar_or(int id, int threads, bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.or.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(r)
        : "r"(id), "r"(threads), "r"(v ? 1 : 0)
        : "memory");
    return r != 0;
}
// Sixteen TMEM columns of this thread's lane; tmem_ld_wait before the values are used.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}
// Waits for this thread's TMEM loads; the values pass through, so that no use of them moves above it.
__device__ __forceinline__ void tmem_ld_pass(float (&v)[16]) {
    asm volatile(""
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}
template <typename... V>
__device__ __forceinline__ void tmem_ld_wait(V &...v) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    (tmem_ld_pass(v), ...);
}
__device__ __forceinline__ void tmem_zero16(uint32_t taddr) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1, %1};" ::"r"(taddr),
        "r"(0)
        : "memory");
}
// Lanes j and j + 16 receive the sum over all 32 lanes of v[j].
__device__ __forceinline__ float transpose_sum16(float (&v)[16], int lane) {
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1) {
        const bool upper = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float send = upper ? v[i] : v[i + s], keep = upper ? v[i + s] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, send, s);
        }
    }
    return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}
// The same for the maximum (sixteen redux, each waited for, took 800 clocks more).
__device__ __forceinline__ float transpose_max16(float (&v)[16], int lane) {
#pragma unroll
    for (int s = 8; s >= 1; s >>= 1) {
        const bool upper = (lane & s) != 0;
#pragma unroll
        for (int i = 0; i < s; ++i) {
            const float send = upper ? v[i] : v[i + s], keep = upper ? v[i + s] : v[i];
            v[i] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, s));
        }
    }
    return fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Four fp16 values as e4m3 codes in a word, and back. Both halves in one statement: codes that pass through 16-bit
// values of their own are widened and joined again.
__device__ __forceinline__ uint32_t e4m3_of_f16x4(uint32_t lo, uint32_t hi) {
    uint32_t c;
    asm("{\n\t.reg .b16 a, b;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 a, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f16x2 b, %2;\n\t"
        "mov.b32 %0, {a, b};\n\t}"
        : "=r"(c)
        : "r"(lo), "r"(hi));
    return c;
}
__device__ __forceinline__ void f16x4_of_e4m3(uint32_t c, uint32_t &lo, uint32_t &hi) {
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(c));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float m;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}
__device__ __forceinline__ uint32_t hsub2_u(uint32_t a, uint32_t b) {
    const __half2 r = __hsub2(*reinterpret_cast<__half2 *>(&a), *reinterpret_cast<__half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t hscale2_u(uint32_t a, float s) {
    const __half2 r = __hmul2(*reinterpret_cast<__half2 *>(&a), __float2half2_rn(s));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// ------------------------------------------------------------------ the work of a CTA
// A unit is (sequence, part, kv head, row tile), in that order, so that the tiles that read the same keys run
// side by side. A sequence of L keys is cut into parts of ceil(L / splits) keys, rounded up to whole chunks:
// the cut depends on the sequence's own length and the call's B and max_span only. A CTA starts with the unit
// of its number and takes the next one from a counter; the order changes no result. Its load warp is
// ahead of the others by up to two units, so that only the first one's page tables and keys are waited for. Where every
// unit has a CTA of its own and a tile at most kQJoin parts, the parts are a cluster: they stay in shared memory and
// each CTA joins its share of the rows.
// With a window the cut starts at the chunk of the first key that any row of the span sees.
struct QCut {
    int origin, keys, parts;  // parts of `keys` keys from `origin` to the sequence's end
};
__device__ __forceinline__ QCut qattn_cut(const QAttnArgs &a, int p0, int S) {
    QCut c;
    c.origin = a.window > 0 ? max(0, p0 - a.window + 1) / kQKeys * kQKeys : 0;
    const int n = p0 + S - c.origin, per = a.by_splits.div(n + a.splits - 1);
    c.keys = (per + kQKeys - 1) / kQKeys * kQKeys;
    c.parts = (n + c.keys - 1) / c.keys;
    return c;
}
// First partial result of span row i of sequence b (by its place in the span, which max_span bounds).
__device__ __forceinline__ size_t qattn_slot(const QAttnArgs &a, int b, int i, int hq) {
    return ((static_cast<size_t>(b) * a.c.max_span + i) * a.nq + hq) * a.splits;
}

// A row of the tile: its row of the call, its q head and its place in the span.
struct QRow {
    int row, hq, i;
};
enum { kUnitEnd, kUnitRows, kUnitRefused };
struct QUnit {
    int state, b, h, split, row0, n_rows, r0, S, p0, lo, first, last, parts;  // lo: first key that any row sees; parts: of its sequence
};
constexpr uint64_t kQUnitWaitNs = 10 * kWaitLimitNs;  // above any sum of the waits that a unit's end depends on

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(QTile<T, D, ROWS>::THREADS, QTile<T, D, ROWS>::CTAS) qcache_attn_kernel(
    const __grid_constant__ CUtensorMap pool, const __grid_constant__ QAttnArgs a) {
    typedef QTile<T, D, ROWS> Q;
    constexpr int CW = Q::CW;
    const QCacheArgs &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int grp = a.grp;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t kv_s = smem, q_s = smem + Q::STAGES * 2 * Q::TILE, p_s = q_s + Q::Q_BYTES;
    __shared__ uint64_t k_full[Q::STAGES], k_empty[Q::STAGES], v_full[Q::STAGES], v_empty[Q::STAGES], s_full[2], p_full, o_full;
    __shared__ uint32_t tmem_s;
    __shared__ __align__(16) float m_neg[ROWS], m_step[ROWS];  // -M of each row, and 2^(M before - M) where M last moved
    __shared__ int pos_s[ROWS];
    __shared__ long long to_s[ROWS];  // where a row's result begins: in `out`, or of its part in part_o
    __shared__ float top_s[4][ROWS], l_s[4][ROWS], amax_s[2][Q::WG * 4];
    __shared__ uint64_t unit_full[2], unit_empty[2], q_full;
    __shared__ QUnit unit_s[2];
    __shared__ float2 ml_s[ROWS];
    float *part_s = reinterpret_cast<float *>(smem_raw + (smem - smem_u32(smem_raw)));  // the first chunk's place, once read
    static_assert(ROWS * D * 4 <= 2 * Q::TILE, "a part's rows in a stage");
    __shared__ int joined_s, joined_rows_s;  // parts and rows that this CTA's cluster has to join
    __shared__ float kv_scale[Q::SCALES][2][kQKeys];
    const bool is_load = warp == Q::WG * 4, is_mma = warp == Q::WG * 4 + 1;
    // what needs no data goes before the wait for the kernel ahead
    if (tid == 0) {
        joined_s = 0;
        for (int i = 0; i < Q::STAGES; ++i) {
            mbar_init(&k_full[i], 33);
            mbar_init(&v_full[i], 33);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&s_full[i], 2);
            mbar_init(&unit_full[i], 1);
            mbar_init(&unit_empty[i], Q::WG * 128 + 1);
        }
        mbar_init(&q_full, Q::WG * 128);
        mbar_init(&p_full, Q::WG * 128);
        mbar_init(&o_full, 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();  // after the wait: what starts behind this kernel may read what came before it

    T *out = static_cast<T *>(a.out);
    bool ok = true;  // false once a wait gave up: the rest runs without waiting, and the status word says so
    // The k-th unit of this CTA, as the load warp leaves it.
    auto take_unit = [&](int k) {
        QUnit u;
        u.state = kUnitEnd;
        if (mbar_wait_for(&unit_full[k % 2], k / 2 & 1, kQUnitWaitNs)) {
            u = unit_s[k % 2];
            mbar_arrive(&unit_empty[k % 2]);
        } else {
            set_status(c.status, SDV_ERR_DEVICE_TIMEOUT);
        }
        return u;
    };
    auto row_of = [&](const QUnit &u, int r) {
        const int i = a.by_grp.div(u.row0 + r);
        return QRow{u.r0 + i, u.h * grp + u.row0 + r - i * grp, i};
    };
    auto chunks_of = [&](const QUnit &u) { return max(0, (u.last - u.first + kQKeys - 1) / kQKeys); };

    // The rows of a tile, shared out over the CTAs of its parts, a warp each: o = sum 2^(M_i - M) o_i / sum 2^(M_i - M) l_i
    // in the order of the parts, every part's values in flight.
    auto join_rows = [&]() {
        constexpr int V = D / 32;
        const int rank = blockIdx.x % a.splits, joined = joined_s, joined_rows = joined_rows_s;
        const uint32_t o_at = smem, ml_at = smem_u32(ml_s);
        for (int r = rank + warp * joined; r < joined_rows; r += joined * Q::WG * 4) {
            alignas(16) float v[kQJoin][V];
            const float2 ml = lane < joined ? ld_dsmem_f2(mapa_shared(ml_at + r * 8, lane)) : make_float2(kQNoRef, 0.f);
#pragma unroll
            for (int p = 0; p < kQJoin; ++p) {
#pragma unroll
                for (int d = 0; d < V; ++d) v[p][d] = 0.f;
                if (p < joined) {
                    const uint32_t src = mapa_shared(o_at + (r * D + lane * V) * 4, p);
                    if constexpr (V == 4)
                        *reinterpret_cast<float4 *>(v[p]) = ld_dsmem_f4(src);
                    else
                        *reinterpret_cast<float2 *>(v[p]) = ld_dsmem_f2(src);
                }
            }
            const float top = redux_max(ml.x), mine = ex2(ml.x - (top == kQNoRef ? 0.f : top)), l = warp_sum(mine * ml.y);
            float o[V];
#pragma unroll
            for (int d = 0; d < V; ++d) o[d] = 0.f;
#pragma unroll
            for (int p = 0; p < kQJoin; ++p) {
                const float f = __shfl_sync(0xffffffffu, mine, p);
#pragma unroll
                for (int d = 0; d < V; ++d) o[d] = fmaf(f, v[p][d], o[d]);
            }
            T *dst = out + to_s[r] + lane * V;
#pragma unroll
            for (int d = 0; d < V; ++d) dst[d] = from_f32<T>(l == 0.f ? 0.f : o[d] / l);
        }
    };

    // ---- the load warp: a chunk's K rows with both scales, then its V rows. Pages of a multiple of eight tokens come in
    // TMA boxes, a lane a box (a box past the pool is zeros); others in 16-byte pieces.
    int at[5], page[5];          // page-table slots and entries of this lane's four keys of a chunk and of its box
    uint32_t rows[4], sc_at[4];  // pool rows and scales of the keys
    int box = 0;                 // pool row of the box
    auto ask = [&](const QUnit &u, int ch) {  // keys past the last read its entry
        const int *table = c.page_table + static_cast<size_t>(u.b) * c.pages_per_seq;
        const int t0 = u.first + ch * kQKeys;
#pragma unroll
        for (int j = 0; j < 5; ++j) {
            at[j] = c.by_page.div(min(t0 + (j < 4 ? j * 32 + lane : lane % 16 * a.box_rows), u.last - 1));
            page[j] = table[at[j]];
        }
    };
    auto place = [&](const QUnit &u, int ch) {
        const int t0 = u.first + ch * kQKeys, tb = t0 + lane % 16 * a.box_rows;
        box = a.pool_rows;
        if (lane % 16 * a.box_rows < kQKeys && tb + a.box_rows > u.lo && tb < u.last && page[4] >= 0 && page[4] < c.n_pages)
            box = (page[4] * 2 * c.nkv + u.h) * c.page_size + tb - at[4] * c.page_size;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + j * 32 + lane;
            rows[j] = 0xffffffffu;
            if (t >= u.lo && t < u.last) {  // pages before the window may be gone
                if (page[j] >= 0 && page[j] < c.n_pages) {
                    const uint32_t ph = static_cast<uint32_t>(page[j]) * 2 * c.nkv + u.h, slot = t - at[j] * c.page_size;
                    rows[j] = ph * c.page_size + slot;
                    sc_at[j] = ph * c.blocks + c.by_block.div(slot);
                } else {
                    set_status(c.status, SDV_ERR_CAPACITY);
                }
            }
        }
    };
    const int v_rows = c.nkv * c.page_size;
    // the K (or V) rows of a chunk into its stage: lanes 0 to 15 bring K's boxes, 16 to 31 V's
    auto copy = [&](uint32_t dst, uint64_t *full, bool v, int box_row, const uint32_t (&row)[4]) {
        if (a.box_rows) {
            if (lane == 0) mbar_arrive_expect_tx(full, Q::TILE);
            __syncwarp();
            const int n = lane % 16;
            if (lane / 16 == (v ? 1 : 0) && n * a.box_rows < kQKeys)
                load_box(dst + n * a.box_rows * D, &pool, full, box_row + (v && box_row < a.pool_rows ? v_rows : 0));
        } else {
            constexpr int PPR = D / 16, RPI = 32 / PPR;  // pieces a row, rows a copy
            const uint8_t *codes = c.codes + lane % PPR * 16 + (v ? static_cast<size_t>(v_rows) * D : 0);
#pragma unroll
            for (int g = 0; g < 4; ++g)
                for (int j = 0; j < 32 / RPI; ++j) {
                    const int r = j * RPI + lane / PPR;
                    const uint32_t from = __shfl_sync(0xffffffffu, row[g], r);
                    const bool in = from != 0xffffffffu;
                    cp_async16(dst + line_offset(g * 32 + r, lane % PPR * 16, D),
                               in ? codes + static_cast<size_t>(from) * D : c.codes, in);
                }
            if (lane == 0) mbar_arrive(full);
        }
    };
    auto load_k = [&](int chunk) {
        const int st = chunk % Q::STAGES;
        if (chunk >= Q::STAGES && ok) ok = mbar_wait(&k_empty[st], (chunk / Q::STAGES - 1) & 1);
        copy(kv_s + st * 2 * Q::TILE, &k_full[st], false, box, rows);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool in = rows[j] != 0xffffffffu;
            const float *sc = c.scales + (in ? sc_at[j] : 0);
            cp_async4(smem_u32(&kv_scale[chunk % Q::SCALES][0][j * 32 + lane]), sc, in);
            cp_async4(smem_u32(&kv_scale[chunk % Q::SCALES][1][j * 32 + lane]), in ? sc + c.nkv * c.blocks : sc, in);
        }
        cp_async_arrive(&k_full[st]);
    };
    auto load_v = [&](int chunk, int box_row, const uint32_t (&row)[4]) {
        const int st = chunk % Q::STAGES;
        if (chunk >= Q::STAGES && ok) ok = mbar_wait(&v_empty[st], (chunk / Q::STAGES - 1) & 1);
        copy(kv_s + (st * 2 + 1) * Q::TILE, &v_full[st], true, box_row, row);
        cp_async_arrive(&v_full[st]);
    };
    if (is_load) {
        int n = blockIdx.x, chunk = 0, k = 0;
        // With more units than CTAs the long sequences' go first, so that what is left for the end is short: lane r holds
        // the sequence of rank r by length (up to 32 sequences; more of them even out by their number).
        int ranked = lane;
        const bool by_length = static_cast<int>(gridDim.x) < a.units && c.B > 1 && c.B <= 32;
        if (by_length) {
            const QSpan s = qcache_span(c, min(lane, c.B - 1));
            const int mine = lane < c.B ? (s.S ? s.p0 + s.S : 0) : -1;
            int rank = 0;
#pragma unroll
            for (int o = 0; o < 32; ++o) {
                const int other = __shfl_sync(0xffffffffu, mine, o);
                rank += other > mine || (other == mine && o < lane);
            }
#pragma unroll
            for (int o = 0; o < 32; ++o)
                if (__shfl_sync(0xffffffffu, rank, o) == lane) ranked = o;
        }
        while (n < a.units) {
            // the next unit's number is on its way while this one's keys are asked for
            int next = a.units;
            if (static_cast<int>(gridDim.x) < a.units) {
                if (lane == 0) next = gridDim.x + atomicAdd(&a.counter[0], 1);
            }
            QUnit u;
            const int nt = a.by_tiles.div(n), ns = a.by_kv.div(nt);
            int tile = n - nt * a.tiles;
            u.h = nt - ns * c.nkv;
            u.b = a.by_splits.div(ns);
            u.split = ns - u.b * a.splits;
            if (a.cluster) {  // the parts side by side
                const int t = a.by_splits.div(n), bh = a.by_tiles.div(t);
                u.split = n - t * a.splits;
                tile = t - bh * a.tiles;
                u.b = a.by_kv.div(bh);
                u.h = bh - u.b * c.nkv;
            }
            if (by_length) u.b = __shfl_sync(0xffffffffu, ranked, u.b);
            const QSpan s = qcache_span(c, u.b);
            u.r0 = s.r0, u.S = s.S, u.p0 = s.p0;
            u.row0 = tile * ROWS;
            u.n_rows = min(ROWS, s.S * grp - u.row0);
            const QCut cut = qattn_cut(a, s.p0, max(s.S, 1));
            u.state = kUnitEnd;
            if (s.S == 0) {
                if (s.code != SDV_OK && u.split == 0) {
                    u.state = kUnitRefused;
                    u.S = s.rows;
                    u.n_rows = tile;
                    if (u.h == 0 && tile == 0 && lane == 0) set_status(c.status, s.code);
                }
            } else if (u.n_rows > 0 && u.split < cut.parts) {
                u.state = kUnitRows;
            }
            if (u.state != kUnitEnd) {
                const int pos_lo = s.p0 + a.by_grp.div(u.row0), pos_hi = s.p0 + a.by_grp.div(u.row0 + max(u.n_rows, 1) - 1);
                u.parts = cut.parts;
                u.first = cut.origin + u.split * cut.keys;
                u.last = min(u.first + cut.keys, pos_hi + 1);
                u.lo = a.window > 0 ? max(0, pos_lo - a.window + 1) : 0;
                u.first = max(u.first, u.lo / kQKeys * kQKeys);
                if (k >= 2 && !mbar_wait_for(&unit_empty[k % 2], (k / 2 - 1) & 1, kQUnitWaitNs)) ok = false;
                if (lane == 0) {
                    unit_s[k % 2] = u;
                    mbar_arrive(&unit_full[k % 2]);
                }
                ++k;
                if (u.state == kUnitRows) {
                    // K a chunk ahead of V (its stages free up sooner), page-table entries a chunk ahead of K
                    const int n_chunks = chunks_of(u);
                    if (n_chunks > 0) {
                        ask(u, 0);
                        place(u, 0);
                        if (n_chunks > 1) ask(u, 1);
                        load_k(chunk);
                    }
                    for (int ch = 0; ch < n_chunks; ++ch, ++chunk) {
                        const int box_v = box;
                        const uint32_t rows_v[4] = {rows[0], rows[1], rows[2], rows[3]};
                        if (ch + 1 < n_chunks) {
                            place(u, ch + 1);
                            if (ch + 2 < n_chunks) ask(u, ch + 2);
                            load_k(chunk + 1);
                        }
                        load_v(chunk, box_v, rows_v);
                    }
                }
            }
            n = __shfl_sync(0xffffffffu, next, 0);
        }
        if (k >= 2 && !mbar_wait_for(&unit_empty[k % 2], (k / 2 - 1) & 1, kQUnitWaitNs)) ok = false;
        if (lane == 0) {
            unit_s[k % 2].state = kUnitEnd;
            mbar_arrive(&unit_full[k % 2]);
            // the last CTA to take its leave sets the counter back for the next call
            if (static_cast<int>(gridDim.x) < a.units && atomicAdd(&a.counter[1], 1) == static_cast<int>(gridDim.x) - 1) {
                a.counter[0] = 0;
                a.counter[1] = 0;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok) {  // no copy may land after this CTA's shared memory is someone else's
            for (int i = max(0, chunk - Q::STAGES); i < chunk; ++i) {
                mbar_wait(&k_full[i % Q::STAGES], (i / Q::STAGES) & 1);
                mbar_wait(&v_full[i % Q::STAGES], (i / Q::STAGES) & 1);
            }
            if (lane == 0) set_status(c.status, SDV_ERR_DEVICE_TIMEOUT);
        }
    } else if (is_mma) {
        tmem_alloc(&tmem_s, Q::COLS);
        tmem_relinquish();
    }
    if (!is_load) {
        tc_fence_before();
        named_bar_sync(6, Q::WG * 128 + 32);  // the TMEM address is there
        tc_fence_after();
    }
    const uint32_t tmem = is_load ? 0 : tmem_s;

    if (is_mma) {
        // ---- MMA issue
        if (lane == 0) {
            const uint32_t id_s = idesc_e4m3(128, Q::NQ, false), id_o = idesc_e4m3(128, Q::NP, true);
            int asked = 0, base = 0;  // chunks whose scores have been issued; chunks of the units before
            auto issue_scores = [&]() {
                const int ch = asked++, st = ch % Q::STAGES;
                const uint32_t k_s = kv_s + st * 2 * Q::TILE, d = tmem + ch % Q::NSB * Q::NQ;
                if (ok) ok = mbar_wait(&k_full[st], (ch / Q::STAGES) & 1);
                fence_async_smem();  // copies in pieces are generic writes; the tensor cores read through the async proxy
#pragma unroll
                for (int k = 0; k < D / 32; ++k)
                    umma_e4m3(d, line_desc(k_s + 32 * k, D), line_desc(q_s + 32 * k, D), id_s, k > 0);
                umma_commit(&s_full[ch % Q::NSB]);
                umma_commit(&k_empty[st]);
                mbar_arrive(&s_full[ch % Q::NSB]);  // passes on the scales' arrival, too
            };
            int queries = 0;
            for (int k = 0;; ++k) {
                const QUnit u = take_unit(k);
                if (u.state == kUnitEnd) break;
                if (u.state != kUnitRows) continue;
                const int end = base + chunks_of(u);
                if (base == end) continue;  // the softmax warps prepare no queries then, either
                if (ok) ok = mbar_wait(&q_full, queries++ & 1);
                tc_fence_after();
                issue_scores();
                for (int ch = base; ch < end; ++ch) {
                    const int st = ch % Q::STAGES;
                    const uint32_t v_s = kv_s + (st * 2 + 1) * Q::TILE;
                    // with room for two, the next scores go out while this chunk's probabilities are awaited, as soon as
                    // their keys are there (asking once only missed them by a little every time)
                    if (ok) {
                        const uint64_t since = globaltimer();
                        while (!mbar_done(&p_full, ch & 1)) {
                            if (Q::NSB == 2 && asked == ch + 1 && asked < end &&
                                mbar_done(&k_full[asked % Q::STAGES], (asked / Q::STAGES) & 1))
                                issue_scores();
                            if (globaltimer() - since > kWaitLimitNs) {
                                ok = false;
                                break;
                            }
                        }
                    }
                    tc_fence_after();
                    if (Q::NSB == 1 && asked < end) issue_scores();
                    if (ok) ok = mbar_wait(&v_full[st], (ch / Q::STAGES) & 1);
                    fence_async_smem();
#pragma unroll
                    for (int k4 = 0; k4 < kQKeys / 32; ++k4)
                        umma_e4m3(tmem + Q::O_COL, line_desc(v_s + 32 * k4 * D, D),
                                  line_desc(p_s + 32 * k4 * Q::W, Q::W, kQKeys * Q::W), id_o, (Q::GROWS && ch > base) || k4 > 0);
                    umma_commit(&o_full);
                    umma_commit(&v_empty[st]);
                    if (Q::NSB == 2 && asked == ch + 1 && asked < end) issue_scores();
                }
                base = end;
            }
            if (!ok) set_status(c.status, SDV_ERR_DEVICE_TIMEOUT);
        }
        __syncwarp();
    } else if (!is_load) {
        // ---- softmax and accumulation: a thread is key (then dim) `tid % 128` of the chunk
        const int g = warp / 4, col0 = g * CW, key = tid % 128;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        int base = 0;  // chunks of the units before
        constexpr int QN = ROWS * D / 8 / (Q::WG * 128);
        Raw8<T> raw[QN];  // this thread's share of a tile's queries
        bool asked_q = false;
        auto ask_q = [&](const QUnit &u) {
#pragma unroll
            for (int n = 0; n < QN; ++n) {
                const int e = n * Q::WG * 128 + tid, r = e / (D / 8), col = e % (D / 8) * 8;
#pragma unroll
                for (int j = 0; j < static_cast<int>(sizeof(T)) / 2; ++j) raw[n].u[j] = make_uint4(0, 0, 0, 0);
                if (r < u.n_rows) {
                    const QRow w = row_of(u, r);
                    const T *src = static_cast<const T *>(a.q) + w.row * a.q_stride + w.hq * D + col;
                    raw[n] = a.q_vec ? load_raw8<T, true>(src) : load_raw8<T, false>(src);
                }
            }
        };
        for (int unit_no = 0;; ++unit_no) {
        const QUnit u = take_unit(unit_no);
        if (u.state == kUnitEnd) break;
        if (u.state == kUnitRefused) {  // NaN rather than stale memory, this kv head's q heads shared over the tiles
            for (int r = u.n_rows; r < u.S; r += a.tiles)
                for (int d = tid; d < grp * D; d += Q::WG * 128)
                    out[(u.r0 + r) * a.out_stride + u.h * grp * D + d] = from_f32<T>(NAN);
            continue;
        }
        const int n_rows = u.n_rows, n_chunks = chunks_of(u), first = u.first, last = u.last;
        const int pos_lo = u.p0 + a.by_grp.div(u.row0), pos_hi = u.p0 + a.by_grp.div(u.row0 + n_rows - 1);
        // the queries' planes [plane x ROWS + row][D], eight values a thread at a time; the scores that read the last
        // unit's have been waited for
        named_bar_sync(5, Q::WG * 128);  // nobody reads the last unit's rows any more
        if (tid < ROWS) {
            const QRow w = row_of(u, min(tid, n_rows - 1));
            m_neg[tid] = -kQNoRef;
            pos_s[tid] = tid < n_rows ? u.p0 + w.i : -1;
            to_s[tid] = u.parts == 1 || a.cluster ? w.row * a.out_stride + w.hq * D
                                : static_cast<long long>(qattn_slot(a, u.b, w.i, w.hq) + u.split) * D;
        }
        if (!asked_q) ask_q(u);
        float x[QN][8], amax = 0.f;
#pragma unroll
        for (int n = 0; n < QN; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                x[n][j] = raw[n].at(j);
                if (fabsf(x[n][j]) < INFINITY)
                    amax = fmaxf(amax, fabsf(x[n][j]));
                else
                    x[n][j] = NAN;  // spoils its own row
            }
        amax = redux_max(amax);
        if (lane == 0) amax_s[unit_no & 1][warp] = amax;
        named_bar_sync(7, Q::WG * 128);
#pragma unroll
        for (int w = 0; w < Q::WG * 4; ++w) amax = fmaxf(amax, amax_s[unit_no & 1][w]);
        // 2^e with amax 2^e in [128, 256); bounded so that both powers stay normal
        const int ex = amax > 0.f ? min(max(7 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), -120), 120) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
        const float unit = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
#pragma unroll
        for (int n = 0; n < QN; ++n) {
            const int e = n * Q::WG * 128 + tid, r = e / (D / 8), col = e % (D / 8) * 8;
            float rest[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) rest[j] = x[n][j] * up;
#pragma unroll
            for (int p = 0; p < Q::PQ; ++p) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    w[j] = e4m3x2(rest[2 * j], rest[2 * j + 1]);
                    const float2 f = e4m3x2_f32(w[j]);
                    rest[2 * j] = (rest[2 * j] - f.x) * 32.f;
                    rest[2 * j + 1] = (rest[2 * j + 1] - f.y) * 32.f;
                }
                const uint32_t dst = q_s + line_offset(p * ROWS + r, col, D);
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(w[0] | w[1] << 16),
                             "r"(w[2] | w[3] << 16)
                             : "memory");
            }
        }
        fence_async_smem();
        if (n_chunks > 0) {
            tc_fence_before();
            mbar_arrive(&q_full);
        }
        float acc[CW], l[CW];
#pragma unroll
        for (int r = 0; r < CW; ++r) acc[r] = l[r] = 0.f;
        // adds the products since the last time, up to that of chunk ch, planes joined
        auto collect = [&](int ch) {
            if (ok) ok = mbar_wait(&o_full, (base + ch) & 1);
            tc_fence_after();
            float v[3][16];
#pragma unroll
            for (int p = 0; p < 3; ++p) tmem_ld16(tmem + lanes + Q::O_COL + p * ROWS + col0, v[p]);
            tmem_ld_wait(v[0], v[1], v[2]);
#pragma unroll
            for (int r = 0; r < 16; r += 2) {
                float2 o = make_float2(acc[r], acc[r + 1]);
#pragma unroll
                for (int p = 0; p < 3; ++p) {
                    const float u = p == 0 ? 0x1p-6f : p == 1 ? 0x1p-12f : 0x1p-17f;
                    o = __ffma2_rn(make_float2(v[p][r], v[p][r + 1]), make_float2(u, u), o);
                }
                acc[r] = o.x, acc[r + 1] = o.y;
            }
        };
        for (int ch = 0; ch < n_chunks; ++ch) {
            const int t0 = first + ch * kQKeys, t = t0 + key;
            const bool masked = t0 + kQKeys - 1 > pos_lo || (a.window > 0 && t0 <= pos_hi - a.window);
            const int gc = base + ch;
            if (ok) ok = mbar_wait(&s_full[gc % Q::NSB], (gc / Q::NSB) & 1);
            tc_fence_after();
            const uint32_t s_col = tmem + lanes + gc % Q::NSB * Q::NQ + col0;
            const float ks = kv_scale[gc % Q::SCALES][0][key] * unit;
            const float vs = t >= u.lo && t < last ? kv_scale[gc % Q::SCALES][1][key] : 1.f, lv = __log2f(vs), lv_ref = fmaxf(lv, kQLeast);
            // sixteen rows' scores of this key in log2 units, -inf where a row does not see it
            float sc[16];
            {
                float v[Q::PQ - 1][16];
                tmem_ld16(s_col, sc);
#pragma unroll
                for (int p = 1; p < Q::PQ; ++p) tmem_ld16(s_col + p * ROWS, v[p - 1]);
                if constexpr (Q::PQ == 2)
                    tmem_ld_wait(sc, v[0]);
                else
                    tmem_ld_wait(sc, v[0], v[1]);
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    float2 z = make_float2(sc[r], sc[r + 1]);
#pragma unroll
                    for (int p = 1; p < Q::PQ; ++p) {
                        const float u = p == 1 ? 0x1p-5f : 0x1p-10f;
                        z = __ffma2_rn(make_float2(v[p - 1][r], v[p - 1][r + 1]), make_float2(u, u), z);
                    }
                    z = __fmul2_rn(z, make_float2(ks, ks));
                    sc[r] = z.x, sc[r + 1] = z.y;
                }
            }
            if (masked) {
#pragma unroll
                for (int r = 0; r < 16; ++r) {
                    const int pos = pos_s[col0 + r];
                    if (t > pos || (a.window > 0 && t <= pos - a.window)) sc[r] = -INFINITY;
                }
            }
            // does a row's w leave the range that its reference covers, w > M + 1?
            float over = -INFINITY;
#pragma unroll
            for (int r = 0; r < 16; r += 4) {
                const float4 m = *reinterpret_cast<const float4 *>(&m_neg[col0 + r]);
                const float2 d = __fadd2_rn(make_float2(sc[r], sc[r + 1]), make_float2(m.x, m.y));
                const float2 e = __fadd2_rn(make_float2(sc[r + 2], sc[r + 3]), make_float2(m.z, m.w));
                over = max3(max3(over, d.x, d.y), e.x, e.y);
            }
            if (!Q::GROWS && ch > 0) collect(ch - 1);
            if (ch == 0 || bar_or(1 + g, 128, over + lv_ref > 1.f)) {  // the first chunk's always do
                float v[16];
#pragma unroll
                for (int r = 0; r < 16; ++r) v[r] = sc[r] + lv_ref;
                const float top = transpose_max16(v, lane);
                if (lane < 16) top_s[warp % 4][col0 + lane] = top;
                named_bar_sync(1 + g, 128);
                if (key < CW) {
                    const int k = col0 + key;
                    const float now = fmaxf(fmaxf(top_s[0][k], top_s[1][k]), fmaxf(top_s[2][k], top_s[3][k])), was = -m_neg[k];
                    const bool moves = now > was + 1.f;
                    m_step[k] = moves ? ex2(was - now) : 1.f;
                    if (moves) m_neg[k] = -now;
                }
                named_bar_sync(1 + g, 128);
                if (ch > 0) {
                    if constexpr (Q::GROWS) {
                        collect(ch - 1);
#pragma unroll
                        for (int p = 0; p < 3; ++p) tmem_zero16(tmem + lanes + Q::O_COL + p * ROWS + col0);
                        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    }
#pragma unroll
                    for (int r = 0; r < 16; r += 4) {
                        const float4 f = *reinterpret_cast<const float4 *>(&m_step[col0 + r]);
                        acc[r] *= f.x, acc[r + 1] *= f.y, acc[r + 2] *= f.z, acc[r + 3] *= f.w;
                        l[r] *= f.x, l[r + 1] *= f.y, l[r + 2] *= f.z, l[r + 3] *= f.w;
                    }
                }
            }
            // x = 64 p as planes; a line of P holds this key's values of every row and plane. l takes x / (64 vs); keys
            // whose scale is 0 or so small that x may vanish beside it (2^-30) send their warp to the exponential.
            const float lv6 = lv + 6.f;
            const bool small = __any_sync(0xffffffffu, !(vs >= 0x1p-30f));
            const float to_l = small ? 0.f : __fdividef(0x1p-6f, vs);
            if (small) {
#pragma unroll
                for (int r = 0; r < 16; ++r) l[r] += ex2(sc[r] + m_neg[col0 + r]);
            }
            uint32_t w[Q::PP][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 m = *reinterpret_cast<const float4 *>(&m_neg[col0 + 4 * j]);
                uint32_t x[2];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const int r = 4 * j + 2 * i;
                    // (s - M) + log2 vs: the first difference is small where it matters
                    const float2 d = __fadd2_rn(make_float2(sc[r], sc[r + 1]), i ? make_float2(m.z, m.w) : make_float2(m.x, m.y));
                    const float2 e = __fadd2_rn(d, make_float2(lv6, lv6)), x2 = make_float2(ex2(e.x), ex2(e.y));
                    const float2 n = __ffma2_rn(x2, make_float2(to_l, to_l), make_float2(l[r], l[r + 1]));
                    l[r] = n.x, l[r + 1] = n.y;
                    x[i] = f16x2(x2.x, x2.y);
                }
#pragma unroll
                for (int p = 0; p < Q::PP; ++p) {
                    w[p][j] = e4m3_of_f16x4(x[0], x[1]);
                    if (p + 1 < Q::PP) {
                        uint32_t lo, hi;
                        f16x4_of_e4m3(w[p][j], lo, hi);
                        x[0] = hscale2_u(hsub2_u(x[0], lo), p == 0 ? 64.f : 32.f);
                        x[1] = hscale2_u(hsub2_u(x[1], hi), p == 0 ? 64.f : 32.f);
                    }
                }
            }
            if (Q::GROWS && ch > 0 && ok) ok = mbar_wait(&o_full, (gc - 1) & 1);  // the last product is done with P
#pragma unroll
            for (int p = 0; p < Q::PP; ++p)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 p_s + (p * ROWS + col0) / Q::W * (kQKeys * Q::W) +
                                 line_offset(key, (p * ROWS + col0) % Q::W, Q::W)),
                             "r"(w[p][0]), "r"(w[p][1]), "r"(w[p][2]), "r"(w[p][3])
                             : "memory");
            if (t0 + kQKeys > last) {  // slots behind the sequence may hold anything, and 0 times a NaN is none
                const int st = gc % Q::STAGES;
                if (ok) ok = mbar_wait(&v_full[st], (gc / Q::STAGES) & 1);
                if (t >= last)
                    for (int j = g; j < D / 16; j += Q::WG)
                        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(kv_s + (st * 2 + 1) * Q::TILE + key * D + j * 16),
                                     "r"(0)
                                     : "memory");
            }
            fence_async_smem();
            tc_fence_before();
            mbar_arrive(&p_full);
        }
        // the next unit's queries are asked for before this one's last product is in
        asked_q = false;
        if (mbar_done(&unit_full[(unit_no + 1) % 2], (unit_no + 1) / 2 & 1)) {
            const QUnit &next = unit_s[(unit_no + 1) % 2];
            if (next.state == kUnitRows) {
                ask_q(next);
                asked_q = true;
            }
        }
        if (n_chunks > 0) collect(n_chunks - 1);
        if (!ok && lane == 0) set_status(c.status, SDV_ERR_DEVICE_TIMEOUT);
        // ---- sums over the keys, and the rows out
        const float mine = transpose_sum16(l, lane);
        if (lane < 16) l_s[warp % 4][col0 + lane] = mine;
        named_bar_sync(1 + g, 128);
        const int rows = min(CW, n_rows - col0);
        if (key < D) {
            if (u.parts == 1) {
#pragma unroll
                for (int r = 0; r < CW; ++r) {
                    const int k = col0 + r;
                    const float total = (l_s[0][k] + l_s[1][k]) + (l_s[2][k] + l_s[3][k]);
                    if (r < rows) out[to_s[k] + key] = from_f32<T>(total == 0.f ? 0.f : __fdividef(acc[r], total));
                }
            } else if (a.cluster) {
#pragma unroll
                for (int r = 0; r < CW; ++r) part_s[(col0 + r) * D + key] = acc[r];
            } else {
#pragma unroll
                for (int r = 0; r < CW; ++r)
                    if (r < rows) a.part_o[to_s[col0 + r] + key] = acc[r];
            }
        }
        if (u.parts > 1 && key < rows) {
            const int k = col0 + key;
            const float2 ml = make_float2(-m_neg[k], (l_s[0][k] + l_s[1][k]) + (l_s[2][k] + l_s[3][k]));
            if (a.cluster)
                ml_s[k] = ml;
            else
                a.part_ml[to_s[k] / D] = ml;
        }
        if (u.parts > 1 && tid == 0) joined_s = u.parts, joined_rows_s = n_rows;
        base += n_chunks;
        }
        tc_fence_before();
    }
    if (a.cluster) {
        __syncwarp();
        cluster_sync();
        if (!is_load && !is_mma && joined_s) join_rows();
        __syncwarp();
        cluster_arrive();
    } else {
        __syncthreads();
    }
    if (is_mma) tmem_dealloc(tmem, Q::COLS);
    if (a.cluster) cluster_wait();  // nobody leaves while its part may be read
}

constexpr int kQMergeThreads = 128;

// Where no cluster does: NW warps join the parts of one (row, q head), every NW-th part a warp, the warps in order.
// NW = 1 up to eight parts (the loads that a warp has under way), else 4.
// Grid (span row x head in groups of 4 / NW, sequence).
template <typename T, int D, int NW>
__global__ void __launch_bounds__(kQMergeThreads) qcache_merge_kernel(const __grid_constant__ QAttnArgs a) {
    constexpr int V = D / 32;
    const int warp = threadIdx.x / 32 % NW, lane = threadIdx.x % 32;
    const int b = blockIdx.y, item = blockIdx.x * (kQMergeThreads / 32 / NW) + threadIdx.x / 32 / NW;
    const int i = a.by_nq.div(item), hq = item - i * a.nq;
    // the spans are no results of the attention before it, which started after whatever wrote them
    const QSpan s = qcache_span(a.c, b);
    const int parts = qattn_cut(a, s.p0, max(s.S, 1)).parts;
    __shared__ float o_s[NW][D], l_s;
    pdl_wait();  // in every CTA: this kernel's end stands for the attention's, too
    pdl_trigger();
    if (i >= s.S || parts == 1) return;
    const size_t slot = qattn_slot(a, b, i, hq);
    // parts without a key of this row hold M = kQNoRef, l = 0, o = 0
    float m = kQNoRef;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.part_ml[slot + p].x);
    m = redux_max(m);
    if (m == kQNoRef) m = 0.f;  // none of them: every weight 0
    float o[V], l = 0.f;
#pragma unroll
    for (int d = 0; d < V; ++d) o[d] = 0.f;
    // 32 parts (8 for one warp) at a time: a lane weighs one, the warp's eight are read at once
    constexpr int P = 8 * NW;
    for (int p0 = 0; p0 < parts; p0 += P) {
        const float2 ml = lane < P && p0 + lane < parts ? a.part_ml[slot + p0 + lane] : make_float2(kQNoRef, 0.f);
        const float mine = ex2(ml.x - m);
        float v[8][V];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = p0 + warp + j * NW;
#pragma unroll
            for (int d = 0; d < V; ++d) v[j][d] = 0.f;
            if (p < parts) {
                const float *src = a.part_o + (slot + p) * D + lane * V;
                if constexpr (V == 4)
                    *reinterpret_cast<float4 *>(v[j]) = *reinterpret_cast<const float4 *>(src);
                else
                    *reinterpret_cast<float2 *>(v[j]) = *reinterpret_cast<const float2 *>(src);
            }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float f = __shfl_sync(0xffffffffu, mine, warp + j * NW);
#pragma unroll
            for (int d = 0; d < V; ++d) o[d] = fmaf(f, v[j][d], o[d]);
        }
        if (warp == 0) l += warp_sum(mine * ml.y);
    }
    T *dst = static_cast<T *>(a.out) + (s.r0 + i) * a.out_stride + hq * D;
    if constexpr (NW == 1) {
#pragma unroll
        for (int d = 0; d < V; ++d) dst[lane * V + d] = from_f32<T>(l == 0.f ? 0.f : o[d] / l);
    } else {
#pragma unroll
        for (int d = 0; d < V; ++d) o_s[warp][lane * V + d] = o[d];
        if (threadIdx.x == 0) l_s = l;
        __syncthreads();
        const int d = threadIdx.x;
        if (d < D) {
            const float num = (o_s[0][d] + o_s[1][d]) + (o_s[2][d] + o_s[3][d]);
            dst[d] = from_f32<T>(l_s == 0.f ? 0.f : num / l_s);
        }
    }
}

}  // namespace sdv
