// Attention over the 8-bit cache on the fp8 tensor cores.
//
// For one kv head, ROWS query rows (span row x head of the group) against 128 keys at a time:
//     S^T [128 keys x rows] = K . Q^T          (A = the K codes as they lie in the cache, B = Q)
//     O^T [dims x rows]     = V^T . P^T        (A = the V codes read along the other axis, B = P)
// so K and V enter the tensor cores as the bytes they are, a key (then a dim) to a TMEM lane, and the
// few query rows of a verify step are the narrow operand: an MMA of 128 lanes costs 45 clocks for any
// width up to 64 (measured), 365 for the eight of a chunk, against the 1,370 that the chunk's 32 KB take
// at this SM's share of HBM.
//
// The 16-bit operand of each product is split into e4m3 planes laid side by side along the width:
//   q = 2^-e (q0 + 2^-5 q1 + 2^-10 q2), e from the tile's largest |q|: two planes hold a bf16's eight
//       bits exactly, three an fp16's eleven (what lies 2^-20 below the largest rounds away). Tiles of 64
//       rows (bf16) add the two planes' products in the accumulator instead, with q1 at q0's own scale:
//       half the columns, exact to 2^-18 of the largest;
//   p = x0 + 2^-6 x1 + 2^-11 x2, x = 64 p in (0, 128]: p is rounded to fp16's eleven bits and the planes hold
//       them down to 2^-26 (two planes lost the tail under one large p: 2% off at p = 2^-16).
// The planes' products are otherwise added in fp32 afterwards.
//
// A key's V scale is not applied to V: it joins the exponent. With s_t the score in log2 units and
// w_t = s_t + log2 vs_t, x_t = 2^(w_t - M) multiplies the bare codes, M being a row's running maximum of w,
// and the sum l takes 2^(s_t - M); o / l is the result, precise relative to the largest contribution
// however far the scales lie apart. M follows the maximum only when that has grown by more than one
// (hence x up to 2 . 64), so the accumulators are rarely rescaled.
#pragma once

#include "qcache.cuh"

namespace sdv {

struct QAttnArgs {
    QCacheArgs c;
    const void *q;
    void *out;
    long long q_stride, out_stride;  // elements between rows
    int nq, window;                  // window: positions a row sees, its own the last (0: all)
    int splits;                      // parts a sequence's keys are cut into at most
    int tiles;                       // row tiles of a span of max_span rows
    int grp;                         // q heads a kv head
    int q_vec;                       // q rows are 16-byte aligned
    FastDiv by_tiles, by_splits, by_grp, by_nq;
    float scale_log2;                // log2(e) / sqrt(D)
    float *part_o;                   // [sequence][span row][q head][splits][D]
    int box_rows;                    // pool rows of a TMA box; 0: pages that no box fits, copied in 16-byte pieces
    int pool_rows;                   // rows of the layer's pool: a box there reads zeros
    float2 *part_ml;                 // [sequence][span row][q head][splits]: (M, l)
};

constexpr int kQKeys = 128;     // keys of a chunk
constexpr int kQStages = 2;     // chunks in shared memory
constexpr float kQNoRef = -1e30f;  // a row's M before it has seen a key: below any w, and w - M is no NaN
template <typename T, int D_, int ROWS_>
struct QTile {
    static constexpr int D = D_, ROWS = ROWS_;
    static constexpr int PQ = sizeof(T) == 2 && !__is_same(T, __half) ? 2 : 3;  // planes of q
    static constexpr int PP = 3;                                                  // planes of p
    static constexpr bool FOLD = ROWS == 64;                                      // q planes share S's columns
    static constexpr int WG = ROWS == 16 ? 1 : 2;                                 // softmax warpgroups
    static constexpr int CW = ROWS / WG;                                          // columns of one
    static constexpr int NQ = PQ * ROWS, NP = PP * ROWS;                          // widths of the two products
    static constexpr int W = ROWS == 32 ? 128 : 64;  // bytes of a key's P line: every plane, or (64 rows) one
    static constexpr int P_LINES = (NP + W - 1) / W;
    static constexpr int TILE = kQKeys * D;                                       // bytes of a K or V chunk
    static constexpr int Q_BYTES = (NQ * D + 1023) / 1024 * 1024, P_BYTES = kQKeys * W * P_LINES;
    static constexpr int SMEM = 1024 + kQStages * 2 * TILE + Q_BYTES + P_BYTES;
    static constexpr int NS = FOLD ? ROWS : NQ;                                   // columns of S^T
    static constexpr int NSB = 2 * NS + NP <= 256 ? 2 : 1;                        // S^T of the next chunk beside this one's
    static constexpr int O_COL = (NSB * NS + 31) / 32 * 32;                       // TMEM column of O^T
    static constexpr int COLS = O_COL + NP <= 128 ? 128 : 256;
    static constexpr int THREADS = WG * 128 + 64;  // softmax warps, the load warp, the MMA warp
    static_assert(ROWS == 16 || ROWS == 32 || (ROWS == 64 && PQ == 2), "tile rows");
    static_assert(O_COL + NP <= COLS, "TMEM columns");
    static_assert(NQ % 16 == 0 && NP % 16 == 0, "MMA widths");
    static_assert(2 * (SMEM + 6144 + 1024) <= 228 * 1024, "two CTAs per SM");
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
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&h);
}
// Two fp16 values as e4m3 codes, and back.
__device__ __forceinline__ uint32_t e4m3_of_f16x2(uint32_t h) {
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(c) : "r"(h));
    return c;
}
__device__ __forceinline__ uint32_t f16x2_of_e4m3(uint32_t c) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
    return h;
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
// Grid ((kv head, row tile), split, sequence): the tiles that read the same keys run side by side. A
// sequence of L keys is cut into parts of ceil(L / splits) keys, rounded up to whole chunks: the cut
// depends on the sequence's own length and the call's B and max_span only.
__device__ __forceinline__ int qattn_part_keys(const QAttnArgs &a, int L) {
    const int per = a.by_splits.div(L + a.splits - 1);
    return (per + kQKeys - 1) / kQKeys * kQKeys;
}
// First partial result of span row i of sequence b (by its place in the span, which max_span bounds).
__device__ __forceinline__ size_t qattn_slot(const QAttnArgs &a, int b, int i, int hq) {
    return ((static_cast<size_t>(b) * a.c.max_span + i) * a.nq + hq) * a.splits;
}

// A row of the tile: its row of the call, its q head and its place in the span.
struct QRow {
    int row, hq, i;
};

template <typename T, int D, int ROWS>
__global__ void __launch_bounds__(QTile<T, D, ROWS>::THREADS, 2) qcache_attn_kernel(
    const __grid_constant__ CUtensorMap pool, const __grid_constant__ QAttnArgs a) {
    typedef QTile<T, D, ROWS> Q;
    constexpr int CW = Q::CW;
    const QCacheArgs &c = a.c;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int grp = a.grp, split = blockIdx.y, b = blockIdx.z;
    const int h = a.by_tiles.div(blockIdx.x), tile = blockIdx.x - h * a.tiles;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const uint32_t kv_s = smem, q_s = smem + kQStages * 2 * Q::TILE, p_s = q_s + Q::Q_BYTES;
    __shared__ uint64_t k_full[kQStages], k_empty[kQStages], v_full[kQStages], v_empty[kQStages], s_full[2], p_full, o_full;
    __shared__ uint32_t tmem_s;
    __shared__ __align__(16) float m_neg[ROWS], m_step[ROWS];  // -M of each row, and 2^(M before - M) where M last moved
    __shared__ uint32_t m_key[ROWS];
    __shared__ int pos_s[ROWS];
    __shared__ float l_s[4][ROWS], amax_s[Q::WG * 4];
    __shared__ float kv_scale[4][2][kQKeys];  // four chunks deep: softmax may still read the one two back
    const bool is_load = warp == Q::WG * 4, is_mma = warp == Q::WG * 4 + 1;
    // what needs no data goes before the wait for the kernel ahead
    if (tid == 0) {
        for (int i = 0; i < kQStages; ++i) {
            mbar_init(&k_full[i], 33);
            mbar_init(&v_full[i], 33);
            mbar_init(&k_empty[i], 1);
            mbar_init(&v_empty[i], 1);
            mbar_init(&s_full[i], 2);
        }
        mbar_init(&p_full, Q::WG * 128);
        mbar_init(&o_full, 1);
        fence_mbar_init();
    }
    if (tid < ROWS) {
        m_neg[tid] = -kQNoRef;
        m_key[tid] = 0;
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();  // after the wait: what starts behind this kernel may read what came before it

    const QSpan s = qcache_span(c, b);
    T *out = static_cast<T *>(a.out);
    if (s.S == 0) {
        if (split == 0 && s.code != SDV_OK) {
            if (blockIdx.x == 0 && tid == 0) set_status(c.status, s.code);
            // refused: NaN rather than stale memory, this kv head's q heads shared over the tiles
            for (int r = tile; r < s.rows; r += a.tiles)
                for (int d = tid; d < grp * D; d += Q::THREADS)
                    out[(s.r0 + r) * a.out_stride + h * grp * D + d] = from_f32<T>(NAN);
        }
        return;
    }
    const int row0 = tile * ROWS, n_rows = min(ROWS, s.S * grp - row0);  // flattened (span row, head) rows
    const int L = s.p0 + s.S, keys = qattn_part_keys(a, L);
    if (n_rows <= 0 || split * static_cast<long long>(keys) >= L) return;
    const bool whole = keys >= L;  // the sequence has one part
    auto row_of = [&](int r) {
        const int i = a.by_grp.div(row0 + r);
        return QRow{s.r0 + i, h * grp + row0 + r - i * grp, i};
    };
    const int pos_lo = s.p0 + a.by_grp.div(row0), pos_hi = s.p0 + a.by_grp.div(row0 + n_rows - 1);
    int first = split * keys;
    const int last = min(first + keys, pos_hi + 1);
    if (a.window > 0) first = max(first, max(0, pos_lo - a.window + 1) / kQKeys * kQKeys);
    const int n_chunks = max(0, (last - first + kQKeys - 1) / kQKeys);

    bool ok = true;  // false once a wait gave up: the rest runs without waiting, and the status word says so
    // ---- the load warp: a chunk's K rows with both scales, then its V rows. Pages of a multiple of eight tokens come in
    // TMA boxes, a lane a box (a box past the pool is zeros); others in 16-byte pieces.
    const int *table = c.page_table + static_cast<size_t>(b) * c.pages_per_seq;
    uint32_t rows[4], sc_at[4];  // pool rows and scales of this lane's four keys of a chunk
    int box = 0;                 // pool row of its box
    auto look = [&](int ch) {
        // the five page-table entries first, so that their latencies pass together; keys past the last read its entry
        const int t0 = first + ch * kQKeys, tb = t0 + lane % 16 * a.box_rows;
        const bool has_box = lane % 16 * a.box_rows < kQKeys && tb < last;
        int at[5], page[5];
#pragma unroll
        for (int j = 0; j < 5; ++j) {
            at[j] = c.by_page.div(min(j < 4 ? t0 + j * 32 + lane : tb, last - 1));
            page[j] = table[at[j]];
        }
        box = a.pool_rows;
        if (has_box && page[4] >= 0 && page[4] < c.n_pages) box = (page[4] * 2 * c.nkv + h) * c.page_size + tb - at[4] * c.page_size;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int t = t0 + j * 32 + lane;
            rows[j] = 0xffffffffu;
            if (t < last) {
                if (page[j] >= 0 && page[j] < c.n_pages) {
                    const uint32_t ph = static_cast<uint32_t>(page[j]) * 2 * c.nkv + h, slot = t - at[j] * c.page_size;
                    rows[j] = ph * c.page_size + slot;
                    sc_at[j] = ph * c.blocks + c.by_block.div(slot);
                } else {
                    set_status(c.status, SDV_ERR_CAPACITY);
                }
            }
        }
    };
    const int v_rows = c.nkv * c.page_size;
    // lanes 0 to 15 bring K's boxes, 16 to 31 V's
    auto load_half = [&](int ch, bool v) {
        const int st = ch % kQStages;
        const uint32_t dst = kv_s + (st * 2 + (v ? 1 : 0)) * Q::TILE;
        uint64_t *full = v ? &v_full[st] : &k_full[st];
        if (ch >= kQStages && ok) ok = mbar_wait(v ? &v_empty[st] : &k_empty[st], (ch / kQStages - 1) & 1);
        if (a.box_rows) {
            if (lane == 0) mbar_arrive_expect_tx(full, Q::TILE);
            __syncwarp();
            const int n = lane % 16;
            if (lane / 16 == (v ? 1 : 0) && n * a.box_rows < kQKeys)
                load_box(dst + n * a.box_rows * D, &pool, full, box + (v && box < a.pool_rows ? v_rows : 0));
        } else {
            constexpr int PPR = D / 16, RPI = 32 / PPR;  // pieces a row, rows a copy
            const uint8_t *codes = c.codes + lane % PPR * 16 + (v ? static_cast<size_t>(v_rows) * D : 0);
#pragma unroll
            for (int g = 0; g < 4; ++g)
                for (int j = 0; j < 32 / RPI; ++j) {
                    const int r = j * RPI + lane / PPR;
                    const uint32_t row = __shfl_sync(0xffffffffu, rows[g], r);
                    const bool in = row != 0xffffffffu;
                    cp_async16(dst + line_offset(g * 32 + r, lane % PPR * 16, D),
                               in ? codes + static_cast<size_t>(row) * D : c.codes, in);
                }
            if (lane == 0) mbar_arrive(full);
        }
        if (!v) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const bool in = rows[j] != 0xffffffffu;
                const float *sc = c.scales + (in ? sc_at[j] : 0);
                cp_async4(smem_u32(&kv_scale[ch % 4][0][j * 32 + lane]), sc, in);
                cp_async4(smem_u32(&kv_scale[ch % 4][1][j * 32 + lane]), in ? sc + c.nkv * c.blocks : sc, in);
            }
        }
        cp_async_arrive(full);
    };
    if (is_load) {
        // on its own from here on: the first chunks are on their way while the queries are prepared
        for (int ch = 0; ch < n_chunks; ++ch) {
            look(ch);
            load_half(ch, false);
            load_half(ch, true);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok && lane == 0) set_status(c.status, SDV_ERR_DEVICE_TIMEOUT);
    } else if (is_mma) {
        tmem_alloc(&tmem_s, Q::COLS);
        tmem_relinquish();
        for (int r = lane; r < ROWS; r += 32) pos_s[r] = r < n_rows ? s.p0 + row_of(r).i : -1;
    }
    // Q: the tile's rows as e4m3 planes [plane x ROWS + row][D], eight values a thread at a time
    float q_unit = 1.f;  // 2^-e: what the planes' products are multiplied by
    constexpr int QN = ROWS * D / 8 / (Q::WG * 128);
    if (!is_load && !is_mma) {
        float x[QN][8], amax = 0.f;
#pragma unroll
        for (int n = 0; n < QN; ++n) {
            const int e = n * Q::WG * 128 + tid, r = e / (D / 8), col = e % (D / 8) * 8;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[n][j] = 0.f;
            if (r < n_rows) {
                const QRow w = row_of(r);
                const T *src = static_cast<const T *>(a.q) + w.row * a.q_stride + w.hq * D + col;
                if (a.q_vec)
                    load8<T, true>(src, x[n]);
                else
                    load8<T, false>(src, x[n]);
            }
        }
#pragma unroll
        for (int n = 0; n < QN; ++n)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (fabsf(x[n][j]) < INFINITY)
                    amax = fmaxf(amax, fabsf(x[n][j]));
                else
                    x[n][j] = NAN;  // spoils its own row
            }
        amax = redux_max(amax);
        if (lane == 0) amax_s[warp] = amax;
        named_bar_sync(7, Q::WG * 128);
#pragma unroll
        for (int w = 0; w < Q::WG * 4; ++w) amax = fmaxf(amax, amax_s[w]);
        // 2^e with amax 2^e in [128, 256); bounded so that both powers stay normal
        const int ex = amax > 0.f ? min(max(7 - (static_cast<int>(__float_as_uint(amax) >> 23) - 127), -120), 120) : 0;
        const float up = __uint_as_float(static_cast<uint32_t>(ex + 127) << 23);
        q_unit = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
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
                    rest[2 * j] = (rest[2 * j] - f.x) * (Q::FOLD ? 1.f : 32.f);
                    rest[2 * j + 1] = (rest[2 * j + 1] - f.y) * (Q::FOLD ? 1.f : 32.f);
                }
                const uint32_t dst = q_s + line_offset(p * ROWS + r, col, D);
                asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(dst), "r"(w[0] | w[1] << 16),
                             "r"(w[2] | w[3] << 16)
                             : "memory");
            }
        }
        fence_async_smem();
    }
    tc_fence_before();
    if (!is_load) named_bar_sync(6, Q::WG * 128 + 32);  // the queries and the TMEM address are there
    tc_fence_after();
    const uint32_t tmem = is_load ? 0 : tmem_s;

    if (is_mma) {
        // ---- MMA issue
        if (lane == 0) {
            const uint32_t id_s = idesc_e4m3(128, Q::NS, false), id_o = idesc_e4m3(128, Q::NP, true);
            int asked = 0;  // chunks whose scores have been issued
            auto issue_scores = [&]() {
                const int ch = asked++, st = ch % kQStages;
                const uint32_t k_s = kv_s + st * 2 * Q::TILE, d = tmem + ch % Q::NSB * Q::NS;
                if (ok) ok = mbar_wait(&k_full[st], (ch / kQStages) & 1);
                fence_async_smem();  // copies in pieces are generic writes; the tensor cores read through the async proxy
#pragma unroll
                for (int k = 0; k < D / 32 * (Q::FOLD ? Q::PQ : 1); ++k)
                    umma_e4m3(d, line_desc(k_s + k % (D / 32) * 32, D),
                              line_desc(q_s + k / (D / 32) * ROWS * D + k % (D / 32) * 32, D), id_s, k > 0);
                umma_commit(&s_full[ch % Q::NSB]);
                umma_commit(&k_empty[st]);
                mbar_arrive(&s_full[ch % Q::NSB]);  // passes on the scales' arrival, too
            };
            if (n_chunks > 0) issue_scores();
            for (int ch = 0; ch < n_chunks; ++ch) {
                const int st = ch % kQStages;
                const uint32_t v_s = kv_s + (st * 2 + 1) * Q::TILE;
                // with room for two, the next scores go out before this chunk's probabilities are there if its keys are
                if (Q::NSB == 2 && asked < n_chunks && mbar_done(&k_full[asked % kQStages], (asked / kQStages) & 1))
                    issue_scores();
                if (ok) ok = mbar_wait(&p_full, ch & 1);
                tc_fence_after();
                if (Q::NSB == 1 && asked < n_chunks) issue_scores();
                if (ok) ok = mbar_wait(&v_full[st], (ch / kQStages) & 1);
                fence_async_smem();
#pragma unroll
                for (int k = 0; k < kQKeys / 32; ++k)
                    umma_e4m3(tmem + Q::O_COL, line_desc(v_s + 32 * k * D, D),
                              line_desc(p_s + 32 * k * Q::W, Q::W, kQKeys * Q::W), id_o, k > 0);
                umma_commit(&o_full);
                umma_commit(&v_empty[st]);
                if (Q::NSB == 2 && asked == ch + 1 && asked < n_chunks) issue_scores();
            }
            if (!ok) set_status(c.status, SDV_ERR_DEVICE_TIMEOUT);
        }
        __syncwarp();
    } else if (!is_load) {
        // ---- softmax and accumulation: a thread is key (then dim) `tid % 128` of the chunk
        const int g = warp / 4, col0 = g * CW, key = tid % 128;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        const float unit = q_unit * a.scale_log2;
        float acc[CW], l[CW];
#pragma unroll
        for (int r = 0; r < CW; ++r) acc[r] = l[r] = 0.f;
        // adds the product of the chunk last sent to the tensor cores
        auto accumulate = [&](int ch) {
            if (ok) ok = mbar_wait(&o_full, ch & 1);
            tc_fence_after();
#pragma unroll
            for (int r0 = 0; r0 < CW; r0 += 16) {
                float v[3][16];
#pragma unroll
                for (int p = 0; p < 3; ++p) tmem_ld16(tmem + lanes + Q::O_COL + p * ROWS + col0 + r0, v[p]);
                tmem_ld_wait(v[0], v[1], v[2]);
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    float2 o = make_float2(acc[r0 + r], acc[r0 + r + 1]);
#pragma unroll
                    for (int p = 0; p < 3; ++p) {
                        const float u = p == 0 ? 0x1p-6f : p == 1 ? 0x1p-12f : 0x1p-17f;
                        o = __ffma2_rn(make_float2(v[p][r], v[p][r + 1]), make_float2(u, u), o);
                    }
                    acc[r0 + r] = o.x, acc[r0 + r + 1] = o.y;
                }
            }
        };
        for (int ch = 0; ch < n_chunks; ++ch) {
            const int t0 = first + ch * kQKeys, t = t0 + key;
            const bool masked = t0 + kQKeys - 1 > pos_lo || (a.window > 0 && t0 <= pos_hi - a.window);
            if (ok) ok = mbar_wait(&s_full[ch % Q::NSB], (ch / Q::NSB) & 1);
            tc_fence_after();
            const uint32_t s_col = tmem + lanes + ch % Q::NSB * Q::NS + col0;
            const float ks = kv_scale[ch % 4][0][key] * unit, vs = t < last ? kv_scale[ch % 4][1][key] : 1.f, lv = __log2f(vs);
            // sixteen rows' scores of this key in log2 units, -inf where a row does not see it
            auto scores = [&](int r0, float (&sc)[16]) {
                float v[Q::FOLD ? 1 : Q::PQ - 1][16];
                tmem_ld16(s_col + r0, sc);
                if constexpr (!Q::FOLD) {
#pragma unroll
                    for (int p = 1; p < Q::PQ; ++p) tmem_ld16(s_col + p * ROWS + r0, v[p - 1]);
                    if constexpr (Q::PQ == 2)
                        tmem_ld_wait(sc, v[0]);
                    else
                        tmem_ld_wait(sc, v[0], v[1]);
                } else {
                    tmem_ld_wait(sc);
                }
#pragma unroll
                for (int r = 0; r < 16; r += 2) {
                    float2 z = make_float2(sc[r], sc[r + 1]);
                    if constexpr (!Q::FOLD) {
#pragma unroll
                        for (int p = 1; p < Q::PQ; ++p) {
                            const float u = p == 1 ? 0x1p-5f : 0x1p-10f;
                            z = __ffma2_rn(make_float2(v[p - 1][r], v[p - 1][r + 1]), make_float2(u, u), z);
                        }
                    }
                    z = __fmul2_rn(z, make_float2(ks, ks));
                    sc[r] = z.x, sc[r + 1] = z.y;
                }
                if (masked) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const int pos = pos_s[col0 + r0 + r];
                        if (t > pos || (a.window > 0 && t <= pos - a.window)) sc[r] = -INFINITY;
                    }
                }
            };
            // does a row's w leave the range that its reference covers, w > M + 1? 64-row tiles read the scores from
            // TMEM twice rather than hold them
            float kept[16], over = -INFINITY;
#pragma unroll
            for (int r0 = 0; r0 < CW; r0 += 16) {
                scores(r0, kept);
#pragma unroll
                for (int r = 0; r < 16; r += 4) {
                    const float4 m = *reinterpret_cast<const float4 *>(&m_neg[col0 + r0 + r]);
                    const float2 d = __fadd2_rn(make_float2(kept[r], kept[r + 1]), make_float2(m.x, m.y));
                    const float2 e = __fadd2_rn(make_float2(kept[r + 2], kept[r + 3]), make_float2(m.z, m.w));
                    over = fmaxf(over, fmaxf(fmaxf(d.x, d.y), fmaxf(e.x, e.y)));
                }
            }
            if (ch > 0) accumulate(ch - 1);
            if (bar_or(1 + g, 128, over + lv > 1.f)) {
#pragma unroll
                for (int r0 = 0; r0 < CW; r0 += 16) {
                    if constexpr (Q::FOLD) scores(r0, kept);
                    float top = -INFINITY;
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float m = redux_max(kept[r] + lv);
                        if (lane == r) top = m;
                    }
                    if (lane < 16 && top > -INFINITY) atomicMax(&m_key[col0 + r0 + lane], orderable(top));
                }
                named_bar_sync(1 + g, 128);
                if (key < CW) {
                    const uint32_t k = m_key[col0 + key];
                    const float now = __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k), was = -m_neg[col0 + key];
                    const bool moves = k != 0 && now > was + 1.f;
                    // without a reference so far l holds keys of scale 0 alone, counted from 0
                    m_step[col0 + key] = moves ? ex2(fminf((was == kQNoRef ? 0.f : was) - now, 120.f)) : 1.f;
                    if (moves) m_neg[col0 + key] = -now;
                }
                named_bar_sync(1 + g, 128);
#pragma unroll
                for (int r = 0; r < CW; r += 4) {
                    const float4 f = *reinterpret_cast<const float4 *>(&m_step[col0 + r]);
                    acc[r] *= f.x, acc[r + 1] *= f.y, acc[r + 2] *= f.z, acc[r + 3] *= f.w;
                    l[r] *= f.x, l[r + 1] *= f.y, l[r + 2] *= f.z, l[r + 3] *= f.w;
                }
            }
            // x = 64 p as planes; a line of P holds this key's values of every row and plane. l takes x / (64 vs); keys
            // whose scale is 0 or so small that x may vanish beside it (2^-60) send their warp to the exponential.
            const float lv6 = lv + 6.f;
            const bool small = __any_sync(0xffffffffu, !(vs >= 0x1p-60f));
            const float to_l = small ? 0.f : __fdividef(0x1p-6f, vs);
#pragma unroll
            for (int r0 = 0; r0 < CW; r0 += 16) {
                if constexpr (Q::FOLD) scores(r0, kept);
                if (small) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) {
                        const float m = m_neg[col0 + r0 + r];
                        l[r0 + r] += ex2(kept[r] + (m == -kQNoRef ? 0.f : m));
                    }
                }
                uint32_t w[Q::PP][8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int r = r0 + 2 * j;
                    const float2 m = *reinterpret_cast<const float2 *>(&m_neg[col0 + r]);
                    // (s - M) + log2 vs: the first difference is small where it matters
                    const float2 e = __fadd2_rn(__fadd2_rn(make_float2(kept[2 * j], kept[2 * j + 1]), m), make_float2(lv6, lv6));
                    const float2 x2 = make_float2(ex2(e.x), ex2(e.y));
                    const float2 n = __ffma2_rn(x2, make_float2(to_l, to_l), make_float2(l[r], l[r + 1]));
                    l[r] = n.x, l[r + 1] = n.y;
                    uint32_t x = f16x2(x2.x, x2.y);
#pragma unroll
                    for (int p = 0; p < Q::PP; ++p) {
                        w[p][j] = e4m3_of_f16x2(x);
                        if (p + 1 < Q::PP) x = hscale2_u(hsub2_u(x, f16x2_of_e4m3(w[p][j])), p == 0 ? 64.f : 32.f);
                    }
                }
#pragma unroll
                for (int p = 0; p < Q::PP; ++p) {
                    const int byte = p * ROWS + col0 + r0;
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                     p_s + byte / Q::W * (kQKeys * Q::W) + line_offset(key, byte % Q::W, Q::W)),
                                 "r"(w[p][0] | w[p][1] << 16), "r"(w[p][2] | w[p][3] << 16), "r"(w[p][4] | w[p][5] << 16),
                                 "r"(w[p][6] | w[p][7] << 16)
                                 : "memory");
                }
            }
            if (t0 + kQKeys > last) {  // slots behind the sequence may hold anything, and 0 times a NaN is none
                const int st = ch % kQStages;
                if (ok) ok = mbar_wait(&v_full[st], (ch / kQStages) & 1);
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
        if (n_chunks > 0) accumulate(n_chunks - 1);
        if (!ok && lane == 0) set_status(c.status, SDV_ERR_DEVICE_TIMEOUT);
        // ---- sums over the keys, and the rows out
#pragma unroll
        for (int r0 = 0; r0 < CW; r0 += 16) {
            float sum[16];
#pragma unroll
            for (int r = 0; r < 16; ++r) sum[r] = l[r0 + r];
            const float mine = transpose_sum16(sum, lane);
            if (lane < 16) l_s[warp % 4][col0 + r0 + lane] = mine;
        }
        named_bar_sync(1 + g, 128);
        const int rows = min(CW, n_rows - col0);
        QRow w = row_of(col0);
        if (whole) {
            if (key < D) {
                T *dst = out + w.row * a.out_stride + w.hq * D + key;
                const long long next = a.out_stride - grp * D;  // from past a row's last head to the next row's first
                int left = grp - (w.hq - h * grp);
#pragma unroll
                for (int r = 0; r < CW; ++r) {
                    const int k = col0 + r;
                    const float total = (l_s[0][k] + l_s[1][k]) + (l_s[2][k] + l_s[3][k]);
                    if (r < rows) *dst = from_f32<T>(total == 0.f ? 0.f : __fdividef(acc[r], total));
                    dst += D;
                    if (--left == 0) dst += next, left = grp;
                }
            }
        } else {
            if (key < D) {
                const size_t step = static_cast<size_t>(a.splits) * D;
                float *dst = a.part_o + (qattn_slot(a, b, w.i, w.hq) + split) * D + key;
                const size_t next = (a.nq - grp) * step;
                int left = grp - (w.hq - h * grp);
#pragma unroll
                for (int r = 0; r < CW; ++r) {
                    if (r < rows) *dst = acc[r];
                    dst += step;
                    if (--left == 0) dst += next, left = grp;
                }
            }
            if (key < rows) {
                const int k = col0 + key;
                w = row_of(k);
                a.part_ml[qattn_slot(a, b, w.i, w.hq) + split] =
                    make_float2(-m_neg[k], (l_s[0][k] + l_s[1][k]) + (l_s[2][k] + l_s[3][k]));
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (is_mma) tmem_dealloc(tmem, Q::COLS);
}

constexpr int kQMergeThreads = 128;

// A CTA joins the parts of one (row, q head): o = sum 2^(M_i - M) o_i / sum 2^(M_i - M) l_i, every fourth part a
// warp, the four in order. Grid (span row x head, sequence).
template <typename T, int D>
__global__ void __launch_bounds__(kQMergeThreads) qcache_merge_kernel(QAttnArgs a) {
    constexpr int V = D / 32, NW = kQMergeThreads / 32;
    const int b = blockIdx.y, i = a.by_nq.div(blockIdx.x), hq = blockIdx.x - i * a.nq;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    // the spans are no results of the attention before it, which started after whatever wrote them
    const QSpan s = qcache_span(a.c, b);
    const int L = s.p0 + s.S, keys = qattn_part_keys(a, max(L, 1));
    const int parts = (L + keys - 1) / keys;
    __shared__ float o_s[NW][D], l_s;
    pdl_wait();  // in every CTA: this kernel's end stands for the attention's, too
    pdl_trigger();
    if (i >= s.S || keys >= L) return;
    const size_t slot = qattn_slot(a, b, i, hq);
    // parts without a key of this row hold M = kQNoRef, l = 0, o = 0
    float m = kQNoRef;
    for (int p = lane; p < parts; p += 32) m = fmaxf(m, a.part_ml[slot + p].x);
    m = redux_max(m);
    if (m == kQNoRef) m = 0.f;
    float o[V], l = 0.f;
#pragma unroll
    for (int d = 0; d < V; ++d) o[d] = 0.f;
    // 32 parts at a time: a lane weighs one, the warp's eight are read at once
    for (int p0 = 0; p0 < parts; p0 += 32) {
        const float2 ml = p0 + lane < parts ? a.part_ml[slot + p0 + lane] : make_float2(kQNoRef, 0.f);
        // l > 0 without a reference: keys of scale 0 alone, counted from 0
        const float mine = ml.y == 0.f ? 0.f : ex2(fminf((ml.x == kQNoRef ? 0.f : ml.x) - m, 120.f));
        float v[32 / NW][V];
#pragma unroll
        for (int j = 0; j < 32 / NW; ++j) {
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
        for (int j = 0; j < 32 / NW; ++j) {
            const float f = __shfl_sync(0xffffffffu, mine, warp + j * NW);
#pragma unroll
            for (int d = 0; d < V; ++d) o[d] = fmaf(f, v[j][d], o[d]);
        }
        if (warp == 0) l += warp_sum(mine * ml.y);
    }
#pragma unroll
    for (int d = 0; d < V; ++d) o_s[warp][lane * V + d] = o[d];
    if (threadIdx.x == 0) l_s = l;
    __syncthreads();
    const int d = threadIdx.x;
    if (d < D) {
        const float num = (o_s[0][d] + o_s[1][d]) + (o_s[2][d] + o_s[3][d]), den = l_s;
        static_cast<T *>(a.out)[(s.r0 + i) * a.out_stride + hq * D + d] = from_f32<T>(den == 0.f ? 0.f : num / den);
    }
}

}  // namespace sdv
