// Attention over a 16-bit paged cache for groups of sequences that share a prefix.
//
// The keys of a group's prefix are the same for every row of the group, so its rows are the rows of one product:
//     S [rows x 128 keys] = Q K^T,   O [rows x dims] += P V,   rows = (row of the group) x (head of the kv head's group)
// and the prefix is read once for all of them. Each sequence's own keys (the rest of its prompt, what it generated, its
// span) are a product of their own. A row's parts join as o = sum 2^(M_i - M) o_i / sum 2^(M_i - M) l_i.
//
// A score is z = cap tanh(q.k / (sqrt(D) cap)) - slope_h (pos - t) for key t <= pos (no cap: q.k / sqrt(D)), within the
// window if there is one.
//
// What bounds it (bf16, 32 heads on 8 of 128 dims; pages of 16; the whole call in a graph):
//   16 x 8 rows after 32,768 shared keys  84 us, 820 TFLOP/s: the tensor cores, whose products take 81 % of a chunk. Those with V
//                                         are twice the scores', as p enters in two 16-bit planes
//   64 sequences of one row after them, up to 512 keys of their own   67 us, 3.0 TB/s: a third of the time are the sequences' own tiles,
//                                         64 x 8 of 4 rows, 11,300 clocks each: two steps of a warpgroup's chain (below) one
//                                         after the other, at 3.4 TB/s; not the memory
//   8 x 8 rows after 848 shared keys      18 us: latency, of the plan (5,600 clocks), of the first loads and of code that no
//                                         cache holds, of the join (4 us)
// Why two planes: one leaves p a relative error of 2^-9, which the sum over alike keys keeps; the result then is up to twice as far off
// as its own rounding. With two that rounding is all of the error.
#pragma once

#include "qcache_attention.cuh"

namespace sdv {

constexpr int kSKeys = 128;      // keys of a chunk
constexpr int kSTile = 256;      // rows of a tile: one of 128 for each of two softmax warpgroups
constexpr int kSGroups = 128;    // groups of a call at most
constexpr int kSBatch = 256;     // sequences of a call at most
constexpr int kSEntries = kSGroups + kSBatch;
constexpr int kSOverhead = 3;    // what a tile's queries and results cost, in chunks
constexpr float kSGrow = 8.f;    // a row's reference follows its maximum once that is more than 2^8 above it
constexpr int kSThreads = 384;   // two softmax warpgroups, a warp for K, one for V, two that issue MMAs; as many as entries

struct SharedArgs {
    const void *q;
    void *out;
    long long q_stride, out_stride;  // elements between rows
    const void *pool;                // the layer's [n_pages][2][nkv][page_size][D]
    const int *page_table, *row_off, *base, *group_off, *prefix_len;
    const float *slopes;             // [nq], or null
    int *status;
    int pages_per_seq, page_size, n_pages, nq, nkv, grp, B, G, max_span, max_rows, max_context, window;
    int q_vec, out_vec;              // rows are 16-byte aligned
    int box_rows, pool_rows;         // rows of a TMA box (0: pages that none fits); rows of the layer's pool: a box there reads zeros
    FastDiv by_page, by_grp, by_nq;
    float scale_log2, cap2, to_u;    // log2(e) / sqrt(D); log2(e) cap or 0, 1 / (sqrt(D) cap)
    int ctas;                        // CTAs of the attention kernel, which the cut into parts follows
    int part_rows;                   // partial rows of a kv head
    float *part_o;                   // partial results: [nkv][part_rows] rows of sequences' own tiles, as many of prefix tiles,
                                     // [ctas][kSTile] of pieces that begin inside of a tile
    float2 *part_ml;                 // (M, l) of each
    // the plan for the kernel that joins the parts: an entry's start on the line, cost of a tile, chunks and cost of one, and its
    // first row and tiles a kv head; the length and overhead of the cut
    int4 *plan;
    int2 *plan_rows, *plan_cut;
    FastDiv *by_cut;
    int2 *row_entry;                 // [max_rows]: a row's entry, kRowNone or kRowRefused, and that of its prefix or -1
};
constexpr int kRowNone = -1, kRowRefused = -2;

// ------------------------------------------------------------------ the work and its cut
// Work is a list of entries, the groups' prefixes and then the sequences' own keys. An entry is tiles of up to kSTile rows
// for each kv head, a tile is chunks. Chunks lie one behind another on a line of costs (a tile's first costs `ov` more, and a
// chunk of more than 128 rows counts twice), and CTA i takes those that begin in [i q, (i + 1) q). So the CTAs finish
// together whatever the lengths are, every one of them knows the whole cut, and a tile is cut where the line is.
// Where there are few tiles, a cut into pieces of one tile only is better, as long as they are no more than the CTAs: a second
// piece costs about kSOverhead chunks (eight sequences of 848 keys with spans of eight: 18.1 us, 22.8 without).
// The lengths are read once, side by side, and all else is worked out in shared memory: as reads that wait for one another it
// took 20 us.
struct SEntry {
    int start, end;   // its part of the line
    int b;            // sequence whose page table is read
    int r0, rows;     // rows of the call
    int p0;           // own: position of the first row; prefix: -1
    int kv0, kv1;     // its keys
    int lo;           // first key that any row sees
    int max_lo, min_hi;  // every row sees [max_lo, min_hi)
    int c0, nc;       // first chunk, chunks
    int per, wc;      // cost of a tile, of a chunk
    int group;        // own: its group, -1 without one
};
struct SPlan {
    SEntry e[kSEntries];
    int row_off[kSBatch + 1], base[kSBatch], group_off[kSGroups + 1], prefix[kSGroups];
    int g_min[kSGroups], g_max[kSGroups];  // lowest and highest position of a group's rows
    int total, q, ov, best;
    int2 warp_sum[kSThreads / 32];
};

__device__ __forceinline__ int shared_last(const int *off, int n, int v) {  // the last of n offsets that is not above v
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (off[mid] <= v) lo = mid; else hi = mid;
    }
    return lo;
}
__device__ __forceinline__ int shared_tiles(const SharedArgs &a, const SEntry &n) { return (n.rows * a.grp + kSTile - 1) / kSTile; }

// The plan, by kSThreads threads. Thread e works out entry e: first the sequences', a sequence being refused as by
// qcache_span or where its rows do not all lie behind its group's prefix, then the groups'.
__device__ __forceinline__ void shared_plan(const SharedArgs &a, SPlan &pl, bool writes) {
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid <= a.B) pl.row_off[tid] = a.row_off[tid];
    if (tid < a.B) pl.base[tid] = a.base[tid];
    if (tid <= a.G && a.G) pl.group_off[tid] = a.group_off[tid];
    if (tid < a.G) pl.prefix[tid] = a.prefix_len[tid], pl.g_min[tid] = 0x7fffffff, pl.g_max[tid] = -1;
    if (tid == 0) pl.best = 0x7fffffff;
    __syncthreads();
    const bool groups_ok = __syncthreads_and(tid >= a.G || (pl.group_off[tid] <= pl.group_off[tid + 1] && (tid > 0 || pl.group_off[0] == 0) &&
                                                            (tid < a.G - 1 || pl.group_off[a.G] == a.B)));
    SEntry n{};
    n.group = -1;
    int code = SDV_OK;
    const int b = tid - a.G;
    if (b >= 0 && b < a.B) {
        n.b = b;
        n.r0 = pl.row_off[b];
        n.rows = pl.row_off[b + 1] - n.r0;
        n.p0 = pl.base[b];
        if (n.rows != 0) {
            if (n.rows < 0 || n.r0 < 0 || n.rows > a.max_rows || n.r0 > a.max_rows - n.rows || n.rows > a.max_span) {
                code = SDV_ERR_ARG;
            } else if (n.p0 < 0 || n.p0 > a.max_context - n.rows) {
                code = SDV_ERR_CAPACITY;
            } else if (a.G) {
                code = SDV_ERR_ARG;
                if (groups_ok) {
                    const int g = shared_last(pl.group_off, a.G, b);
                    const int first = pl.row_off[pl.group_off[g]], last = pl.row_off[pl.group_off[g + 1]];
                    n.kv0 = pl.prefix[g];
                    if (n.kv0 >= 0 && n.kv0 <= n.p0 && first >= 0 && last <= a.max_rows && n.r0 >= first && n.r0 + n.rows <= last) {
                        code = SDV_OK;
                        n.group = g;
                        atomicMin(&pl.g_min[g], n.p0);
                        atomicMax(&pl.g_max[g], n.p0 + n.rows - 1);
                    }
                }
            }
            if (code != SDV_OK) {
                n.rows = 0;
                if (writes) set_status(a.status, code);
            }
        }
        n.kv1 = n.p0 + n.rows;
        n.lo = a.window > 0 ? max(n.kv0, n.p0 - a.window + 1) : n.kv0;
        n.max_lo = a.window > 0 ? max(n.kv0, n.kv1 - a.window) : n.kv0;
        n.min_hi = n.p0 + 1;
    }
    __syncthreads();
    if (tid < a.G && groups_ok && pl.g_min[tid] <= pl.g_max[tid]) {  // some row of the group is read
        n.p0 = -1;
        n.b = pl.group_off[tid];
        n.r0 = pl.row_off[n.b];
        n.rows = pl.row_off[pl.group_off[tid + 1]] - n.r0;
        n.kv1 = pl.prefix[tid];
        n.lo = a.window > 0 ? max(0, pl.g_min[tid] - a.window + 1) : 0;
        n.max_lo = a.window > 0 ? max(0, pl.g_max[tid] - a.window + 1) : 0;
        n.min_hi = n.kv1;
    }
    n.c0 = n.lo / kSKeys;
    n.nc = n.rows && n.lo < n.kv1 ? (n.kv1 + kSKeys - 1) / kSKeys - n.c0 : 0;
    n.wc = n.rows * a.grp > kSTile / 2 ? 2 : 1;
    const int tiles = n.nc ? a.nkv * shared_tiles(a, n) : 0, one = n.nc * n.wc, steps = tiles * one;
    // sums over the entries before this one, of costs and of tiles
    int sum = steps, count = tiles;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o), u = __shfl_up_sync(0xffffffffu, count, o);
        if (lane >= o) sum += v, count += u;
    }
    if (lane == 31) pl.warp_sum[warp] = make_int2(sum, count);
    pl.e[tid].nc = one, pl.e[tid].rows = tiles;  // for a moment: cost of a tile, tiles
    __syncthreads();
    int2 all = make_int2(0, 0), before = make_int2(0, 0);
#pragma unroll
    for (int w = 0; w < kSThreads / 32; ++w) {
        const int2 v = pl.warp_sum[w];
        all.x += v.x, all.y += v.y;
        if (w < warp) before.x += v.x, before.y += v.y;
    }
    int ov = kSOverhead, cost = steps + ov * tiles, per = ov + one, total = all.x + ov * all.y;
    int end = before.x + sum + ov * (before.y + count), q = max(1, (total + a.ctas - 1) / a.ctas);
    if (all.y <= a.ctas && all.y > 0) {  // pieces of one tile each: a warp tries a length
        const int tried = (all.x + a.ctas - 1) / a.ctas + warp;
        int pieces = 0;
        for (int e = lane; e < a.G + a.B; e += 32) pieces += pl.e[e].rows * ((pl.e[e].nc + tried - 1) / tried);
        pieces = __reduce_add_sync(0xffffffffu, pieces);
        if (lane == 0 && pieces <= a.ctas) atomicMin(&pl.best, tried);
        __syncthreads();
        if (pl.best <= q + 2) {
            q = pl.best;
            ov = 0;
            per = (one + q - 1) / q * q;  // every tile begins with a CTA
            cost = sum = tiles * per;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, sum, o);
                if (lane >= o) sum += v;
            }
            if (lane == 31) pl.warp_sum[warp].x = sum;
            __syncthreads();
            total = 0;
            end = sum;
#pragma unroll
            for (int w = 0; w < kSThreads / 32; ++w) {
                const int v = pl.warp_sum[w].x;
                total += v;
                if (w < warp) end += v;
            }
        }
    }
    n.end = end;
    n.start = end - cost;
    n.per = per;
    pl.e[tid] = n;
    if (tid == 0) pl.total = total, pl.ov = ov, pl.q = q;
    __syncthreads();
    if (writes) {
        if (tid < a.G + a.B) {
            a.plan[tid] = make_int4(n.start, n.per, n.nc, n.wc);
            a.plan_rows[tid] = make_int2(n.r0, shared_tiles(a, n));
        }
        if (tid == kSThreads - 1) {  // as FastDiv::of
            const int l = q > 1 ? 32 - __clz(q - 1) : 0;
            *a.by_cut = FastDiv{static_cast<uint32_t>((1ull << (31 + l)) / q + 1), 31 + l};
            *a.plan_cut = make_int2(q, ov);
        }
        for (int r = tid; r < a.max_rows; r += kSThreads) {
            const int of = shared_last(pl.row_off, a.B, r);
            const bool in = r >= pl.row_off[of] && r < pl.row_off[of + 1];
            const SEntry &m = pl.e[a.G + of];
            a.row_entry[r] = make_int2(!in ? kRowNone : m.rows ? a.G + of : kRowRefused, m.group >= 0 && pl.e[m.group].nc ? m.group : -1);
        }
    }
}
// First chunk of a tile that begins at or after `rel` on the line, from the tile's start.
__device__ __forceinline__ int shared_chunk(int chunks, int wc, int ov, int rel) {
    if (rel <= 0) return 0;
    return min(chunks, rel <= ov + wc ? 1 : (rel - ov + wc - 1) >> (wc - 1));  // wc is 1 or 2
}
// The part of a tile that a CTA does. Each warp steps from one to the next by itself.
struct SPiece {
    int entry, h, tile, at;  // kv head, tile, where the tile starts on the line
    int rows;                // rows x heads of the tile
    int c0, n;               // its first chunk, from the entry's first, and how many
    int tiles;             // tiles a kv head
};
// Takes the tile that p names; false where none of its chunks lies in [x, x1).
__device__ __forceinline__ bool shared_take(const SharedArgs &a, const SPlan &pl, int x, int x1, SPiece &p) {
    const SEntry &n = pl.e[p.entry];
    p.c0 = shared_chunk(n.nc, n.wc, pl.ov, x - p.at);
    p.n = (x1 >= p.at + n.per ? n.nc : shared_chunk(n.nc, n.wc, pl.ov, x1 - p.at)) - p.c0;
    p.rows = min(kSTile, n.rows * a.grp - p.tile * kSTile);
    return p.n > 0;
}
// The first piece of [x, x1) or the next one, false at the end.
__device__ __forceinline__ bool shared_next(const SharedArgs &a, const SPlan &pl, int x, int x1, SPiece &p) {
    do {
        const SEntry &n = pl.e[p.entry];
        p.at += n.per;
        if (p.at >= x1) return false;
        if (++p.tile == p.tiles) {
            p.tile = 0;
            if (++p.h == a.nkv) {
                p.h = 0;
                do ++p.entry;
                while (pl.e[p.entry].end == p.at);  // entries without work; the line goes on, so one comes
                p.tiles = shared_tiles(a, pl.e[p.entry]);
            }
        }
    } while (!shared_take(a, pl, x, x1, p));
    return true;
}
__device__ __forceinline__ bool shared_first(const SharedArgs &a, const SPlan &pl, int x, int x1, SPiece &p) {
    if (x >= x1) return false;
    int lo = 0, hi = a.G + a.B - 1;  // the first entry that ends behind x
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (pl.e[mid].end > x) hi = mid; else lo = mid + 1;
    }
    const SEntry &n = pl.e[lo];
    const int th = (x - n.start) / n.per;
    p.entry = lo;
    p.tiles = shared_tiles(a, n);
    p.h = th / p.tiles;
    p.tile = th - p.h * p.tiles;
    p.at = n.start + th * n.per;
    return shared_take(a, pl, x, x1, p) || shared_next(a, pl, x, x1, p);
}

// Where a tile's partial result lies: its first row.
__device__ __forceinline__ long long shared_slot(const SharedArgs &a, bool prefix, int r0, int h, int tile, int cta) {
    const long long side = static_cast<long long>(a.nkv) * a.part_rows;
    if (cta >= 0) return 2 * side + static_cast<long long>(cta) * kSTile;
    return (prefix ? side : 0) + static_cast<long long>(h) * a.part_rows + r0 * a.grp + tile * kSTile;
}

// ------------------------------------------------------------------ PTX
// D[tmem] (+)= A[tmem] * B[smem desc], kind::f16.
__device__ __forceinline__ void umma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Instruction descriptor, kind::f16: fp32 D; bf16 or fp16 operands; mn: B runs along N in memory.
template <typename T>
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool mn) {
    constexpr uint32_t t = __is_same(T, bf16) ? 1u : 0u;
    return (1u << 4) | (t << 7) | (t << 10) | (mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
           (static_cast<uint32_t>(M >> 4) << 24);
}
// 32 TMEM columns of this thread's lane; tmem_wait_ld before the values are used.
__device__ __forceinline__ void tmem_get32(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]),
          "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]),
          "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]),
          "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ void tmem_pass32(float *v) {
#pragma unroll
    for (int i = 0; i < 32; i += 8)
        asm volatile("" : "+f"(v[i]), "+f"(v[i + 1]), "+f"(v[i + 2]), "+f"(v[i + 3]), "+f"(v[i + 4]), "+f"(v[i + 5]), "+f"(v[i + 6]),
                          "+f"(v[i + 7]));
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_put32(uint32_t taddr, const float *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]), "f"(v[8]), "f"(v[9]), "f"(v[10]),
        "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]), "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]),
        "f"(v[21]), "f"(v[22]), "f"(v[23]), "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]),
        "f"(v[31])
        : "memory");
}
__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t *v) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]), "r"(v[10]),
        "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}
// 32 bytes, a whole sector: lanes hold rows of their own.
__device__ __forceinline__ void store8(float *dst, const float *v) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]),
                 "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
// True in one lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t e;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(e));
    return e != 0;
}
// A box of 64 columns of the pool's rows into shared memory, completion counted on `bar`.
__device__ __forceinline__ void load_box_at(uint32_t dst, const CUtensorMap *tm, uint64_t *bar, int col, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(col), "r"(row)
        : "memory");
}

// Two probabilities, rounded to a pair of 16-bit planes, each two to a word: p = hi + lo to 2^-17 (bf16) or 2^-23 (fp16).
template <typename T>
__device__ __forceinline__ void split_p(float2 p, uint32_t &hi, uint32_t &lo) {
    if constexpr (__is_same(T, bf16)) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(p.x, p.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        const float2 r = __fadd2_rn(p, make_float2(-__uint_as_float(hi << 16), -__uint_as_float(hi & 0xffff0000u)));
        const __nv_bfloat162 l = __floats2bfloat162_rn(r.x, r.y);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(p.x, p.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        const float2 f = __half22float2(h), r = __fadd2_rn(p, make_float2(-f.x, -f.y));
        const __half2 l = __floats2half2_rn(r.x, r.y);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}
template <typename T>
__device__ __forceinline__ uint32_t pack16(float x, float y) {
    if constexpr (__is_same(T, bf16)) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    } else {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
}
// cap2 tanh(u) of two u. tanh(u) = u P(u^2) / Q(u^2), fitted to 2^-24 for |u| <= 8.5, where tanh is 1 - 2^-23.5 and is left so; in fp32
// 2^-21.3 of the result, however far below the cap. NaN stays NaN.
__device__ __forceinline__ float2 cap_tanh(float2 u, float cap2) {
    auto within = [](float x) {
        float y;
        asm("{\n\t.reg .f32 t;\n\t"
            "min.NaN.f32 t, %1, 0f41080000;\n\t"
            "max.NaN.f32 %0, t, 0fC1080000;\n\t}"
            : "=f"(y)
            : "f"(x));
        return y;
    };
    u = make_float2(within(u.x), within(u.y));
    const float2 w = __fmul2_rn(u, u);
    auto step = [&](float2 p, float c) { return __ffma2_rn(p, w, make_float2(c, c)); };
    const float2 p = step(step(step(step(make_float2(1.2462526e-8f, 1.2462526e-8f), 2.0059697e-5f), 3.4660716e-3f), 0.13357386f), 0.99999994f);
    const float2 q = step(step(step(step(make_float2(7.4397485e-7f, 7.4397485e-7f), 3.234685e-4f), 2.5768507e-2f), 0.4669072f), 1.f);
    const float2 n = __fmul2_rn(__fmul2_rn(u, make_float2(cap2, cap2)), p);
    return make_float2(__fdividef(n.x, q.x), __fdividef(n.y, q.y));
}
// Of 32 keys those in [lo, hi), as bits.
__device__ __forceinline__ uint32_t seen_bits(int lo, int hi) {
    const uint32_t above = hi <= 0 ? 0u : hi >= 32 ? 0xffffffffu : (1u << hi) - 1;
    return above & (lo <= 0 ? 0xffffffffu : lo >= 32 ? 0u : ~((1u << lo) - 1));
}
// Whether any of eight 16-bit values is an infinity or a NaN.
template <typename T>
__device__ __forceinline__ bool not_finite8(uint4 u) {
    constexpr uint32_t e = __is_same(T, bf16) ? 0x7f80u : 0x7c00u, ee = e | e << 16;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = (i == 0 ? u.x : i == 1 ? u.y : i == 2 ? u.z : u.w) & ee;
        bad |= (w & 0xffffu) == e || (w >> 16) == e;
    }
    return bad;
}

template <int N>
struct Int {
    static constexpr int value = N;
};
struct SShared {
    uint64_t full[8], empty[8], s_full[2], p_half[2], p_full[2], o_done[2], q_full, q_empty, q_first, turn[2];
    uint32_t tmem;
    // keys of a chunk that are not finite, as bits: [chunks that one warpgroup looks at, that both do][turn][warpgroup that found them]
    uint32_t bad[2][2][2][4];
    float2 ml[2][128];  // (M, l) of the rows that two warpgroups share
    SPlan plan;
};

template <typename T, int D_>
struct STile {
    static constexpr int D = D_, HALVES = D / 64;
    static constexpr int SLOT = kSKeys * D * 2;              // bytes of a K or V chunk, as halves of 64 columns
    static constexpr int Q_BYTES = 128 * D * 2;              // and of 128 rows of Q
    static constexpr int DEPTH = D == 128 ? 2 : 4;           // K chunks, and V chunks, in shared memory
    static constexpr int SLOTS = 2 * DEPTH;
    static constexpr int SMEM = 2 * Q_BYTES + SLOTS * SLOT + static_cast<int>((sizeof(SShared) + 127) / 128 * 128);
    static constexpr int O_COL = 256;                        // TMEM: S of each warpgroup, then O of each
    // p carries a factor 2^6 in fp16, whose smallest values lie at 2^-24; 2^(6 + kSGrow) is its largest
    static constexpr float BIAS = __is_same(T, bf16) ? 0.f : 6.f;
    static_assert(SMEM <= 227 * 1024, "shared memory");
};
// ------------------------------------------------------------------ attention
// One CTA an SM; a piece of the line after another. EXTRA: scores with a cap or a bias.
// A batch of 16 sequences of 512 to 4,096 keys, up to 32 rows a tile, takes 41 us, 48 with a cap: each warpgroup's chain of scores, softmax
// and product, 5,600 clocks a chunk or 7,400, of which two run at once (of 512 to 2,048 keys 28.7 us, 26.4 where L2 holds them).
template <typename T, int D, bool EXTRA>
__global__ void __launch_bounds__(kSThreads, 1) shared_attn_kernel(const __grid_constant__ CUtensorMap pool,
                                                                   const __grid_constant__ SharedArgs a) {
    typedef STile<T, D> Q;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t q_s = smem_u32(smem_raw), kv_s = q_s + 2 * Q::Q_BYTES;
    SShared &sh = *reinterpret_cast<SShared *>(smem_raw + 2 * Q::Q_BYTES + Q::SLOTS * Q::SLOT);
    if (tid < 32) sh.bad[tid / 16][tid / 8 % 2][tid / 4 % 2][tid % 4] = 0;
    if (tid == 0) {
        for (int i = 0; i < Q::SLOTS; ++i) {
            mbar_init(&sh.full[i], a.box_rows ? 1 : 32);
            mbar_init(&sh.empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh.s_full[i], 1);
            mbar_init(&sh.p_half[i], 128);
            mbar_init(&sh.p_full[i], 128);
            mbar_init(&sh.o_done[i], 1);
            mbar_init(&sh.turn[i], 1);
        }
        mbar_init(&sh.q_full, 256);
        mbar_init(&sh.q_empty, 2);
        mbar_init(&sh.q_first, 256);
        fence_mbar_init();
    }
    if (warp == 10) {
        tmem_alloc(&sh.tmem, 512);
        tmem_relinquish();
    }
    pdl_wait();
    pdl_trigger();  // after the wait: what starts behind this kernel may read what came before it
    tc_fence_before();
    shared_plan(a, sh.plan, blockIdx.x == 0);
    tc_fence_after();
    const SPlan &pl = sh.plan;
    const uint32_t tmem = sh.tmem;
    const int cta = blockIdx.x;
    const int x = cta * pl.q, x1 = min(pl.total, x + pl.q);
    bool ok = true;  // false once a wait gave up: the rest runs without waiting, and the status word says so
    SPiece p;
    bool more = shared_first(a, pl, x, x1, p);  // by all warps alike: the code comes in once

    // K of chunk c of a piece lies in slot c % DEPTH, V in DEPTH more. A slot is filled once more for every chunk: `used` counts
    // the fillings before the piece, and tells the phase of the slot's barriers.
    int used[Q::DEPTH] = {};
    auto filling = [&](int c) {
        int u = used[0];
#pragma unroll
        for (int i = 1; i < Q::DEPTH; ++i) u = c % Q::DEPTH == i ? used[i] : u;
        return u + c / Q::DEPTH;
    };
    auto next_piece = [&](int n) {
#pragma unroll
        for (int i = 0; i < Q::DEPTH; ++i) used[i] += (n + Q::DEPTH - 1 - i) / Q::DEPTH;
    };

    if (warp == 8 || warp == 9) {
        // ---- the load warps: one brings K chunks, one V chunks
        const bool v = warp == 9;
        const int nb = a.box_rows ? kSKeys / a.box_rows : 0;
        bool first = true;
        for (; more; more = shared_next(a, pl, x, x1, p)) {
            const SEntry &en = pl.e[p.entry];
            const int *table = a.page_table + static_cast<size_t>(en.b) * a.pages_per_seq;
            const int n = p.n, t00 = (en.c0 + p.c0) * kSKeys, seen_lo = en.lo, seen_hi = en.kv1;
            // In boxes a lane brings one; its page is asked for a chunk ahead.
            const int j = a.box_rows ? lane % nb : 0, half = a.box_rows ? lane / nb : 0;
            auto wants = [&](int c) {  // some row sees a key of the box
                const int t = t00 + c * kSKeys + j * a.box_rows;
                return c < n && half < Q::HALVES && t + a.box_rows > seen_lo && t < seen_hi;
            };
            auto ask = [&](int c) { return wants(c) ? table[a.by_page.div(t00 + c * kSKeys + j * a.box_rows)] : -1; };
            int page = a.box_rows ? ask(0) : 0;
            // at the start the queries come first: behind everybody's keys they would wait for 5,000 clocks. A barrier of their own,
            // of one phase: the second queries may be there before this warp looks, and then the phase of q_full has passed by.
            if (first && v && ok) ok = mbar_wait(&sh.q_first, 0);
#pragma unroll 1
            for (int c = 0; c < n; ++c) {
                const int st = (v ? Q::DEPTH : 0) + c % Q::DEPTH, use = filling(c), t0 = t00 + c * kSKeys;
                const uint32_t dst = kv_s + st * Q::SLOT;
                uint64_t *full = &sh.full[st];
                if (first && !v && c == 1 && ok) ok = mbar_wait(&sh.q_first, 0);
                if (a.box_rows) {
                    int row = a.pool_rows;  // zeros
                    if (!wants(c)) {
                    } else if (page >= 0 && page < a.n_pages) {
                        const int t = t0 + j * a.box_rows;
                        row = ((page * 2 + (v ? 1 : 0)) * a.nkv + p.h) * a.page_size + t - a.by_page.div(t) * a.page_size;
                    } else {
                        set_status(a.status, SDV_ERR_CAPACITY);
                    }
                    page = ask(c + 1);
                    if (use > 0 && ok) ok = mbar_wait(&sh.empty[st], (use - 1) & 1);
                    if (lane == 0) mbar_arrive_expect_tx(full, Q::SLOT);
                    __syncwarp();
                    if (lane < nb * Q::HALVES)
                        load_box_at(dst + half * (kSKeys * 128) + j * a.box_rows * 128, &pool, full, half * 64, row);
                } else {
                    if (use > 0 && ok) ok = mbar_wait(&sh.empty[st], (use - 1) & 1);
                    constexpr int PPR = D / 8, RPI = 32 / PPR;  // 16-byte pieces of a row, rows a copy
                    const int piece = lane % PPR;
#pragma unroll 4
                    for (int r = lane / PPR; r < kSKeys; r += RPI) {
                        const int t = t0 + r;
                        const uint8_t *src = static_cast<const uint8_t *>(a.pool);
                        bool in = false;
                        if (t >= seen_lo && t < seen_hi) {
                            const int at = a.by_page.div(t), id = table[at];
                            in = id >= 0 && id < a.n_pages;
                            if (in)
                                src += (((static_cast<size_t>(id) * 2 + (v ? 1 : 0)) * a.nkv + p.h) * a.page_size + t -
                                        at * a.page_size) * (D * 2) + piece * 16;
                            else
                                set_status(a.status, SDV_ERR_CAPACITY);
                        }
                        cp_async16(dst + piece / 8 * (kSKeys * 128) + line_offset(r, piece % 8 * 16, 128), src, in);
                    }
                    cp_async_arrive(full);
                }
            }
            first = false;
            next_piece(n);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        if (!ok) {  // no copy may land after this CTA's shared memory is someone else's
            for (int i = 0; i < Q::DEPTH; ++i)
                if (used[i]) mbar_wait(&sh.full[(v ? Q::DEPTH : 0) + i], (used[i] - 1) & 1);
            if (lane == 0) set_status(a.status, SDV_ERR_DEVICE_TIMEOUT);
        }
    } else if (warp >= 10) {
        // ---- MMA issue, a warp for each softmax warpgroup: for its own 128 rows of a tile of more than 128 and every chunk, else
        // for the tile's rows and every other chunk. The warps take turns, a step's products with V and the next scores a turn,
        // so that one warpgroup's softmax runs beside the other's products; a warp waits for what it needs before its turn, while
        // the other's MMAs run (a step's products take 1,536 clocks and a step 1,750; 2,090 with one warp for both, 2,450 by two
        // without turns, which fell into step). The whole warp loops and one lane issues: with a lane of its own (lane 0 alone in the loop)
        // an MMA took 80 to 100 clocks to issue, 61 so. What steers the loop passes through a shuffle, so that it is known to
        // be the same in every lane, and a wait that needs none is a single look.
        constexpr uint32_t id_s = idesc_16<T>(128, kSKeys, false), id_o = idesc_16<T>(128, D, true);
        auto same = [](uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); };
        const uint32_t w = same(warp - 10), tm = same(tmem), s_t = tm + w * kSKeys, o_t = tm + Q::O_COL + w * 128;
        uint32_t k_bits = 0, v_bits = 0, p_bit = 0, q_bit = 0, turn_bit = 0;  // the phase of each barrier that comes next
        bool turns = w;  // the first turn of all is warp 0's without a wait
        auto await = [&](uint64_t *bar, uint32_t parity) {
            if (!mbar_try_wait(bar, parity) && ok) ok = mbar_wait(bar, parity);
        };
        for (; more; more = shared_next(a, pl, x, x1, p)) {
            const bool wide = same(p.rows) > 128;
            const int n = same(p.n), steps = wide ? n : (n + 1 - static_cast<int>(w)) >> 1, rounds = wide ? n : (n + 1) >> 1;
            await(&sh.q_full, q_bit);
            q_bit ^= 1;
            tc_fence_after();
            fence_async_smem();  // copies in pieces are generic writes; the tensor cores read through the async proxy
            const uint64_t qd = sw128_desc(q_s + (wide && w ? Q::Q_BYTES : 0));
            // Slots are filled for the other warp, too: their phases count every chunk of the piece.
#pragma unroll 1
            for (int j = -1; j < rounds; ++j) {  // the products with V of step j, the scores of step j + 1
                const int c = wide ? j : 2 * j + static_cast<int>(w), next = wide ? j + 1 : c + 2;
                const bool mine = j >= 0 && j < steps, ahead = j + 1 < steps;
                const int v_at = c % Q::DEPTH, k_at = next % Q::DEPTH;
                const uint64_t vd = line_desc(kv_s + (Q::DEPTH + v_at) * Q::SLOT, 128, kSKeys * 128);
                auto half = [&](int h) {  // 64 keys: of 16 the hi plane, then lo, eight columns each
#pragma unroll
                    for (int i = 0; i < kSKeys / 16; ++i) {
                        const int k = h * (kSKeys / 16) + i;
                        umma_f16_ts(o_t, s_t + k / 4 * 32 + k % 2 * 16 + k / 2 % 2 * 8, vd + (k / 2 * 2048 >> 4), id_o, h > 0 || j > 0 || i > 0);
                    }
                };
                if (mine) {
                    await(&sh.p_half[w], p_bit);
                    await(&sh.full[Q::DEPTH + v_at], v_bits >> v_at & 1);
                    v_bits ^= 1u << v_at;
                }
                if (ahead) {
                    await(&sh.full[k_at], k_bits >> k_at & 1);
                    k_bits ^= 1u << k_at;
                }
                if (turns) {
                    await(&sh.turn[w], turn_bit);
                    turn_bit ^= 1;
                }
                turns = true;
                tc_fence_after();
                if (!a.box_rows) fence_async_smem();
                if (mine) {
                    if (elect_one()) half(0);
                    await(&sh.p_full[w], p_bit);
                    p_bit ^= 1;
                    tc_fence_after();
                }
                if (elect_one()) {
                    if (mine) {
                        half(1);
                        umma_commit(&sh.o_done[w]);
                        umma_commit(&sh.empty[Q::DEPTH + v_at]);
                        if (!wide) umma_commit(&sh.empty[Q::DEPTH + v_at]);  // for the other warp, which does not read it
                    }
                    if (ahead) {
                        const uint64_t kd = sw128_desc(kv_s + k_at * Q::SLOT);
#pragma unroll
                        for (int k = 0; k < D / 16; ++k) {
                            const uint32_t off = (k / 4 * (128 * 128) + k % 4 * 32) >> 4;
                            umma_bf16(s_t, qd + off, kd + off, id_s, k > 0);
                        }
                        umma_commit(&sh.s_full[w]);
                        umma_commit(&sh.empty[k_at]);
                        if (!wide) umma_commit(&sh.empty[k_at]);
                        if (j + 2 == steps) umma_commit(&sh.q_empty);
                    }
                    mbar_arrive(&sh.turn[1 - w]);
                }
                __syncwarp();
            }
            if (steps == 0 && lane == 0) mbar_arrive(&sh.q_empty);
            if (!wide) {  // the slots that the other warp used moved on as well
#pragma unroll
                for (int i = 0; i < Q::DEPTH; ++i) {
                    if (i % 2 == static_cast<int>(w)) continue;
                    const uint32_t odd = (n + Q::DEPTH - 1 - i) / Q::DEPTH & 1;
                    k_bits ^= odd << i;
                    v_bits ^= odd << i;
                }
            }
        }
        if (!ok && lane == 0) set_status(a.status, SDV_ERR_DEVICE_TIMEOUT);
        __syncwarp();
    } else if (warp < 8) {
        // ---- softmax: a thread is a row of its warpgroup's 128
        const int w = warp / 4, m = tid % 128;
        const uint32_t lanes = static_cast<uint32_t>(warp % 4 * 32) << 16;
        const uint32_t s_t = tmem + lanes + w * kSKeys, o_t = tmem + lanes + Q::O_COL + w * 128;
        int done = 0, pieces = 0;  // this warpgroup's steps, pieces
        uint32_t looks = 0;        // whose turn the marks in `bad` are: bit 0 alone, bit 1 (the same in both warpgroups) together
        // The queries of a piece go into their swizzled halves as soon as the last one's scores have read theirs, beside its last
        // products and results. Rows behind the tile's keep what lies there: they only make results that nobody reads.
        auto load_q = [&](const SPiece &p) {
            constexpr int PPR = D / 8, RPI = 256 / PPR;  // 16-byte pieces of a row, rows a copy
            const int piece = tid % PPR, r00 = pl.e[p.entry].r0;
            if (pieces > 0 && ok) ok = mbar_wait(&sh.q_empty, (pieces - 1) & 1);
            ++pieces;
#pragma unroll 4
            for (int r = tid / PPR; r < p.rows; r += RPI) {
                const int mm = p.tile * kSTile + r, i = a.by_grp.div(mm);
                const T *src = static_cast<const T *>(a.q) + (r00 + i) * a.q_stride + (p.h * a.grp + mm - i * a.grp) * D + piece * 8;
                const uint32_t to = q_s + r / 128 * Q::Q_BYTES + piece / 8 * (128 * 128) + line_offset(r % 128, piece % 8 * 16, 128);
                if (a.q_vec) {
                    cp_async16(to, src, true);
                } else {
                    const Raw8<T> raw = load_raw8<T, false>(src);
                    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(raw.u[0].x), "r"(raw.u[0].y),
                                 "r"(raw.u[0].z), "r"(raw.u[0].w)
                                 : "memory");
                }
            }
            if (a.q_vec) {
                cp_async_arrive(&sh.q_full);
                if (pieces == 1) cp_async_arrive(&sh.q_first);
            } else {
                fence_async_smem();
                mbar_arrive(&sh.q_full);
                if (pieces == 1) mbar_arrive(&sh.q_first);
            }
        };
        if (more) load_q(p);
        while (more) {
            const SEntry &en = pl.e[p.entry];
            const bool wide = p.rows > 128, prefix = en.p0 < 0;
            const int n = p.n, r00 = en.r0, kv_lo = en.lo, kv_end = en.kv1, t00 = (en.c0 + p.c0) * kSKeys, steps = wide ? n : (n + 1 - w) >> 1;
            const int all_lo = en.max_lo, all_hi = en.min_hi;  // what every row sees
            const int m0 = p.tile * kSTile, row0 = wide ? w * 128 : 0, n_rows = min(128, p.rows - row0);
            named_bar_sync(1, 256);  // nobody reads the last piece's results any more
            // this thread's row: its position and the keys it sees
            const int mm = m0 + row0 + max(0, min(m, n_rows - 1)), i = a.by_grp.div(mm), row = r00 + i;
            const int hq = p.h * a.grp + mm - i * a.grp;
            int pos = en.p0 + i;
            if (prefix && (a.window > 0 || EXTRA)) {  // a prefix's rows belong to several sequences
                const int b = shared_last(pl.row_off, a.B, row);
                pos = pl.base[b] + row - pl.row_off[b];
            }
            const int see_hi = prefix ? kv_end : pos + 1, see_lo = a.window > 0 ? max(en.kv0, pos - a.window + 1) : en.kv0;
            float slope2 = 0.f;  // log2(e) slope
            if constexpr (EXTRA) slope2 = a.slopes ? a.slopes[hq] * 1.4426950408889634f : 0.f;
            const bool live = warp % 4 * 32 < n_rows;  // rows of this warp
            float M = kQNoRef;
            float2 l2 = make_float2(0.f, 0.f);
            bool poisoned = false;
            for (int j = 0; j < steps; ++j) {
                const int c = wide ? j : 2 * j + w, t0 = t00 + c * kSKeys;
                const bool masked = t0 + kSKeys > all_hi || t0 < all_lo;
                if (ok) ok = mbar_wait(&sh.s_full[w], (done + j) & 1);
                tc_fence_after();
                if (masked) {
                    // V rows that some row does not see must not reach it: 0 times an infinity or a NaN is none. What lies outside
                    // of the keys is cleared (boxes without any are zeros), and what not all rows see where it is not finite,
                    // which then spoils the rows that do. Rows [a0, a1) and [b0, b1) of the chunk, 16 bytes a thread.
                    constexpr int PPR = D / 8;
                    const int box = a.box_rows ? a.box_rows : 1;
                    auto in_chunk = [&](int t) { return min(max(t - t0, 0), kSKeys); };
                    const int a0 = in_chunk(kv_lo & -box), a1 = max(a0, in_chunk(all_lo)), b0 = max(a1, in_chunk(all_hi));
                    const int rows_a = a1 - a0, rows = rows_a + max(0, in_chunk((kv_end + box - 1) & -box) - b0);
                    if (rows > 0) {
                        const int st = Q::DEPTH + c % Q::DEPTH;
                        uint32_t(&found)[2][2][4] = sh.bad[wide];
                        const uint32_t turn = looks >> (wide ? 1 : 0) & 1;
                        looks ^= wide ? 2u : 1u;
                        if (ok) ok = mbar_wait(&sh.full[st], filling(c) & 1);
                        bool wrote = false;
                        for (int i = wide ? tid : m; i < rows * PPR; i += wide ? 256 : 128) {
                            const int r = i / PPR, row = r < rows_a ? a0 + r : b0 + r - rows_a, t = t0 + row, k = i % PPR;
                            const uint32_t at = kv_s + st * Q::SLOT + k / 8 * (kSKeys * 128) + line_offset(row, k % 8 * 16, 128);
                            uint4 u;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "r"(at));
                            const bool in = t >= kv_lo && t < kv_end, bad = in && not_finite8<T>(u);
                            if (!in || bad) {
                                asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
                                wrote = true;
                            }
                            if (bad) atomicOr(&found[turn][w][row / 32], 1u << row % 32);
                        }
                        if (wrote) fence_async_smem();
                        if (wide)
                            named_bar_sync(2, 256);
                        else if (w == 0)
                            named_bar_sync(3, 128);
                        else
                            named_bar_sync(4, 128);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const uint32_t b = found[turn][w][k] | (wide ? found[turn][1 - w][k] : 0u);
                            if (b) poisoned |= (b & seen_bits(see_lo - t0 - 32 * k, see_hi - t0 - 32 * k)) != 0;
                        }
                        // Marks stand for this chunk's keys alone. Those of the chunk that was looked at before, by the same
                        // threads, were read by all of them before they came here; a turn is a chunk that is looked at, not a
                        // step, of which others lie between and of which the warpgroups can have done different numbers.
                        if (m < 4) found[1 - turn][w][m] = 0;
                    }
                }
                if (live) {
                    // 32 keys at a time, in loops that stay loops: unrolled, a piece's first step waited 6,000 clocks for its
                    // own instructions
                    float mx = -INFINITY;
#pragma unroll 1
                    for (int k0 = 0; k0 < kSKeys; k0 += 64) {
                        float s[64];
                        tmem_get32(s_t + k0, s);
                        tmem_get32(s_t + k0 + 32, s + 32);
                        tmem_wait_ld();
                        tmem_pass32(s);
                        tmem_pass32(s + 32);
                        if constexpr (EXTRA) {
                            // in log2 units. Caps of up to 64 by cap tanh(z / cap) = cap (1 - 2 / (1 + 2^(2 log2(e) z / cap))), whose
                            // error is 2^-21 of the cap, 2^-15 at most: twice as far off as p's planes. Larger ones by a form
                            // whose error goes with z instead (16 sequences of 512 to 4,096 keys 48 us, 57 by it).
                            if (a.cap2 > 64.f * 1.4426950408889634f) {
#pragma unroll
                                for (int k = 0; k < 64; k += 2) {
                                    const float2 z = cap_tanh(__fmul2_rn(make_float2(s[k], s[k + 1]), make_float2(a.to_u, a.to_u)), a.cap2);
                                    s[k] = z.x, s[k + 1] = z.y;
                                }
                            } else if (a.cap2 > 0.f) {
                                const float up = a.to_u * (2.f * 1.4426950408889634f);
#pragma unroll
                                for (int k = 0; k < 64; ++k) s[k] = a.cap2 - __fdividef(2.f * a.cap2, 1.f + ex2(s[k] * up));
                            } else {
#pragma unroll
                                for (int k = 0; k < 64; ++k) s[k] *= a.scale_log2;
                            }
                            if (a.slopes) {
                                const float away = static_cast<float>(t0 + k0 - pos);
#pragma unroll
                                for (int k = 0; k < 64; ++k) s[k] = fmaf(slope2, away + k, s[k]);
                            }
                        }
                        if (masked) {
#pragma unroll
                            for (int h = 0; h < 64; h += 32) {
                                const uint32_t seen = seen_bits(see_lo - t0 - k0 - h, see_hi - t0 - k0 - h);
#pragma unroll
                                for (int k = 0; k < 32; ++k) s[h + k] = seen & (1u << k) ? s[h + k] : -INFINITY;
                            }
                        }
                        if (EXTRA || masked) {
                            tmem_put32(s_t + k0, s);
                            tmem_put32(s_t + k0 + 32, s + 32);
                        }
                        float t[4] = {mx, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int k = 0; k < 64; k += 8)
#pragma unroll
                            for (int u = 0; u < 4; ++u) t[u] = max3(t[u], s[k + 2 * u], s[k + 2 * u + 1]);
                        mx = fmaxf(max3(t[0], t[1], t[2]), t[3]);
                    }
                    if (EXTRA || masked) tmem_wait_st();
                    if constexpr (!EXTRA) mx *= a.scale_log2;
                    mx = fmaxf(mx, kQNoRef);
                    if (j == 0) {
                        M = mx;
                    } else if (__any_sync(0xffffffffu, mx > M + kSGrow)) {
                        // the reference moves: what O and l hold is brought to the new one
                        if (ok) ok = mbar_wait(&sh.o_done[w], (done + j - 1) & 1);
                        tc_fence_after();
                        const bool moves = mx > M + kSGrow;
                        const float f = moves ? ex2(M - mx) : 1.f;
                        if (moves) M = mx;
                        l2.x *= f, l2.y *= f;
#pragma unroll 1
                        for (int k = 0; k < D; k += 32) {
                            float o[32];
                            tmem_get32(o_t + k, o);
                            tmem_wait_ld();
                            tmem_pass32(o);
#pragma unroll
                            for (int d = 0; d < 32; ++d) o[d] *= f;
                            tmem_put32(o_t + k, o);
                        }
                        tmem_wait_st();
                    }
                    const float neg = Q::BIAS - M, unit = EXTRA ? 1.f : a.scale_log2;
                    float s[2][32];
                    tmem_get32(s_t, s[0]);
#pragma unroll 1
                    for (int k0 = 0; k0 < kSKeys; k0 += 64) {  // the probabilities take their scores' columns
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t hi[16], lo[16];
                            tmem_wait_ld();
                            tmem_pass32(s[h]);
                            if (h == 0 || k0 == 0) tmem_get32(s_t + k0 + 32 * h + 32, s[1 - h]);  // the next ones, meanwhile
#pragma unroll
                            for (int u = 0; u < 16; ++u) {
                                const float2 e = __ffma2_rn(make_float2(s[h][2 * u], s[h][2 * u + 1]), make_float2(unit, unit), make_float2(neg, neg));
                                const float2 pr = make_float2(ex2(e.x), ex2(e.y));
                                l2 = __fadd2_rn(l2, pr);
                                split_p<T>(pr, hi[u], lo[u]);
                            }
                            tmem_put16(s_t + k0 + 32 * h, hi);
                            tmem_put16(s_t + k0 + 32 * h + 16, lo);
                        }
                        if (k0 == 0) {  // the products with these 64 keys can begin
                            tmem_wait_st();
                            tc_fence_before();
                            mbar_arrive(&sh.p_half[w]);
                        }
                    }
                    tmem_wait_st();
                } else {
                    mbar_arrive(&sh.p_half[w]);
                }
                tc_fence_before();
                mbar_arrive(&sh.p_full[w]);
            }
            done += steps;
            next_piece(n);
            SPiece after = p;
            more = shared_next(a, pl, x, x1, after);
            if (more) load_q(after);
            // ---- results: both warpgroups' columns of their own rows, or half of the columns each of the rows they share
            if (steps > 0 && ok) ok = mbar_wait(&sh.o_done[w], (done - 1) & 1);
            tc_fence_after();
            if (!ok && lane == 0) set_status(a.status, SDV_ERR_DEVICE_TIMEOUT);
            float l = poisoned ? NAN : l2.x + l2.y, f0 = 1.f, f1 = 0.f;
            if (!wide) {
                if (steps > 0) sh.ml[w][m] = make_float2(M, l);
                tc_fence_before();
                named_bar_sync(1, 256);
                tc_fence_after();
                const float2 x0 = sh.ml[0][m], x1 = n > 1 ? sh.ml[1][m] : make_float2(kQNoRef, 0.f);
                M = fmaxf(x0.x, x1.x);
                f0 = ex2(x0.x - M);
                f1 = ex2(x1.x - M);
                l = f0 * x0.y + f1 * x1.y;
            }
            const SPiece here = p;
            p = after;
            if (!live) continue;
            // the whole of its rows' keys: the result; else a part of it
            const bool direct = n == en.nc && !prefix && (en.group < 0 || pl.e[en.group].nc == 0), mine = m < n_rows;
            const int cols = wide ? D : D / 2, col0 = wide ? 0 : w * (D / 2);
            const long long slot = shared_slot(a, prefix, r00, here.h, here.tile, here.c0 > 0 ? cta : -1) + row0;
            if (!direct && mine && (wide || w == 0)) a.part_ml[slot + m] = make_float2(M, l);
            const float inv = direct ? 1.f / l : 1.f;
            f0 *= inv, f1 *= inv;
            T *out = static_cast<T *>(a.out) + row * a.out_stride + hq * D + col0;
            float *part = a.part_o + (slot + m) * D + col0;
#pragma unroll 1
            for (int k = 0; k < cols; k += 32) {
                float o[32];
                __syncwarp();
                tmem_get32((wide ? o_t : tmem + lanes + Q::O_COL) + col0 + k, o);
                tmem_wait_ld();
                tmem_pass32(o);
#pragma unroll
                for (int d = 0; d < 32; ++d) o[d] *= f0;
                if (!wide && n > 1) {
                    float v[32];
                    tmem_get32(tmem + lanes + Q::O_COL + 128 + col0 + k, v);
                    tmem_wait_ld();
                    tmem_pass32(v);
#pragma unroll
                    for (int d = 0; d < 32; ++d) o[d] = fmaf(f1, v[d], o[d]);
                }
                if (!mine) continue;
                if (!direct) {
#pragma unroll
                    for (int d = 0; d < 32; d += 8) store8(part + k + d, o + d);
                } else if (a.out_vec) {
#pragma unroll
                    for (int d = 0; d < 32; d += 8)
                        *reinterpret_cast<uint4 *>(out + k + d) = make_uint4(pack16<T>(o[d], o[d + 1]), pack16<T>(o[d + 2], o[d + 3]),
                                                                             pack16<T>(o[d + 4], o[d + 5]), pack16<T>(o[d + 6], o[d + 7]));
                } else {
#pragma unroll
                    for (int d = 0; d < 32; ++d) out[k + d] = from_f32<T>(o[d]);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 10) tmem_dealloc(tmem, 512);
}

// ------------------------------------------------------------------ joining the parts
constexpr int kSMergeThreads = 256;

// A warp joins the parts of one (row, q head): those of its own tile, then those of the prefix's, CTA by CTA along the line.
// Rows that one piece holds alone were written by the attention, those of refused spans become NaN. Eight parts are on their way
// at once (sixteen were slower: registers); 4 us for few rows, most of it three loads that wait for one another.
template <typename T, int D>
__global__ void __launch_bounds__(kSMergeThreads, 3) shared_merge_kernel(const __grid_constant__ SharedArgs a) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x % 32, idx = blockIdx.x * (kSMergeThreads / 32) + threadIdx.x / 32;
    pdl_wait();  // in every CTA: this kernel's end stands for the attention's, too
    pdl_trigger();
    const int row = a.by_nq.div(idx), hq = idx - row * a.nq, h = a.by_grp.div(hq);
    if (row >= a.max_rows) return;
    const int2 of = a.row_entry[row], cut = *a.plan_cut;
    const FastDiv by_cut = *a.by_cut;
    if (of.x == kRowNone) return;
    T *out = static_cast<T *>(a.out) + row * a.out_stride + hq * D + lane * V;
    if (of.x == kRowRefused) {
#pragma unroll
        for (int d = 0; d < V; ++d) out[d] = from_f32<T>(NAN);
        return;
    }
    // of the row's own tile and of the prefix's: start on the line, the CTA that it begins in and the number of those it
    // touches, and the row's place in the partial results that begin with the tile, and in those of a CTA
    int4 e[2];
    int at[2], i0[2], n[2], r[2];
    long long slot0[2];
    const long long side = static_cast<long long>(a.nkv) * a.part_rows;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        n[k] = 0;
        const int at_entry = k ? of.y : of.x;
        if (at_entry < 0) continue;
        e[k] = a.plan[at_entry];
        const int2 rows = a.plan_rows[at_entry];
        const int m = (row - rows.x) * a.grp + hq - h * a.grp, tile = m / kSTile;
        r[k] = m - tile * kSTile;
        slot0[k] = k * side + static_cast<long long>(h) * a.part_rows + rows.x * a.grp + m;
        at[k] = e[k].x + (h * rows.y + tile) * e[k].y;
        i0[k] = by_cut.div(at[k]);
        n[k] = by_cut.div(at[k] + e[k].y - 1) - i0[k] + 1;
    }
    const int n_own = n[0], n_pre = n[1];
    // row of part k in the partial results, -1 where that CTA has no chunk of the tile
    auto part = [&](int k) -> long long {
        if (k >= n_own + n_pre) return -1;
        const bool p = k >= n_own;
        const int4 t = p ? e[1] : e[0];
        const int i = p ? i0[1] + k - n_own : i0[0] + k, rel = i * cut.x - (p ? at[1] : at[0]);
        const int from = shared_chunk(t.z, t.w, cut.y, rel), stop = rel + cut.x >= t.y ? t.z : shared_chunk(t.z, t.w, cut.y, rel + cut.x);
        if (stop <= from) return -1;
        return from > 0 ? 2 * side + static_cast<long long>(i) * kSTile + (p ? r[1] : r[0]) : p ? slot0[1] : slot0[0];
    };
    const int count = n_own + n_pre;
    long long slot = part(lane);
    if (n_pre == 0 && n_own <= 32 && __popc(__ballot_sync(0xffffffffu, slot >= 0)) == 1) return;  // written already
    // eight parts' values on their way at once, the first beside their maxima
    constexpr int N = 8;
    float v[N][V];
    auto ask = [&](int p0) {
#pragma unroll
        for (int u = 0; u < N; ++u) {
            const long long s = __shfl_sync(0xffffffffu, slot, p0 + u);
#pragma unroll
            for (int d = 0; d < V; ++d) v[u][d] = 0.f;
            if (s >= 0) {
                const float *src = a.part_o + s * D + lane * V;
                if constexpr (V == 4)
                    *reinterpret_cast<float4 *>(v[u]) = *reinterpret_cast<const float4 *>(src);
                else
                    *reinterpret_cast<float2 *>(v[u]) = *reinterpret_cast<const float2 *>(src);
            }
        }
    };
    float2 ml = slot >= 0 ? a.part_ml[slot] : make_float2(kQNoRef, 0.f);
    ask(0);
    float M = ml.x;
    for (int k = 32 + lane; k - lane < count; k += 32) {
        const long long s = part(k);
        if (s >= 0) M = fmaxf(M, a.part_ml[s].x);
    }
    M = redux_max(M);
    float o[V], l = 0.f;
#pragma unroll
    for (int d = 0; d < V; ++d) o[d] = 0.f;
    for (int k0 = 0; k0 < count; k0 += 32) {
        if (k0 > 0) {
            slot = part(k0 + lane);
            ml = slot >= 0 ? a.part_ml[slot] : make_float2(kQNoRef, 0.f);
        }
        const float mine = slot >= 0 ? ex2(ml.x - M) : 0.f;
        l += warp_sum(slot >= 0 ? mine * ml.y : 0.f);
#pragma unroll 1
        for (int p0 = 0; p0 < min(32, count - k0); p0 += N) {
            if (k0 + p0 > 0) ask(p0);
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const float f = __shfl_sync(0xffffffffu, mine, p0 + u);
#pragma unroll
                for (int d = 0; d < V; ++d) o[d] = fmaf(f, v[u][d], o[d]);
            }
        }
    }
    const float inv = 1.f / l;
#pragma unroll
    for (int d = 0; d < V; ++d) out[d] = from_f32<T>(o[d] * inv);
}

}  // namespace sdv
