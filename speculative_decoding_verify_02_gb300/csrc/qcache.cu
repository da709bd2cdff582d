// C ABI of the 8-bit KV cache: quantising rows as they are written, reading them back, and attention
// over the codes.
#include <algorithm>
#include <cmath>
#include <new>
#include <vector>

#include "qcache_attention.cuh"

using namespace sdv;

struct sdv_qcache {
    sdv_qcache_cfg c{};
    int device = 0, sm_count = 0, pages_per_seq = 0;
    uint8_t *codes = nullptr;
    float *scales = nullptr;
    uint8_t *ws = nullptr;
    size_t layer_codes = 0, layer_scales = 0;
    FastDiv by_page{}, by_block{}, by_heads{};
    int box_rows = 0;                 // pool rows of a TMA box (0: the page size fits none)
    std::vector<CUtensorMap> pools;   // one map a layer over its pool rows
    int clusters[kQJoin + 1] = {};    // clusters of 2..kQJoin attention CTAs of 64 rows that the device holds at once
};

namespace {

constexpr int kQWaves = 4;       // turns of the CTAs that an attention is cut into at most
constexpr double kQMerge = .5;   // what a merge kernel costs over a cluster's joining, in chunks
constexpr double kQTurn = 4;     // what a unit costs besides its chunks, in chunks (16 ragged sequences: 46 us with 1, 38 with 4)

int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

int check_cfg(const sdv_qcache_cfg *c) {
    if (!c) return SDV_ERR_ARG;
    if (c->n_layers <= 0 || c->n_q_heads <= 0 || c->n_kv_heads <= 0 || c->n_q_heads % c->n_kv_heads) return SDV_ERR_ARG;
    if (c->page_size <= 0 || c->n_pages <= 0 || c->scale_block <= 0 || c->page_size % c->scale_block)
        return SDV_ERR_ARG;
    if (c->max_batch <= 0 || c->max_batch > 256 || c->max_rows <= 0 || c->max_span <= 0 ||
        c->max_span > c->max_rows || c->max_context < c->max_span)
        return SDV_ERR_ARG;
    if (c->head_dim != 64 && c->head_dim != 128) return SDV_ERR_UNSUPPORTED;
    // a row of the layer's pool is indexed in 32 bits
    if (static_cast<double>(c->n_pages) * 2 * c->n_kv_heads * c->page_size > 4294967294.0) return SDV_ERR_UNSUPPORTED;
    if (c->n_q_heads > 1024 || c->max_rows > (1 << 20) || c->max_context > (1 << 30) || c->page_size > (1 << 20))
        return SDV_ERR_UNSUPPORTED;
    return SDV_OK;
}

size_t layer_codes(const sdv_qcache_cfg &c) {
    return static_cast<size_t>(c.n_pages) * 2 * c.n_kv_heads * c.page_size * c.head_dim;
}
size_t layer_scales(const sdv_qcache_cfg &c) {
    return static_cast<size_t>(c.n_pages) * 2 * c.n_kv_heads * (c.page_size / c.scale_block);
}

// Rows of a TMA box: the largest power of two up to a chunk that divides the page size, from eight (a swizzle atom).
int box_rows_of(const sdv_qcache_cfg &c) {
    if (static_cast<long long>(c.n_pages) * 2 * c.n_kv_heads * c.page_size >= (1ll << 31)) return 0;  // box rows are int
    int r = 1;
    while (r < kQKeys && c.page_size % (2 * r) == 0) r *= 2;
    return r >= 8 ? r : 0;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// A layer's pool as [row][D] bytes; a box is box_rows rows, with the swizzle of their width.
bool encode_pool_rows(CUtensorMap *tm, void *codes, const sdv_qcache_cfg &c, int box_rows) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return false;
    const cuuint64_t D = c.head_dim;
    cuuint64_t dims[2] = {D, static_cast<cuuint64_t>(c.n_pages) * 2 * c.n_kv_heads * c.page_size}, strides[1] = {D};
    cuuint32_t box[2] = {static_cast<cuuint32_t>(D), static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
    return reinterpret_cast<EncodeTiledFn>(fn)(tm, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, codes, dims, strides, box, es,
                                               CU_TENSOR_MAP_INTERLEAVE_NONE,
                                               D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... KArgs, typename... Args>
int launch_clusters(void (*kern)(KArgs...), int cluster, dim3 grid, dim3 block, size_t smem, void *stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {static_cast<unsigned>(cluster), 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? SDV_OK : SDV_ERR_CUDA;
}
template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, void *stream, Args &&...args) {
    return launch_clusters(kern, 1, grid, block, smem, stream, std::forward<Args>(args)...);
}

// Arguments that every call shares, checked; SDV_OK and the kernels' block, or the error.
int common_args(const sdv_qcache *q, int layer, int rows, const int32_t *table, const int32_t *row_off,
                const int32_t *base, int B, int max_span, QCacheArgs *a) {
    if (!q || !table || !row_off || !base || layer < 0 || layer >= q->c.n_layers || rows <= 0 || B <= 0 || B > q->c.max_batch ||
        max_span <= 0 || max_span > q->c.max_span)
        return SDV_ERR_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != q->device) return SDV_ERR_ARG;
    a->codes = q->codes + q->layer_codes * layer;
    a->scales = q->scales + q->layer_scales * layer;
    a->status = reinterpret_cast<int *>(q->ws);
    a->page_table = table;
    a->row_off = row_off;
    a->base = base;
    a->pages_per_seq = q->pages_per_seq;
    a->page_size = q->c.page_size;
    a->n_pages = q->c.n_pages;
    a->scale_block = q->c.scale_block;
    a->nkv = q->c.n_kv_heads;
    a->B = B;
    a->max_span = max_span;
    a->max_rows = std::min(rows, q->c.max_rows);
    a->max_context = q->c.max_context;
    a->by_page = q->by_page;
    a->by_block = q->by_block;
    a->by_heads = q->by_heads;
    a->blocks = q->c.page_size / q->c.scale_block;
    return SDV_OK;
}

size_t dtype_size(int dtype) { return dtype == SDV_FP32 ? 4 : 2; }
bool aligned16(const void *p, int64_t stride, int dtype) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * static_cast<int64_t>(dtype_size(dtype)) % 16 == 0;
}
bool element_aligned(const void *p, int dtype) { return reinterpret_cast<uintptr_t>(p) % dtype_size(dtype) == 0; }

// ---- attention: tile rows, parts of a sequence and workspace
// Rows of a tile: 16, 32 or 64, the smallest that holds a span's rows of one kv head. Long spans read every key once a
// tile, out of L2: with tiles of 32 rows, two CTAs an SM waited for keys a third of the time (128 rows at 32K: 240 us
// against 212 with 64, now 193).
int attn_rows(int span_rows) { return span_rows <= 16 ? 16 : span_rows <= 32 ? 32 : 64; }

struct AttnPlan {
    int rows, tiles, splits, ctas;
    bool cluster;  // a tile's parts are a cluster
};
AttnPlan attn_plan(const sdv_qcache *q, int B, int max_span, int window) {
    AttnPlan p;
    const int span_rows = max_span * (q->c.n_q_heads / q->c.n_kv_heads);
    p.rows = attn_rows(span_rows);
    p.tiles = cdiv(span_rows, p.rows);
    p.ctas = (p.rows == 64 ? 1 : 2) * q->sm_count;
    // Parts: the number that the CTAs get through soonest at the cache's full context (16 x 8 rows of 4,096 keys take 42.3 us
    // in a cache of 4,104 positions, two parts, and 63.8 in one of 32,776, nine); a unit costs its chunks and about
    // kQTurn more for its queries, first maximum and results. One sequence's units are alike and go in turns; a batch's
    // differ, so that past one turn a CTA has its share of the work (of sequences 0.6 of the longest on average) and
    // then waits for the longest unit. Parts that no cluster joins cost a kernel more. What a sequence's parts are depends on its own length and on this number only.
    const long long units = static_cast<long long>(B) * q->c.n_kv_heads * p.tiles;
    const int keys = window > 0 ? std::min(q->c.max_context, window + max_span) : q->c.max_context;
    const int chunks = cdiv(keys, kQKeys);
    double best = 0;
    p.splits = 1;
    p.cluster = false;
    for (int s = 1; s <= chunks && units * s <= static_cast<long long>(kQWaves) * p.ctas; ++s) {
        const double unit = cdiv(chunks, s) + kQTurn;
        double t = B == 1 || units * s <= p.ctas ? static_cast<double>((units * s + p.ctas - 1) / p.ctas) * unit
                                : units * (0.6 * chunks + s * kQTurn) / p.ctas + unit;
        const bool cluster = s > 1 && s <= kQJoin && units * s <= p.ctas && (p.rows < 64 || units <= q->clusters[s]);
        if (s > 1 && !cluster) t += kQMerge;
        if (s == 1 || t < best) best = t, p.splits = s, p.cluster = cluster;
    }
    return p;
}

// Floats of attention's partial results: rows x heads x splits of the largest call, D + 2 each. splits >= 2 only
// while B nkv tiles splits <= 2 SMs x waves, and a tile holds at most 64 rows (of half as many CTAs).
size_t attn_partials(const sdv_qcache_cfg &c, int sm_count) {
    const size_t all = static_cast<size_t>(c.max_batch) * c.max_span * c.n_q_heads * cdiv(c.max_context, kQKeys);
    const size_t cut = static_cast<size_t>(2) * sm_count * kQWaves * 32;
    return std::min(all, cut);
}

template <typename T, int D, int ROWS>
int launch_attn_rows(const CUtensorMap &pool, const QAttnArgs &a, const AttnPlan &p, void *stream) {
    typedef QTile<T, D, ROWS> Q;
    const dim3 grid(static_cast<unsigned>(std::min(a.units, p.ctas)));
    const int r = launch_clusters(qcache_attn_kernel<T, D, ROWS>, a.cluster ? p.splits : 1, grid, Q::THREADS, Q::SMEM,
                                  stream, pool, a);
    if (r != SDV_OK || p.splits == 1 || a.cluster) return r;
    const long long items = static_cast<long long>(a.c.max_span) * a.nq;
    if (p.splits <= kQJoin)
        return launch(qcache_merge_kernel<T, D, 1>, dim3(cdiv(items, 4), a.c.B), kQMergeThreads, 0, stream, a);
    return launch(qcache_merge_kernel<T, D, 4>, dim3(static_cast<unsigned>(items), a.c.B), kQMergeThreads, 0, stream, a);
}
template <typename T, int D>
int launch_attn(const CUtensorMap &pool, const QAttnArgs &a, const AttnPlan &p, void *stream) {
    if (p.rows == 16) return launch_attn_rows<T, D, 16>(pool, a, p, stream);
    if (p.rows == 64) return launch_attn_rows<T, D, 64>(pool, a, p, stream);
    return launch_attn_rows<T, D, 32>(pool, a, p, stream);
}

// Every kernel asks for the largest shared-memory carveout: an SM that changes it between an attention and its merge
// drains first, and with the default one attention CTA fits instead of two.
template <typename K>
cudaError_t set_carveout(K kern) {
    return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
}
template <typename T, int D, int ROWS>
cudaError_t set_attn() {
    cudaError_t e = cudaFuncSetAttribute(qcache_attn_kernel<T, D, ROWS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         QTile<T, D, ROWS>::SMEM);
    return e == cudaSuccess ? set_carveout(qcache_attn_kernel<T, D, ROWS>) : e;
}
// Clusters of each size that run at once, of CTAs that fill an SM: their SMs must be neighbours (15 clusters of eight
// on 152 SMs), and one that waits costs a whole turn (two sequences of 8,164 keys and 14 rows: 50 us, 28 without). Of
// smaller CTAs two share an SM, and those over start soon (four sequences of 1,000 keys and 8 rows, 32 clusters of
// eight: 11.4 us, 12.5 without).
cudaError_t count_clusters(int (&n)[kQJoin + 1]) {
    typedef QTile<bf16, 128, 64> Q;  // the other types fill an SM, too
    for (int s = 2; s <= kQJoin; ++s) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(s);
        cfg.blockDim = dim3(Q::THREADS);
        cfg.dynamicSmemBytes = Q::SMEM;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim = {static_cast<unsigned>(s), 1, 1};
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&n[s], qcache_attn_kernel<bf16, 128, 64>, &cfg);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}
template <typename T, int D>
cudaError_t set_attn_all() {
    cudaError_t e = set_carveout(qcache_merge_kernel<T, D, 1>);
    if (e == cudaSuccess) e = set_carveout(qcache_merge_kernel<T, D, 4>);
    if (e == cudaSuccess) e = set_attn<T, D, 16>();
    if (e == cudaSuccess) e = set_attn<T, D, 32>();
    if (e == cudaSuccess) e = set_attn<T, D, 64>();
    return e;
}

template <typename T, int D>
int write_rows(const QCacheArgs &a, const void *k, int64_t ks, const void *v, int64_t vs, bool vec, void *stream) {
    constexpr int kWindow = kQHold * 32 / (D / 8);
    const bool small = a.scale_block < 16 && (a.scale_block & (a.scale_block - 1)) == 0;
    const int unit = small ? kWindow : a.scale_block;  // tokens of a warp
    const int units = (a.max_span + unit - 2) / unit + 1;  // a span touches at most
    const dim3 grid(cdiv(static_cast<long long>(units) * 2 * a.nkv, kQWriteThreads / 32), a.B);
    const T *kp = static_cast<const T *>(k), *vp = static_cast<const T *>(v);
    const long long k_stride = ks, v_stride = vs;
    auto *kern = small ? (vec ? qcache_write_small_kernel<T, D, true> : qcache_write_small_kernel<T, D, false>)
                       : (vec ? qcache_write_kernel<T, D, true> : qcache_write_kernel<T, D, false>);
    return launch(kern, grid, kQWriteThreads, 0, stream, a, kp, vp, k_stride, v_stride);
}

template <typename T, int D>
int read_rows(const QCacheArgs &a, void *k, int64_t ks, void *v, int64_t vs, bool vec, void *stream) {
    const dim3 grid(2 * a.nkv, cdiv(a.max_span, kQReadThreads / (D / 8) * kQReadRows), a.B);
    T *kp = static_cast<T *>(k), *vp = static_cast<T *>(v);
    const long long k_stride = ks, v_stride = vs;
    return vec ? launch(qcache_read_kernel<T, D, true>, grid, kQReadThreads, 0, stream, a, kp, vp, k_stride, v_stride)
               : launch(qcache_read_kernel<T, D, false>, grid, kQReadThreads, 0, stream, a, kp, vp, k_stride, v_stride);
}

}  // namespace

extern "C" {

int sdv_qcache_bytes(const sdv_qcache_cfg *cfg, size_t *codes, size_t *scales, size_t *workspace) {
    const int r = check_cfg(cfg);
    if (r) return r;
    if (!codes || !scales || !workspace) return SDV_ERR_ARG;
    *codes = layer_codes(*cfg) * cfg->n_layers;
    *scales = layer_scales(*cfg) * cfg->n_layers * sizeof(float);
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess)
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    else
        cudaGetLastError();  // no device to ask: the part's 152
    const size_t slots = attn_partials(*cfg, sms);
    *workspace = 256 + slots * sizeof(float2) / 256 * 256 + 256 + slots * cfg->head_dim * sizeof(float);
    return SDV_OK;
}

int sdv_qcache_create(const sdv_qcache_cfg *cfg, void *d_codes, void *d_scales, void *d_workspace, void *stream,
                      sdv_qcache **out) {
    const int r = check_cfg(cfg);
    if (r) return r;
    if (!d_codes || !d_scales || !d_workspace || !out) return SDV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(d_codes) % 16 || reinterpret_cast<uintptr_t>(d_scales) % 16 ||
        reinterpret_cast<uintptr_t>(d_workspace) % 256)
        return SDV_ERR_ARG;
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SDV_ERR_CUDA;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, qcache_write_kernel<bf16, 128, true>) != cudaSuccess) {
        cudaGetLastError();
        return SDV_ERR_UNSUPPORTED;  // no sm_103a image for this device
    }
    if (set_attn_all<bf16, 128>() != cudaSuccess || set_attn_all<bf16, 64>() != cudaSuccess ||
        set_attn_all<__half, 128>() != cudaSuccess || set_attn_all<__half, 64>() != cudaSuccess)
        return SDV_ERR_CUDA;
    sdv_qcache *q = new (std::nothrow) sdv_qcache();
    if (!q) return SDV_ERR_ARG;
    q->c = *cfg;
    q->device = dev;
    q->sm_count = sms;
    q->pages_per_seq = cdiv(cfg->max_context, cfg->page_size);
    q->codes = static_cast<uint8_t *>(d_codes);
    q->scales = static_cast<float *>(d_scales);
    q->ws = static_cast<uint8_t *>(d_workspace);
    q->layer_codes = layer_codes(*cfg);
    q->layer_scales = layer_scales(*cfg);
    q->by_page = FastDiv::of(cfg->page_size);
    q->by_block = FastDiv::of(cfg->scale_block);
    q->by_heads = FastDiv::of(2 * cfg->n_kv_heads);
    q->box_rows = box_rows_of(*cfg);
    if (count_clusters(q->clusters) != cudaSuccess) {
        delete q;
        return SDV_ERR_CUDA;
    }
    bool maps = true;
    try {
        q->pools.resize(cfg->n_layers);
        for (int l = 0; l < cfg->n_layers && q->box_rows && maps; ++l)
            maps = encode_pool_rows(&q->pools[l], q->codes + q->layer_codes * l, *cfg, q->box_rows);
    } catch (const std::bad_alloc &) {
        maps = false;
    }
    if (!maps) {
        delete q;
        return SDV_ERR_CUDA;
    }
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    cudaError_t e = cudaMemsetAsync(q->codes, 0, q->layer_codes * cfg->n_layers, st);
    if (e == cudaSuccess) e = cudaMemsetAsync(q->scales, 0, q->layer_scales * cfg->n_layers * sizeof(float), st);
    if (e == cudaSuccess) e = cudaMemsetAsync(q->ws, 0, 256, st);
    if (e != cudaSuccess) {
        delete q;
        return SDV_ERR_CUDA;
    }
    *out = q;
    return SDV_OK;
}

int sdv_qcache_destroy(sdv_qcache *cache) {
    delete cache;
    return SDV_OK;
}

int sdv_qcache_write(sdv_qcache *cache, int layer, const void *d_k, int64_t k_stride, const void *d_v, int64_t v_stride,
                     int dtype, int rows, const int32_t *d_page_table, const int32_t *d_row_off, const int32_t *d_base, int B,
                     int max_span, void *stream) {
    QCacheArgs a{};
    const int r = common_args(cache, layer, rows, d_page_table, d_row_off, d_base, B, max_span, &a);
    if (r) return r;
    const int D = cache->c.head_dim, width = cache->c.n_kv_heads * D;
    if (dtype != SDV_BF16 && dtype != SDV_FP16 && dtype != SDV_FP32) return SDV_ERR_UNSUPPORTED;
    if (!d_k || !d_v || k_stride < width || v_stride < width || !element_aligned(d_k, dtype) ||
        !element_aligned(d_v, dtype))
        return SDV_ERR_ARG;
    const bool vec = aligned16(d_k, k_stride, dtype) && aligned16(d_v, v_stride, dtype);
#define SDV_QWRITE(T)                                                                     \
    return D == 128 ? write_rows<T, 128>(a, d_k, k_stride, d_v, v_stride, vec, stream) \
                    : write_rows<T, 64>(a, d_k, k_stride, d_v, v_stride, vec, stream)
    if (dtype == SDV_BF16) SDV_QWRITE(bf16);
    if (dtype == SDV_FP16) SDV_QWRITE(__half);
    SDV_QWRITE(float);
#undef SDV_QWRITE
}

int sdv_qcache_read(sdv_qcache *cache, int layer, const int32_t *d_page_table, const int32_t *d_row_off,
                    const int32_t *d_base, int B, int max_span, void *d_k, int64_t k_stride, void *d_v,
                    int64_t v_stride, int dtype, int rows, void *stream) {
    QCacheArgs a{};
    const int r = common_args(cache, layer, rows, d_page_table, d_row_off, d_base, B, max_span, &a);
    if (r) return r;
    const int D = cache->c.head_dim, width = cache->c.n_kv_heads * D;
    if (dtype != SDV_BF16 && dtype != SDV_FP16 && dtype != SDV_FP32) return SDV_ERR_UNSUPPORTED;
    if (!d_k || !d_v || k_stride < width || v_stride < width || !element_aligned(d_k, dtype) ||
        !element_aligned(d_v, dtype))
        return SDV_ERR_ARG;
    const bool vec = aligned16(d_k, k_stride, dtype) && aligned16(d_v, v_stride, dtype);
#define SDV_QREAD(T)                                                                     \
    return D == 128 ? read_rows<T, 128>(a, d_k, k_stride, d_v, v_stride, vec, stream) \
                    : read_rows<T, 64>(a, d_k, k_stride, d_v, v_stride, vec, stream)
    if (dtype == SDV_BF16) SDV_QREAD(bf16);
    if (dtype == SDV_FP16) SDV_QREAD(__half);
    SDV_QREAD(float);
#undef SDV_QREAD
}

int sdv_qcache_attention(sdv_qcache *cache, int layer, const void *d_q, int64_t q_stride, int dtype, int rows,
                         const int32_t *d_page_table, const int32_t *d_row_off, const int32_t *d_base, int B,
                         int max_span, int window, void *d_out, int64_t out_stride, void *stream) {
    QAttnArgs a{};
    const int r = common_args(cache, layer, rows, d_page_table, d_row_off, d_base, B, max_span, &a.c);
    if (r) return r;
    const int D = cache->c.head_dim, width = cache->c.n_q_heads * D;
    if (dtype != SDV_BF16 && dtype != SDV_FP16) return SDV_ERR_UNSUPPORTED;
    if (!d_q || !d_out || window < 0 || q_stride < width || out_stride < width || !element_aligned(d_q, dtype) ||
        !element_aligned(d_out, dtype))
        return SDV_ERR_ARG;
    a.q = d_q;
    a.out = d_out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.nq = cache->c.n_q_heads;
    a.window = window = window >= cache->c.max_context ? 0 : window;
    a.q_vec = aligned16(d_q, q_stride, dtype);
    a.scale_log2 = 1.4426950408889634f / std::sqrt(static_cast<float>(D));
    const AttnPlan p = attn_plan(cache, B, max_span, window);
    const size_t slots = attn_partials(cache->c, cache->sm_count);
    a.splits = p.splits;
    a.tiles = p.tiles;
    a.grp = a.nq / a.c.nkv;
    const long long units = static_cast<long long>(B) * p.splits * a.c.nkv * p.tiles;
    if (units > (1 << 30)) return SDV_ERR_UNSUPPORTED;
    a.units = static_cast<int>(units);
    a.cluster = p.cluster;
    a.counter = reinterpret_cast<int *>(cache->ws) + 1;
    a.by_tiles = FastDiv::of(a.tiles);
    a.by_kv = FastDiv::of(a.c.nkv);
    a.by_splits = FastDiv::of(a.splits);
    a.by_grp = FastDiv::of(a.grp);
    a.by_nq = FastDiv::of(a.nq);
    a.part_ml = reinterpret_cast<float2 *>(cache->ws + 256);
    a.part_o = reinterpret_cast<float *>(cache->ws + 512 + slots * sizeof(float2) / 256 * 256);
    a.box_rows = cache->box_rows;
    a.pool_rows = cache->box_rows ? cache->c.n_pages * 2 * a.c.nkv * a.c.page_size : 0;
    const CUtensorMap &pool = cache->pools[layer];
    if (dtype == SDV_BF16)
        return D == 128 ? launch_attn<bf16, 128>(pool, a, p, stream) : launch_attn<bf16, 64>(pool, a, p, stream);
    return D == 128 ? launch_attn<__half, 128>(pool, a, p, stream) : launch_attn<__half, 64>(pool, a, p, stream);
}

int sdv_qcache_get_status(sdv_qcache *cache, int32_t *h_status) {
    if (!cache || !h_status) return SDV_ERR_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return SDV_ERR_CUDA;
    int v = 0;
    const int zero = 0;
    if (cudaMemcpy(&v, cache->ws, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return SDV_ERR_CUDA;
    if (cudaMemcpy(cache->ws, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return SDV_ERR_CUDA;
    *h_status = v;
    return SDV_OK;
}

}  // extern "C"
