// C ABI of the attention for groups of sequences that share a prefix.
#include <algorithm>
#include <cfloat>
#include <cmath>
#include <new>
#include <vector>

#include "shared_attention.cuh"

using namespace sdv;

struct sdv_shared {
    sdv_shared_cfg c{};
    int device = 0, sm_count = 0, pages_per_seq = 0, grp = 0;
    const uint8_t *pool = nullptr;
    uint8_t *ws = nullptr;
    size_t layer_bytes = 0;
    FastDiv by_page{}, by_grp{}, by_nq{};
    int box_rows = 0;                // pool rows of a TMA box (0: the page size fits none)
    std::vector<CUtensorMap> pools;  // one map a layer over its pool rows
};

namespace {

int cdiv(long long a, long long b) { return static_cast<int>((a + b - 1) / b); }

int check_cfg(const sdv_shared_cfg *c) {
    if (!c) return SDV_ERR_ARG;
    if (c->n_layers <= 0 || c->n_q_heads <= 0 || c->n_kv_heads <= 0 || c->n_q_heads % c->n_kv_heads) return SDV_ERR_ARG;
    if (c->page_size <= 0 || c->n_pages <= 0) return SDV_ERR_ARG;
    if (c->max_batch <= 0 || c->max_batch > kSBatch || c->max_rows <= 0 || c->max_span <= 0 || c->max_span > c->max_rows ||
        c->max_context < c->max_span)
        return SDV_ERR_ARG;
    if (c->dtype != SDV_BF16 && c->dtype != SDV_FP16) return SDV_ERR_UNSUPPORTED;
    if (c->head_dim != 64 && c->head_dim != 128) return SDV_ERR_UNSUPPORTED;
    if (c->n_q_heads > 1024 || c->max_rows > (1 << 16) || c->max_context > (1 << 30) || c->page_size > (1 << 20))
        return SDV_ERR_UNSUPPORTED;
    // a row of the layer's pool is an int, as box coordinates are
    if (static_cast<double>(c->n_pages) * 2 * c->n_kv_heads * c->page_size > 2147483000.0) return SDV_ERR_UNSUPPORTED;
    // costs along the line of work are ints: every chunk of every tile of every head
    const double rows = static_cast<double>(c->max_rows) * (c->n_q_heads / c->n_kv_heads);
    const double tiles = (2 * rows / kSTile + c->max_batch + kSGroups) * c->n_kv_heads;
    if (tiles * (2.0 * (c->max_context / kSKeys + 2) + kSOverhead) > 1.0e9) return SDV_ERR_UNSUPPORTED;
    return SDV_OK;
}

size_t layer_bytes(const sdv_shared_cfg &c) {
    return static_cast<size_t>(c.n_pages) * 2 * c.n_kv_heads * c.page_size * c.head_dim * 2;
}
// Rows of a TMA box: the largest power of two up to a chunk that divides the page size, from eight (a swizzle atom).
int box_rows_of(const sdv_shared_cfg &c) {
    int r = 1;
    while (r < kSKeys && c.page_size % (2 * r) == 0) r *= 2;
    return r >= 8 ? r : 0;
}
// Rows of partial results of a kv head, and of all: a row's part of its own tile and of the prefix's, and a tile for each CTA.
int part_rows(const sdv_shared_cfg &c) { return c.max_rows * (c.n_q_heads / c.n_kv_heads); }
size_t part_slots(const sdv_shared_cfg &c, int sms) {
    return static_cast<size_t>(2) * c.n_kv_heads * part_rows(c) + static_cast<size_t>(sms) * kSTile;
}
// Offsets into the workspace: the status word and the cut, the plan's entries, the rows' entries, (M, l), O.
struct Workspace {
    size_t plan, plan_rows, row_entry, ml, o, end;
};
Workspace workspace(const sdv_shared_cfg &c, int sms) {
    auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    Workspace w;
    w.plan = 256;
    w.plan_rows = up(w.plan + sizeof(int4) * kSEntries);
    w.row_entry = up(w.plan_rows + sizeof(int2) * kSEntries);
    w.ml = up(w.row_entry + sizeof(int2) * c.max_rows);
    w.o = up(w.ml + sizeof(float2) * part_slots(c, sms));
    w.end = w.o + sizeof(float) * part_slots(c, sms) * c.head_dim;
    return w;
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
// A layer's pool as [row][D] 16-bit words; a box is 64 columns of box_rows rows, with the swizzle of that width. Its values pass
// through as they are, so one type of map serves both.
bool encode_pool_rows(CUtensorMap *tm, const void *pool, const sdv_shared_cfg &c, int box_rows) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
        return false;
    const cuuint64_t D = c.head_dim;
    cuuint64_t dims[2] = {D, static_cast<cuuint64_t>(c.n_pages) * 2 * c.n_kv_heads * c.page_size}, strides[1] = {2 * D};
    cuuint32_t box[2] = {64, static_cast<cuuint32_t>(box_rows)}, es[2] = {1, 1};
    return reinterpret_cast<EncodeTiledFn>(fn)(tm, CU_TENSOR_MAP_DATA_TYPE_UINT16, 2, const_cast<void *>(pool), dims, strides, box,
                                               es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                                               CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                                               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename... KArgs, typename... Args>
int launch(void (*kern)(KArgs...), dim3 grid, dim3 block, size_t smem, void *stream, Args &&...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = static_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...) == cudaSuccess ? SDV_OK : SDV_ERR_CUDA;
}

template <typename T, int D, bool EXTRA>
cudaError_t set_attn() {
    return cudaFuncSetAttribute(shared_attn_kernel<T, D, EXTRA>, cudaFuncAttributeMaxDynamicSharedMemorySize, STile<T, D>::SMEM);
}
template <typename T, int D>
cudaError_t set_attn_all() {
    const cudaError_t e = set_attn<T, D, false>();
    return e == cudaSuccess ? set_attn<T, D, true>() : e;
}
template <typename T, int D>
int launch_attn(const CUtensorMap &pool, const SharedArgs &a, void *stream) {
    const bool extra = a.cap2 > 0.f || a.slopes;
    const int r = launch(extra ? shared_attn_kernel<T, D, true> : shared_attn_kernel<T, D, false>, dim3(a.ctas), kSThreads,
                         STile<T, D>::SMEM, stream, pool, a);
    if (r != SDV_OK) return r;
    return launch(shared_merge_kernel<T, D>, dim3(cdiv(static_cast<long long>(a.max_rows) * a.nq, kSMergeThreads / 32)),
                  kSMergeThreads, 0, stream, a);
}

int device_sms(int dev) {
    int sms = 0;
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}

}  // namespace

extern "C" {

int sdv_shared_bytes(const sdv_shared_cfg *cfg, size_t *pool, size_t *workspace) {
    const int r = check_cfg(cfg);
    if (r) return r;
    if (!pool || !workspace) return SDV_ERR_ARG;
    *pool = layer_bytes(*cfg) * cfg->n_layers;
    int dev = 0, sms = 152;
    if (cudaGetDevice(&dev) == cudaSuccess)
        sms = device_sms(dev);
    else
        cudaGetLastError();  // no device to ask: the part's 152
    *workspace = ::workspace(*cfg, sms).end;
    return SDV_OK;
}

int sdv_shared_create(const sdv_shared_cfg *cfg, const void *d_pool, void *d_workspace, void *stream, sdv_shared **out) {
    const int r = check_cfg(cfg);
    if (r) return r;
    if (!d_pool || !d_workspace || !out) return SDV_ERR_ARG;
    if (reinterpret_cast<uintptr_t>(d_pool) % 16 || reinterpret_cast<uintptr_t>(d_workspace) % 256) return SDV_ERR_ARG;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return SDV_ERR_CUDA;
    cudaFuncAttributes fa;
    if (cudaFuncGetAttributes(&fa, shared_attn_kernel<bf16, 128, false>) != cudaSuccess) {
        cudaGetLastError();
        return SDV_ERR_UNSUPPORTED;  // no sm_103a image for this device
    }
    if (set_attn_all<bf16, 128>() != cudaSuccess || set_attn_all<bf16, 64>() != cudaSuccess ||
        set_attn_all<__half, 128>() != cudaSuccess || set_attn_all<__half, 64>() != cudaSuccess)
        return SDV_ERR_CUDA;
    sdv_shared *s = new (std::nothrow) sdv_shared();
    if (!s) return SDV_ERR_ARG;
    s->c = *cfg;
    s->device = dev;
    s->sm_count = device_sms(dev);
    s->grp = cfg->n_q_heads / cfg->n_kv_heads;
    s->pages_per_seq = cdiv(cfg->max_context, cfg->page_size);
    s->pool = static_cast<const uint8_t *>(d_pool);
    s->ws = static_cast<uint8_t *>(d_workspace);
    s->layer_bytes = layer_bytes(*cfg);
    s->by_page = FastDiv::of(cfg->page_size);
    s->by_grp = FastDiv::of(s->grp);
    s->by_nq = FastDiv::of(cfg->n_q_heads);
    s->box_rows = box_rows_of(*cfg);
    bool maps = true;
    try {
        s->pools.resize(cfg->n_layers);
        for (int l = 0; l < cfg->n_layers && s->box_rows && maps; ++l)
            maps = encode_pool_rows(&s->pools[l], s->pool + s->layer_bytes * l, *cfg, s->box_rows);
    } catch (const std::bad_alloc &) {
        maps = false;
    }
    if (!maps || cudaMemsetAsync(s->ws, 0, 256, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
        delete s;
        return SDV_ERR_CUDA;
    }
    *out = s;
    return SDV_OK;
}

int sdv_shared_destroy(sdv_shared *s) {
    delete s;
    return SDV_OK;
}

int sdv_shared_attention(sdv_shared *s, int layer, const void *d_q, int64_t q_stride, int rows, const int32_t *d_page_table,
                         const int32_t *d_row_off, const int32_t *d_base, int B, const int32_t *d_group_off,
                         const int32_t *d_prefix_len, int G, int max_span, int window, float softcap, const float *d_slopes,
                         void *d_out, int64_t out_stride, void *stream) {
    if (!s || !d_q || !d_out || d_q == d_out || !d_page_table || !d_row_off || !d_base || layer < 0 || layer >= s->c.n_layers || rows <= 0 ||
        B <= 0 || B > s->c.max_batch || max_span <= 0 || max_span > s->c.max_span || window < 0)
        return SDV_ERR_ARG;
    if (G < 0 || G > B || G > kSGroups || (G > 0 && (!d_group_off || !d_prefix_len))) return SDV_ERR_ARG;
    if (!(softcap >= 0.f && softcap < INFINITY)) return SDV_ERR_ARG;
    const int64_t width = static_cast<int64_t>(s->c.n_q_heads) * s->c.head_dim;
    if (q_stride < width || out_stride < width || reinterpret_cast<uintptr_t>(d_q) % 2 || reinterpret_cast<uintptr_t>(d_out) % 2)
        return SDV_ERR_ARG;
    int dev = -1;
    if (cudaGetDevice(&dev) != cudaSuccess || dev != s->device) return SDV_ERR_ARG;
    const sdv_shared_cfg &c = s->c;
    SharedArgs a{};
    a.q = d_q;
    a.out = d_out;
    a.q_stride = q_stride;
    a.out_stride = out_stride;
    a.pool = s->pool + s->layer_bytes * layer;
    a.page_table = d_page_table;
    a.row_off = d_row_off;
    a.base = d_base;
    a.group_off = d_group_off;
    a.prefix_len = d_prefix_len;
    a.slopes = d_slopes;
    a.status = reinterpret_cast<int *>(s->ws);
    a.pages_per_seq = s->pages_per_seq;
    a.page_size = c.page_size;
    a.n_pages = c.n_pages;
    a.nq = c.n_q_heads;
    a.nkv = c.n_kv_heads;
    a.grp = s->grp;
    a.B = B;
    a.G = G;
    a.max_span = max_span;
    a.max_rows = static_cast<int>(std::min<int64_t>({rows, c.max_rows, static_cast<int64_t>(B) * max_span}));
    a.max_context = c.max_context;
    a.window = window >= c.max_context ? 0 : window;
    a.q_vec = reinterpret_cast<uintptr_t>(d_q) % 16 == 0 && q_stride % 8 == 0;
    a.out_vec = reinterpret_cast<uintptr_t>(d_out) % 16 == 0 && out_stride % 8 == 0;
    a.box_rows = s->box_rows;
    a.pool_rows = c.n_pages * 2 * c.n_kv_heads * c.page_size;
    a.by_page = s->by_page;
    a.by_grp = s->by_grp;
    a.by_nq = s->by_nq;
    const float scale = 1.f / std::sqrt(static_cast<float>(c.head_dim));
    a.scale_log2 = 1.4426950408889634f * scale;
    if (softcap > 0.f) {  // where 1 / cap is a normal number: below, its infinity would make a score of zero no number
        const float cap = std::min(std::max(softcap, FLT_MIN), 1e30f);
        a.cap2 = 1.4426950408889634f * cap;
        a.to_u = scale / cap;
    }
    a.ctas = s->sm_count;
    const Workspace w = workspace(c, s->sm_count);
    a.part_rows = part_rows(c);
    a.plan_cut = reinterpret_cast<int2 *>(s->ws + 64);
    a.by_cut = reinterpret_cast<FastDiv *>(s->ws + 96);
    a.plan = reinterpret_cast<int4 *>(s->ws + w.plan);
    a.plan_rows = reinterpret_cast<int2 *>(s->ws + w.plan_rows);
    a.row_entry = reinterpret_cast<int2 *>(s->ws + w.row_entry);
    a.part_ml = reinterpret_cast<float2 *>(s->ws + w.ml);
    a.part_o = reinterpret_cast<float *>(s->ws + w.o);
    const CUtensorMap &pool = s->pools[layer];
    if (c.dtype == SDV_BF16)
        return c.head_dim == 128 ? launch_attn<bf16, 128>(pool, a, stream) : launch_attn<bf16, 64>(pool, a, stream);
    return c.head_dim == 128 ? launch_attn<__half, 128>(pool, a, stream) : launch_attn<__half, 64>(pool, a, stream);
}

int sdv_shared_get_status(sdv_shared *s, int32_t *h_status) {
    if (!s || !h_status) return SDV_ERR_ARG;
    if (cudaDeviceSynchronize() != cudaSuccess) return SDV_ERR_CUDA;
    int v = 0;
    const int zero = 0;
    if (cudaMemcpy(&v, s->ws, sizeof(int), cudaMemcpyDeviceToHost) != cudaSuccess) return SDV_ERR_CUDA;
    if (cudaMemcpy(s->ws, &zero, sizeof(int), cudaMemcpyHostToDevice) != cudaSuccess) return SDV_ERR_CUDA;
    *h_status = v;
    return SDV_OK;
}

}  // extern "C"
