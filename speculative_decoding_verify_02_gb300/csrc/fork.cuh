// Sequences that continue another one's prompt: forking shares the pages that the source has filled, copies the partial one,
// and takes over its loop state and n-gram index.
//
// extra[page] counts a page's holders beyond the first; a page goes back to the free stack when its last holder lets go. Only
// whole pages below a sequence's length are shared and those are never written again, so a shared page sits in the same
// page-table slot of all its holders.
#pragma once

#include "small.cuh"

namespace sdv {

constexpr int kForkMost = 256;     // forks of a call: max_batch at most
constexpr int kForkThreads = kForkMost;
constexpr int kCopyThreads = 256;
constexpr int kForkIndexBlocks = 8;  // CTAs that copy a sequence's n-gram index

struct ForkArgs {
    DevState s;
    const int *src, *dst;
    int n;
    int4 *copies;  // [n]: partial page, its copy, slots filled (0: none), 1 if the fork takes place
    bf16 *pool;
    size_t layer_stride;  // elements of a layer
    int n_layers, nkv, D;
};

// All of the forks or none of them, by one CTA.
__global__ void __launch_bounds__(kForkThreads) fork_kernel(ForkArgs p) {
    pdl_trigger();
    pdl_wait();
    DevState &s = p.s;
    __shared__ int taken[kForkMost], warp_sum[kForkThreads / 32], ok_s, added;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    if (tid < kForkMost) taken[tid] = 0;
    if (tid == 0) ok_s = SDV_OK, added = 0;
    __syncthreads();
    const bool mine = tid < p.n;
    const int src = mine ? p.src[tid] : 0, dst = mine ? p.dst[tid] : 0;
    bool ok = true;
    if (mine) {
        ok = src >= 0 && src < s.max_batch && dst >= 0 && dst < s.max_batch;
        if (ok) ok = atomicExch(&taken[dst], 1) == 0 && s.seq_len[dst] == 0 && s.n_pages[dst] == 0;
    }
    if (!ok) atomicCAS(&ok_s, SDV_OK, SDV_ERR_ARG);
    __syncthreads();
    if (mine && ok && taken[src]) atomicCAS(&ok_s, SDV_OK, SDV_ERR_ARG);  // a source that is a destination, too
    const int L = mine && ok ? s.seq_len[src] : 0, full = L / s.page_size, fill = L - full * s.page_size, need = fill > 0;
    int at = need;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += v;
    }
    if (lane == 31) warp_sum[warp] = at;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kForkThreads / 32; ++w) {
        if (w < warp) at += warp_sum[w];
        total += warp_sum[w];
    }
    at -= need;  // pages that the forks before take
    const int top = *s.free_top;
    if (tid == 0 && ok_s == SDV_OK && total > top) ok_s = SDV_ERR_CAPACITY;
    __syncthreads();
    if (ok_s != SDV_OK) {
        if (tid == 0) set_status(s.status, ok_s);
        if (mine) p.copies[tid] = make_int4(0, 0, 0, 0);
        return;
    }
    if (mine) {
        int page = -1;
        if (need) {
            page = s.free_stack[top - 1 - at];
            s.page_table[static_cast<size_t>(dst) * s.pages_per_seq + full] = page;
        }
        p.copies[tid] = make_int4(need ? s.page_table[static_cast<size_t>(src) * s.pages_per_seq + full] : 0, page, fill, 1);
        s.n_pages[dst] = full + need;
        s.seq_len[dst] = L;
        s.hist_len[dst] = s.hist_len[src];
        s.cur_tok[dst] = s.cur_tok[src];
        s.generated[dst] = s.generated[src];
        s.budget[dst] = s.budget[src];
        s.kcur[dst] = s.kcur[src];
        atomicAdd(&added, full);
    }
    __syncthreads();
    if (tid == 0) {
        *s.free_top = top - total;
        *s.n_extra += added;
    }
}

// The filled slots of the partial pages: CTA (fork, layer), a warp a head; behind the layers a CTA for the whole pages' entries and
// those that copy the n-gram index. Bound by launch and latency for a few forks, else by memory.
__global__ void __launch_bounds__(kCopyThreads) fork_copy_kernel(ForkArgs p) {
    pdl_trigger();
    pdl_wait();
    const DevState &s = p.s;
    const int4 c = p.copies[blockIdx.x];
    if (!c.w) return;
    const int layer = blockIdx.y, tid = threadIdx.x;
    if (layer < p.n_layers) {
        if (c.z == 0 || c.x < 0 || c.x >= s.n_pages_total) return;
        const size_t page = static_cast<size_t>(2) * p.nkv * s.page_size * p.D;
        const int row = p.D / 8, run = c.z * row;  // 16-byte pieces of a slot, and filled ones of a head
        const size_t whole = static_cast<size_t>(s.page_size) * row;
        const uint4 *from = reinterpret_cast<const uint4 *>(p.pool + layer * p.layer_stride + c.x * page);
        uint4 *to = reinterpret_cast<uint4 *>(p.pool + layer * p.layer_stride + c.y * page);
        for (int head = tid / 32; head < 2 * p.nkv; head += kCopyThreads / 32)
#pragma unroll 4
            for (int i = tid % 32; i < run; i += 32) to[head * whole + i] = from[head * whole + i];
        return;
    }
    const int src = p.src[blockIdx.x], dst = p.dst[blockIdx.x];
    if (layer == p.n_layers) {
        const int *have = s.page_table + static_cast<size_t>(src) * s.pages_per_seq;
        int *get = s.page_table + static_cast<size_t>(dst) * s.pages_per_seq;
        const int full = s.seq_len[dst] / s.page_size;
#pragma unroll 4
        for (int j = tid; j < full; j += kCopyThreads) {
            const int held = have[j];
            get[j] = held;
            atomicAdd(&s.extra[held], 1);
        }
        return;
    }
    const size_t slots = static_cast<size_t>(s.ng_orders) * s.ng_slots;
    const int first = (layer - p.n_layers - 1) * kCopyThreads + tid, step = kForkIndexBlocks * kCopyThreads;
    for (size_t i = first; i < slots; i += step) {
        s.ng_keys[dst * slots + i] = s.ng_keys[src * slots + i];
        s.ng_vals[dst * slots + i] = s.ng_vals[src * slots + i];
    }
    for (int i = first; i < s.hist_len[src]; i += step)
        s.hist[static_cast<size_t>(dst) * s.ngram_cap + i] = s.hist[static_cast<size_t>(src) * s.ngram_cap + i];
}

}  // namespace sdv
