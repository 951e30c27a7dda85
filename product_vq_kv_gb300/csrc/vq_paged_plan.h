// vq_paged_plan.h -- what the entry points of the paged caches share: checks of a
// pool's sizes, and the plan of an attention call, its kernels' launches and parts of
// the workspace (internal; not part of the C ABI).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "vq_encode.h"
#include "vq_host.h"
#include "vq_paged_host.h"
#include "vq_pagescan.cuh"
#include "vq_pattn.cuh"

namespace vqp {

inline int page_shift(int32_t page_size)
{
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

inline vq_status check_page(int32_t page_size)
{
    if (page_size < 1 || (page_size & (page_size - 1))) return VQ_ERR_INVALID_ARG;
    return page_size > VQ_PAGED_MAX_PAGE ? VQ_ERR_UNSUPPORTED : VQ_OK;
}

// A launch of one cluster of `blocks` blocks.
inline cudaLaunchConfig_t cluster_launch(int blocks, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute *attr)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)blocks;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = blocks > 1 ? 1 : 0;  // one block is a cluster by itself
    return cfg;
}

inline vq_status check_pool(int64_t requests, int64_t max_blocks, int32_t page_size, int64_t num_pages)
{
    if (requests < 0 || max_blocks < 0 || num_pages < 0) return VQ_ERR_INVALID_ARG;
    const vq_status s = check_page(page_size);
    if (s != VQ_OK) return s;
    if (requests > vqk::kPageMaxRequests || num_pages > INT32_MAX ||
        max_blocks > VQ_PAGED_MAX_TOKENS / page_size)
        return VQ_ERR_UNSUPPORTED;
    return VQ_OK;
}

inline bool aligned4(const void *p) { return (uintptr_t)p % 4 == 0; }

// ------------------------------------------------------------------ attention plans

struct AttnCall {
    vqk::PagedArgs a;
    vq_dtype dtype;
    int64_t max_new;
    int sms;
    cudaStream_t stream;
};

// One kernel's launch: its blocks, rows per item and share of the workspace.
struct AttnPart {
    int blocks = 0;
    int32_t tile_tokens = 0, gc = 0, gch = 0, tile_rows = 0, item_cost = 0;
    size_t notes = 0, ml = 0, part = 0, end = 0;  // workspace offsets
};

inline size_t up256(size_t v) { return (v + 255) / 256 * 256; }

inline void lay_out(AttnPart *p, int32_t dim, size_t at)
{
    p->notes = at;
    p->ml = up256(p->notes + (size_t)p->blocks * sizeof(vqk::PagedNote));
    p->part = up256(p->ml + (size_t)2 * p->blocks * p->tile_rows * 2 * sizeof(float));
    p->end = up256(p->part + (size_t)2 * p->blocks * p->tile_rows * dim * sizeof(float));
}

constexpr int kSimpleBlocksPerSm = 4;

inline AttnPart simple_part(int sms, int32_t group, int32_t dim, size_t at)
{
    AttnPart p;
    p.blocks = sms * kSimpleBlocksPerSm;
    p.tile_tokens = 1;
    p.gc = group < vqk::kSimpleRows ? group : vqk::kSimpleRows;
    p.gch = (group + p.gc - 1) / p.gc;
    p.tile_rows = p.gc;
    lay_out(&p, dim, at);
    return p;
}

// The tensor kernels of a cache format at one head size.
struct TensorKernels {
    int few_rows, few_blocks_per_sm;  // the few-row kernel: rows of an item
    int chunk_tiles;                  // the chunk kernel: tiles of 128 rows an item has
    int32_t few_items;                // items of a request up to which the few-row kernel takes it
    int32_t item_cost;                // set-up, merge of the warps and write of its item, in units
    vq_status (*few)(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st);
    vq_status (*chunk)(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st);
};

// Which tensor kernels a call launches: requests of up to `few_tokens` new
// tokens go to the few-row kernel, the others to the chunk kernel.
struct TensorPlan {
    bool few, chunk;
    int32_t few_tokens;
};

inline TensorPlan tensor_plan(const TensorKernels &k, int64_t requests, int64_t tokens, int64_t max_new, int32_t group)
{
    TensorPlan p{};
    const int64_t most = max_new > 0 && max_new < tokens ? max_new : tokens;  // new tokens of a request, as far as known
    const int32_t item_tokens = group < k.few_rows ? k.few_rows / group : 1;
    p.few_tokens = group > k.few_rows ? 1 : k.few_items * item_tokens;
    p.chunk = most > p.few_tokens;
    p.few = requests != 1 || !p.chunk;
    return p;
}

inline AttnPart few_part(const TensorKernels &k, int sms, int32_t group, int32_t dim, size_t at)
{
    AttnPart p;
    p.blocks = sms * k.few_blocks_per_sm;
    p.gc = group < k.few_rows ? group : k.few_rows;
    p.gch = (group + p.gc - 1) / p.gc;
    p.tile_tokens = k.few_rows / p.gc;
    p.tile_rows = k.few_rows;
    p.item_cost = k.item_cost;
    lay_out(&p, dim, at);
    return p;
}

inline AttnPart chunk_part(const TensorKernels &k, int sms, int32_t group, int32_t dim, size_t at)
{
    AttnPart p;
    p.blocks = sms;
    p.gc = group < 128 ? group : 128;
    p.gch = (group + p.gc - 1) / p.gc;
    p.tile_tokens = k.chunk_tiles * (128 / p.gc);
    p.tile_rows = k.chunk_tiles * 128;
    lay_out(&p, dim, at);
    return p;
}

// The parts of a call's tensor kernels, one behind the other.
inline size_t tensor_parts(const TensorKernels &k, const TensorPlan &t, int sms, int32_t group, int32_t dim, AttnPart *few,
                           AttnPart *chunk)
{
    size_t at = 0;
    if (t.few) {
        *few = few_part(k, sms, group, dim, at);
        at = up256(few->end);
    }
    if (t.chunk) {
        *chunk = chunk_part(k, sms, group, dim, at);
        at = up256(chunk->end);
    }
    return at;
}

inline void use_part(vqk::PagedArgs *a, const AttnPart &p, unsigned char *ws)
{
    a->tile_tokens = p.tile_tokens;
    a->gc = p.gc;
    a->gch = p.gch;
    a->tile_rows = p.tile_rows;
    a->item_cost = p.item_cost;
    a->items = a->tokens / p.tile_tokens + a->requests + 1;
    a->notes = reinterpret_cast<vqk::PagedNote *>(ws + p.notes);
    a->ml = reinterpret_cast<float *>(ws + p.ml);
    a->part = reinterpret_cast<float *>(ws + p.part);
}

// Units of cached tokens up to which an item is better left to one block.
constexpr int64_t kWholeUnits = 8;

inline vq_status launch_tensor(const AttnCall &c, const TensorKernels &k, unsigned char *ws)
{
    const TensorPlan t = tensor_plan(k, c.a.requests, c.a.tokens, c.max_new, c.a.group);
    AttnPart few, chunk;
    (void)tensor_parts(k, t, c.sms, c.a.group, c.a.dim, &few, &chunk);
    if (t.chunk) {
        vqk::PagedArgs a = c.a;
        use_part(&a, chunk, ws);
        a.cls = t.few ? 2 : 0;
        a.cls_tokens = t.few_tokens;
        vq_status s = k.chunk(a, c.dtype, chunk.blocks, c.stream);
        if (s == VQ_OK) s = vqh_paged_merge(a, c.dtype, chunk.blocks, c.stream);
        if (s != VQ_OK) return s;
    }
    if (t.few) {
        vqk::PagedArgs a = c.a;
        use_part(&a, few, ws);
        a.cls = t.chunk ? 1 : 0;
        a.cls_tokens = t.few_tokens;
        // Short caches and few of them: an item a block, none split, no merge to
        // launch.  One token, 8 heads, whole against split, us on the device (a graph's
        // replay) and as a call: one request of 300 12.3 : 14.4 (26.6 : 29.7), of 777 16.4 :
        // 14.4 (25.9 : 28.8); eight of 300 13.5 : 18.4 (26.3 : 29.7), of 777 16.4 : 19.8
        // (26.7 : 29.7).  Over 4-bit codes, on the device: one of 300 19.6 : 21.7, of 777 21.7 :
        // 21.7, of 1000 21.7 : 23.7; eight 19.6 : 23.7, 23.6 : 25.7, 23.6 : 25.7.  The host knows no
        // lengths: what counts is how long the table lets them be, and a wider table takes the split.
        const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
        a.no_split = cap <= kWholeUnits * vqk::kUnit && a.items * a.hkv * a.gch <= few.blocks;
        vq_status s = k.few(a, c.dtype, few.blocks, c.stream);
        if (s == VQ_OK && !a.no_split) s = vqh_paged_merge(a, c.dtype, few.blocks, c.stream);
        if (s != VQ_OK) return s;
    }
    return VQ_OK;
}

}  // namespace vqp
