// vq_paged.cu -- C ABI entry points of the paged code cache: page reservation
// and trimming, and attention of new tokens over the pages (see
// include/vq_encode.h for the contract of each function).
//
// Host side only: validate arguments, choose kernels and launch shapes, launch
// on the caller's stream.  The library allocates no memory.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "vq_encode.h"
#include "vq_host.h"
#include "vq_paged_host.h"
#include "vq_pages.cuh"
#include "vq_pattn.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_paged)

namespace {

int page_shift(int32_t page_size)
{
    int s = 0;
    while ((1 << s) < page_size) ++s;
    return s;
}

vq_status check_page(int32_t page_size)
{
    if (page_size < 1 || (page_size & (page_size - 1))) return VQ_ERR_INVALID_ARG;
    return page_size > VQ_PAGED_MAX_PAGE ? VQ_ERR_UNSUPPORTED : VQ_OK;
}

// A launch of one cluster of `blocks` blocks.
cudaLaunchConfig_t cluster_launch(int blocks, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute *attr)
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

vq_status check_pool(int64_t requests, int64_t max_blocks, int32_t page_size, int64_t num_pages)
{
    if (requests < 0 || max_blocks < 0 || num_pages < 0) return VQ_ERR_INVALID_ARG;
    const vq_status s = check_page(page_size);
    if (s != VQ_OK) return s;
    if (requests > vqk::kPageMaxRequests || num_pages > INT32_MAX ||
        max_blocks > VQ_PAGED_MAX_TOKENS / page_size)
        return VQ_ERR_UNSUPPORTED;
    return VQ_OK;
}

bool aligned4(const void *p) { return (uintptr_t)p % 4 == 0; }

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

size_t up256(size_t v) { return (v + 255) / 256 * 256; }

void lay_out(AttnPart *p, int32_t dim, size_t at)
{
    p->notes = at;
    p->ml = up256(p->notes + (size_t)p->blocks * sizeof(vqk::PagedNote));
    p->part = up256(p->ml + (size_t)2 * p->blocks * p->tile_rows * 2 * sizeof(float));
    p->end = up256(p->part + (size_t)2 * p->blocks * p->tile_rows * dim * sizeof(float));
}

constexpr int kSimpleBlocksPerSm = 4;

AttnPart simple_part(int sms, int32_t group, int32_t dim, size_t at)
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

// The tensor kernels take fp16 and bf16, head sizes 64, 128 and 256 in
// sub-vectors of 4 or 8, and pages of 16 tokens or more (the tokens of one
// matrix instruction lie in one page).
bool tensor_shape(vq_dtype dtype, int32_t dim, int32_t sub, int32_t page_size)
{
    return (dtype == VQ_F16 || dtype == VQ_BF16) && (dim == 64 || dim == 128 || dim == 256) &&
           (sub == 4 || sub == 8) && page_size >= 16;
}

// and pages whose rows can be read in vectors.
bool tensor_layout(const vqk::PagedArgs &a)
{
    return (uintptr_t)a.k_codes % 16 == 0 && (uintptr_t)a.v_codes % 16 == 0 && a.page_stride % 16 == 0;
}

// Which tensor kernels a call launches: requests of up to `few_tokens` new
// tokens go to the few-row kernel, the others to the chunk kernel.
struct TensorPlan {
    bool few, chunk;
    int32_t few_tokens;
};

TensorPlan tensor_plan(int64_t requests, int64_t tokens, int64_t max_new, int32_t group, int32_t dim)
{
    TensorPlan p{};
    const int64_t most = max_new > 0 && max_new < tokens ? max_new : tokens;  // new tokens of a request, as far as known
    // Up to three items of 8 rows, two at dim 256: the chunk kernel takes the time of a
    // tile of 128 rows however few there are, the few-row kernel that of its items.  16
    // requests of 8000 (2 of 30000), few-row against chunk kernel, us: dim 128 with two
    // items 77 : 101 (45 : 64), three 107 : 101 (58 : 66), four 135 : 102 (70 : 66); dim 64
    // three 74 : 84 (43 : 56), four 93 : 84 (51 : 56); dim 256 two 72 : 80 (43 : 51), three
    // 99 : 80 (54 : 54).  Other head groups and sub-vectors lie alike.
    const int32_t items = dim == 256 ? 2 : 3;
    const int32_t item_tokens = group < vqh_few_rows() ? vqh_few_rows() / group : 1;
    p.few_tokens = group > vqh_few_rows() ? 1 : items * item_tokens;
    p.chunk = most > p.few_tokens;
    p.few = requests != 1 || !p.chunk;
    return p;
}

AttnPart few_part(int sms, int32_t group, int32_t dim, size_t at)
{
    AttnPart p;
    p.blocks = sms * vqh_few_blocks_per_sm(dim);
    p.gc = group < vqh_few_rows() ? group : vqh_few_rows();
    p.gch = (group + p.gc - 1) / p.gc;
    p.tile_tokens = vqh_few_rows() / p.gc;
    p.tile_rows = vqh_few_rows();
    // set-up, merge of the warps and write of an item, in units: 2 : 3 : 4 : 5 give drafts of
    // 16 requests 60.7 : 57.3 : 56.0 : 55.4 us, 32 uneven decodes 148.8 : 147.7 : 146.9 : 146.5
    p.item_cost = 4;
    lay_out(&p, dim, at);
    return p;
}

AttnPart chunk_part(int sms, int32_t group, int32_t dim, size_t at)
{
    AttnPart p;
    p.blocks = sms;
    p.gc = group < 128 ? group : 128;
    p.gch = (group + p.gc - 1) / p.gc;
    p.tile_tokens = vqh_chunk_tiles(dim) * (128 / p.gc);
    p.tile_rows = vqh_chunk_tiles(dim) * 128;
    lay_out(&p, dim, at);
    return p;
}

// The parts of a call's tensor kernels, one behind the other.
size_t tensor_parts(const TensorPlan &t, int sms, int32_t group, int32_t dim, AttnPart *few, AttnPart *chunk)
{
    size_t at = 0;
    if (t.few) {
        *few = few_part(sms, group, dim, at);
        at = up256(few->end);
    }
    if (t.chunk) {
        *chunk = chunk_part(sms, group, dim, at);
        at = up256(chunk->end);
    }
    return at;
}

void use_part(vqk::PagedArgs *a, const AttnPart &p, unsigned char *ws)
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

template <typename T>
vq_status launch_merge(const vqk::PagedArgs &a, const AttnPart &p, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)p.blocks, (unsigned)((p.tile_rows + vqk::kMergeRows - 1) / vqk::kMergeRows));
    cfg.blockDim = dim3(vqk::kMergeThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // as many registers as the head size needs: the rows of a chunk are many
    auto kernel = a.dim % 4 != 0 ? vqk::paged_attn_merge<T, false, 16>
                  : a.dim <= 128 ? vqk::paged_attn_merge<T, true, 1>
                  : a.dim <= 256 ? vqk::paged_attn_merge<T, true, 2>
                                 : vqk::paged_attn_merge<T, true, 4>;
    if (cudaLaunchKernelEx(&cfg, kernel, (const float *)a.part, (const float *)a.ml,
                           (const vqk::PagedNote *)a.notes, p.tile_rows, a.dim, a.hq, a.tokens,
                           static_cast<T *>(a.out), a.lse) != cudaSuccess)
        return vqh_failed();
    return vqh_launched(st, vqh_status_paged);
}

template <typename T>
vq_status launch_simple(const AttnCall &c, const AttnPart &p, unsigned char *ws)
{
    vqk::PagedArgs a = c.a;
    use_part(&a, p, ws);
    a.cls = 0;
    const size_t smem = (size_t)vqk::kSimpleRows * a.dim * sizeof(float);
    vqk::paged_attn_simple<T><<<(unsigned)p.blocks, vqk::kUnit, smem, c.stream>>>(a);
    const vq_status s = vqh_launched(c.stream, vqh_status_paged);
    return s != VQ_OK ? s : launch_merge<T>(a, p, c.stream);
}

// Units of cached tokens up to which an item is better left to one block.
constexpr int64_t kWholeUnits = 8;

template <typename T>
vq_status launch_tensor(const AttnCall &c, unsigned char *ws)
{
    const TensorPlan t = tensor_plan(c.a.requests, c.a.tokens, c.max_new, c.a.group, c.a.dim);
    AttnPart few, chunk;
    (void)tensor_parts(t, c.sms, c.a.group, c.a.dim, &few, &chunk);
    if (t.chunk) {
        vqk::PagedArgs a = c.a;
        use_part(&a, chunk, ws);
        a.cls = t.few ? 2 : 0;
        a.cls_tokens = t.few_tokens;
        vq_status s = vqh_paged_chunk(a, c.dtype, chunk.blocks, c.stream);
        if (s == VQ_OK) s = launch_merge<T>(a, chunk, c.stream);
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
        // (26.7 : 29.7).  The host knows no lengths: what counts is how long the table
        // lets them be, and a wider table takes the split.
        const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
        a.no_split = cap <= kWholeUnits * vqk::kUnit && a.items * a.hkv * a.gch <= few.blocks;
        vq_status s = vqh_paged_few(a, c.dtype, few.blocks, c.stream);
        if (s == VQ_OK && !a.no_split) s = launch_merge<T>(a, few, c.stream);
        if (s != VQ_OK) return s;
    }
    return VQ_OK;
}

vq_status check_shape(int64_t requests, int64_t tokens, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                      int32_t sub_dim, int32_t n_centroids, int32_t page_size)
{
    if (requests < 0 || tokens < 0) return VQ_ERR_INVALID_ARG;
    if (heads_q < 1 || heads_kv < 1 || heads_q % heads_kv) return VQ_ERR_INVALID_ARG;
    if (sub_dim < 1 || head_dim < 1 || head_dim % sub_dim) return VQ_ERR_INVALID_ARG;
    if (head_dim > VQ_PAGED_MAX_HEAD_DIM || heads_q > VQ_PAGED_MAX_HEADS || n_centroids < 1 || n_centroids > 256)
        return VQ_ERR_UNSUPPORTED;
    if (requests > (1 << 24) || tokens > VQ_PAGED_MAX_TOKENS) return VQ_ERR_UNSUPPORTED;
    return check_page(page_size);
}

}  // namespace

extern "C" {

vq_status vq_paged_reserve(const int32_t *lens, const int32_t *new_lens, int64_t requests,
                           const int32_t *free_pages, const int32_t *free_count, int64_t num_pages,
                           int32_t *block_table, int64_t max_blocks, int32_t page_size,
                           int64_t total_new, int32_t *lens_out, int32_t *free_count_out,
                           int32_t *cu_new, int64_t *slots, vq_stream_t stream)
{
    vq_status s = check_pool(requests, max_blocks, page_size, num_pages);
    if (s != VQ_OK) return s;
    if (total_new < 0) return VQ_ERR_INVALID_ARG;
    if (total_new > VQ_PAGED_MAX_TOKENS) return VQ_ERR_UNSUPPORTED;
    if (!free_count || !free_count_out || !cu_new || (num_pages > 0 && !free_pages) || (total_new > 0 && !slots))
        return VQ_ERR_INVALID_ARG;
    if (requests > 0 && (!lens || !new_lens || !lens_out || (max_blocks > 0 && !block_table)))
        return VQ_ERR_INVALID_ARG;
    for (const void *p : {(const void *)lens, (const void *)new_lens, (const void *)free_pages,
                          (const void *)free_count, (const void *)block_table, (const void *)lens_out,
                          (const void *)free_count_out, (const void *)cu_new})
        if (!aligned4(p)) return VQ_ERR_INVALID_ARG;
    if ((uintptr_t)slots % 8) return VQ_ERR_INVALID_ARG;
    const size_t smem = vqk::page_reserve_smem(requests);
    if (smem > 48 * 1024 && !vqh_allow_smem(vqk::page_reserve, vqk::page_reserve_smem(vqk::kPageMaxRequests)))
        return vqh_failed();
    // one small block for a decode step; more where there are slots to write
    const int threads = requests <= vqk::kPageFewThreads && total_new <= 2 * vqk::kPageFewThreads ? vqk::kPageFewThreads
                                                                                                  : vqk::kPageThreads;
    int blocks = 1;
    while (blocks < 8 && total_new > (int64_t)blocks * vqk::kPageThreads) blocks *= 2;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = cluster_launch(blocks, threads, smem, st, attr);
    if (cudaLaunchKernelEx(&cfg, vqk::page_reserve, lens, new_lens, (int32_t)requests, free_pages, free_count,
                           (int32_t)num_pages, block_table, (int32_t)max_blocks, (int32_t)page_shift(page_size),
                           total_new, lens_out, free_count_out, cu_new, slots) != cudaSuccess)
        return vqh_failed();
    return vqh_launched(st, vqh_status_paged);
}

vq_status vq_paged_trim(const int32_t *lens, const int32_t *keep_lens, int64_t requests,
                        const int32_t *block_table, int64_t max_blocks, int32_t page_size,
                        int32_t *free_pages, const int32_t *free_count, int64_t num_pages,
                        int32_t *lens_out, int32_t *free_count_out, vq_stream_t stream)
{
    vq_status s = check_pool(requests, max_blocks, page_size, num_pages);
    if (s != VQ_OK) return s;
    if (!free_count || !free_count_out || (num_pages > 0 && !free_pages)) return VQ_ERR_INVALID_ARG;
    if (requests > 0 && (!lens || !keep_lens || !lens_out || (max_blocks > 0 && !block_table)))
        return VQ_ERR_INVALID_ARG;
    for (const void *p : {(const void *)lens, (const void *)keep_lens, (const void *)free_pages,
                          (const void *)free_count, (const void *)block_table, (const void *)lens_out,
                          (const void *)free_count_out})
        if (!aligned4(p)) return VQ_ERR_INVALID_ARG;
    const size_t smem = vqk::page_trim_smem(requests);
    if (smem > 48 * 1024 && !vqh_allow_smem(vqk::page_trim, vqk::page_trim_smem(vqk::kPageMaxRequests)))
        return vqh_failed();
    const int threads = requests <= vqk::kPageFewThreads ? vqk::kPageFewThreads : vqk::kPageThreads;
    int blocks = 1;  // a warp returns the pages of a request at a time
    while (blocks < 8 && requests > (int64_t)blocks * 64) blocks *= 2;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    cudaLaunchConfig_t cfg = cluster_launch(blocks, threads, smem, st, attr);
    if (cudaLaunchKernelEx(&cfg, vqk::page_trim, lens, keep_lens, (int32_t)requests, block_table,
                           (int32_t)max_blocks, (int32_t)page_shift(page_size), free_pages, free_count,
                           (int32_t)num_pages, lens_out, free_count_out) != cudaSuccess)
        return vqh_failed();
    return vqh_launched(st, vqh_status_paged);
}

size_t vq_paged_attention_workspace_bytes(int64_t requests, int64_t tokens, int64_t max_new,
                                          int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                                          int32_t sub_dim, int32_t n_centroids, int32_t page_size)
{
    if (max_new < 0 ||
        check_shape(requests, tokens, heads_q, heads_kv, head_dim, sub_dim, n_centroids, page_size) != VQ_OK)
        return 0;
    const int sms = vqh_device_sms() > 0 ? vqh_device_sms() : 152;
    const int32_t group = heads_q / heads_kv;
    size_t need = simple_part(sms, group, head_dim, 0).end;
    if (tensor_shape(VQ_F16, head_dim, sub_dim, page_size)) {
        AttnPart few, chunk;
        const TensorPlan plan = tensor_plan(requests, tokens, max_new, group, head_dim);
        const size_t t = tensor_parts(plan, sms, group, head_dim, &few, &chunk);
        if (t > need) need = t;
    }
    return need;
}

vq_status vq_paged_attention_slots(const void *q, int64_t q_stride, const int32_t *cu_new, const int32_t *lens,
                                   const int64_t *slots, int64_t requests, int64_t tokens, int64_t max_new,
                                   const int32_t *block_table, int64_t max_blocks, const uint8_t *k_codes,
                                   const uint8_t *v_codes, int64_t num_pages, int32_t page_size, int64_t page_stride,
                                   const void *k_codebooks, const void *v_codebooks, int32_t heads_q,
                                   int32_t heads_kv, int32_t head_dim, int32_t sub_dim, int32_t n_centroids,
                                   int64_t window, float scale, vq_dtype dtype, void *out, float *lse,
                                   void *workspace, size_t workspace_bytes, vq_stream_t stream)
{
    if (dtype != VQ_F16 && dtype != VQ_BF16 && dtype != VQ_F32) return VQ_ERR_INVALID_ARG;
    vq_status s = check_shape(requests, tokens, heads_q, heads_kv, head_dim, sub_dim, n_centroids, page_size);
    if (s != VQ_OK) return s;
    if (max_new < 0 || max_blocks < 0 || num_pages < 0 || window < 0 || !(scale == scale)) return VQ_ERR_INVALID_ARG;
    if (num_pages > INT32_MAX || max_blocks > VQ_PAGED_MAX_TOKENS / page_size) return VQ_ERR_UNSUPPORTED;
    const int32_t ns = head_dim / sub_dim;
    if (page_stride < (int64_t)heads_kv * page_size * ns) return VQ_ERR_INVALID_ARG;
    if (num_pages > 1 && page_stride > INT64_MAX / num_pages) return VQ_ERR_INVALID_ARG;
    if (q_stride < (int64_t)heads_q * head_dim) return VQ_ERR_INVALID_ARG;
    if (q_stride > INT64_MAX / 8 / VQ_PAGED_MAX_TOKENS) return VQ_ERR_UNSUPPORTED;
    if (tokens == 0) return VQ_OK;
    const uintptr_t es = dtype == VQ_F32 ? 4 : 2;
    if (!q || !cu_new || !k_codebooks || !v_codebooks || !out || !workspace) return VQ_ERR_INVALID_ARG;
    if (requests > 0 && (!lens || (max_blocks > 0 && !block_table))) return VQ_ERR_INVALID_ARG;
    if (num_pages > 0 && (!k_codes || !v_codes)) return VQ_ERR_INVALID_ARG;
    if ((uintptr_t)q % es || (uintptr_t)k_codebooks % es || (uintptr_t)v_codebooks % es || (uintptr_t)out % es ||
        !aligned4(cu_new) || !aligned4(lens) || !aligned4(block_table) || !aligned4(lse) || (uintptr_t)slots % 8 ||
        (uintptr_t)workspace % 16)
        return VQ_ERR_INVALID_ARG;

    AttnCall c{};
    c.dtype = dtype;
    c.max_new = max_new;
    c.sms = vqh_device_sms() > 0 ? vqh_device_sms() : 152;
    c.stream = reinterpret_cast<cudaStream_t>(stream);
    vqk::PagedArgs &a = c.a;
    a.q = q;
    a.k_codes = k_codes;
    a.v_codes = v_codes;
    a.kcb = k_codebooks;
    a.vcb = v_codebooks;
    a.out = out;
    a.lse = lse;
    a.cu = cu_new;
    a.lens = lens;
    a.slots = slots;
    a.table = block_table;
    a.tokens = tokens;
    a.q_stride = q_stride;
    a.page_stride = page_stride;
    a.num_pages = num_pages;
    a.requests = (int32_t)requests;
    a.max_blocks = (int32_t)max_blocks;
    a.page_shift = page_shift(page_size);
    a.hq = heads_q;
    a.hkv = heads_kv;
    a.group = heads_q / heads_kv;
    a.dim = head_dim;
    a.sub = sub_dim;
    a.ns = ns;
    a.nc = n_centroids;
    a.window = window >= INT32_MAX ? 0 : (int32_t)window;
    a.kappa = (scale > 0.f ? scale : 1.0f / sqrtf((float)head_dim)) * 1.4426950408889634f;

    if (workspace_bytes < vq_paged_attention_workspace_bytes(requests, tokens, max_new, heads_q, heads_kv, head_dim,
                                                             sub_dim, n_centroids, page_size))
        return VQ_ERR_INVALID_ARG;
    unsigned char *ws = static_cast<unsigned char *>(workspace);
    if (tensor_shape(dtype, head_dim, sub_dim, page_size) && tensor_layout(a))
        return dtype == VQ_F16 ? launch_tensor<__half>(c, ws) : launch_tensor<__nv_bfloat16>(c, ws);
    const AttnPart p = simple_part(c.sms, a.group, head_dim, 0);
    switch (dtype) {
    case VQ_F16: return launch_simple<__half>(c, p, ws);
    case VQ_BF16: return launch_simple<__nv_bfloat16>(c, p, ws);
    case VQ_F32: return launch_simple<float>(c, p, ws);
    }
    return VQ_ERR_INTERNAL;
}

vq_status vq_paged_attention(const void *q, int64_t q_stride, const int32_t *cu_new, const int32_t *lens,
                             int64_t requests, int64_t tokens, int64_t max_new, const int32_t *block_table,
                             int64_t max_blocks, const uint8_t *k_codes, const uint8_t *v_codes,
                             int64_t num_pages, int32_t page_size, int64_t page_stride,
                             const void *k_codebooks, const void *v_codebooks, int32_t heads_q,
                             int32_t heads_kv, int32_t head_dim, int32_t sub_dim, int32_t n_centroids,
                             int64_t window, float scale, vq_dtype dtype, void *out, float *lse,
                             void *workspace, size_t workspace_bytes, vq_stream_t stream)
{
    return vq_paged_attention_slots(q, q_stride, cu_new, lens, nullptr, requests, tokens, max_new, block_table,
                                    max_blocks, k_codes, v_codes, num_pages, page_size, page_stride, k_codebooks,
                                    v_codebooks, heads_q, heads_kv, head_dim, sub_dim, n_centroids, window, scale,
                                    dtype, out, lse, workspace, workspace_bytes, stream);
}

}  // extern "C"
