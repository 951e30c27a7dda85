// vq_scache.cu -- C ABI entry points of attention over the paged cache of 4-bit scalar
// codes (see include/vq_encode.h for the contract).  Host side only.

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "vq_encode.h"
#include "vq_host.h"
#include "vq_paged_host.h"
#include "vq_paged_plan.h"
#include "vq_sattn.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_scache)

namespace {

using namespace vqp;

// The tensor kernels take fp16 and bf16, head sizes 64, 128 and 256, and pages of 16 tokens
// or more (the tokens of one matrix instruction lie in one page).
bool tensor_shape(vq_dtype dtype, int32_t dim, int32_t page_size)
{
    return (dtype == VQ_F16 || dtype == VQ_BF16) && (dim == 64 || dim == 128 || dim == 256) && page_size >= 16;
}

// and pages whose rows and scales can be read in 16-byte pieces.
bool tensor_layout(const vqk::PagedArgs &a)
{
    for (const void *p : {(const void *)a.k_codes, (const void *)a.v_codes, a.k_scales, a.v_scales})
        if ((uintptr_t)p % 16) return false;
    return a.page_stride % 16 == 0 && a.scale_stride % 8 == 0;
}

TensorKernels tensor_kernels(int32_t dim, int32_t group, int64_t max_new)
{
    // Four items of 8 rows: the chunk kernel takes the time of a tile of 128 rows however few
    // there are, the few-row kernel that of its items.  16 requests of 8000 (2 of 30000), few-row
    // against chunk kernel, us: dim 128 three 128 : 160 (69 : 99), four 163 : 161 (83 : 102), five
    // 196 : 163 (95 : 104); dim 64 four 122 : 128 (64 : 83), five 147 : 128 (73 : 85); dim 256
    // three 116 : 143 (65 : 89), four 145 : 145 (77 : 89), five 173 : 145 (89 : 89).
    // items of 4 rows where no request has more
    const int rows = max_new > 0 && group <= 4 && max_new * group <= 4 ? 4 : vqh_few_rows();
    // An item's cost: 2 : 4 : 8 : 12 give drafts of 16 requests 70.8 : 64.6 : 62.6 : 66.7 us, 32
    // uneven decodes 156.8 : 154.8 : 152.7 : 150.7, 64 short ones 56.4 : 54.4 : 52.3 : 52.3
    return TensorKernels{rows, 1, vqh_chunk_tiles(dim), 4, 8, vqh_paged_sfew, vqh_paged_schunk};
}

template <typename T>
vq_status launch_simple(const AttnCall &c, const AttnPart &p, unsigned char *ws)
{
    vqk::PagedArgs a = c.a;
    use_part(&a, p, ws);
    a.cls = 0;
    const size_t smem = (size_t)vqk::kSimpleRows * a.dim * sizeof(float);
    vqk::paged_attn_scalar_simple<T><<<(unsigned)p.blocks, vqk::kUnit, smem, c.stream>>>(a);
    const vq_status s = vqh_launched(c.stream, vqh_status_scache);
    return s != VQ_OK ? s : vqh_paged_merge(a, c.dtype, p.blocks, c.stream);
}

vq_status check_shape(int64_t requests, int64_t tokens, int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                      int32_t page_size)
{
    if (requests < 0 || tokens < 0) return VQ_ERR_INVALID_ARG;
    if (heads_q < 1 || heads_kv < 1 || heads_q % heads_kv || head_dim < 2 || head_dim % 2) return VQ_ERR_INVALID_ARG;
    if (head_dim > VQ_PAGED_MAX_HEAD_DIM || heads_q > VQ_PAGED_MAX_HEADS) return VQ_ERR_UNSUPPORTED;
    if (requests > (1 << 24) || tokens > VQ_PAGED_MAX_TOKENS) return VQ_ERR_UNSUPPORTED;
    return check_page(page_size);
}

}  // namespace

extern "C" {

size_t vq_paged_scalar_attention_workspace_bytes(int64_t requests, int64_t tokens, int64_t max_new,
                                                 int32_t heads_q, int32_t heads_kv, int32_t head_dim,
                                                 int32_t page_size)
{
    if (max_new < 0 || check_shape(requests, tokens, heads_q, heads_kv, head_dim, page_size) != VQ_OK) return 0;
    const int sms = vqh_device_sms() > 0 ? vqh_device_sms() : 152;
    const int32_t group = heads_q / heads_kv;
    size_t need = simple_part(sms, group, head_dim, 0).end;
    if (tensor_shape(VQ_F16, head_dim, page_size)) {
        AttnPart few, chunk;
        const TensorKernels k = tensor_kernels(head_dim, group, max_new);
        const size_t t = tensor_parts(k, tensor_plan(k, requests, tokens, max_new, group), sms, group, head_dim, &few, &chunk);
        if (t > need) need = t;
    }
    return need;
}

vq_status vq_paged_scalar_attention(const void *q, int64_t q_stride, const int32_t *cu_new, const int32_t *lens,
                                    const int64_t *slots, int64_t requests, int64_t tokens, int64_t max_new,
                                    const int32_t *block_table, int64_t max_blocks, const uint8_t *k_codes,
                                    const uint8_t *v_codes, const void *k_scales, const void *v_scales,
                                    int64_t num_pages, int32_t page_size, int64_t page_stride, int64_t scale_stride,
                                    const float *k_centroids, const float *v_centroids, int32_t heads_q,
                                    int32_t heads_kv, int32_t head_dim, int32_t n_centroids, int64_t window,
                                    float scale, vq_dtype dtype, void *out, float *lse, void *workspace,
                                    size_t workspace_bytes, vq_stream_t stream)
{
    if (dtype != VQ_F16 && dtype != VQ_BF16 && dtype != VQ_F32) return VQ_ERR_INVALID_ARG;
    vq_status s = check_shape(requests, tokens, heads_q, heads_kv, head_dim, page_size);
    if (s != VQ_OK) return s;
    if (n_centroids < 1 || n_centroids > VQ_PAGED_SCALAR_MAX_CENTROIDS) return VQ_ERR_UNSUPPORTED;
    if (max_new < 0 || max_blocks < 0 || num_pages < 0 || window < 0 || !(scale == scale)) return VQ_ERR_INVALID_ARG;
    if (num_pages > INT32_MAX || max_blocks > VQ_PAGED_MAX_TOKENS / page_size) return VQ_ERR_UNSUPPORTED;
    const int64_t page_rows = (int64_t)heads_kv * page_size;
    if (page_stride < page_rows * (head_dim / 2) || scale_stride < page_rows) return VQ_ERR_INVALID_ARG;
    if (num_pages > 1 && (page_stride > INT64_MAX / num_pages || scale_stride > INT64_MAX / 4 / num_pages))
        return VQ_ERR_INVALID_ARG;
    if (q_stride < (int64_t)heads_q * head_dim) return VQ_ERR_INVALID_ARG;
    if (q_stride > INT64_MAX / 8 / VQ_PAGED_MAX_TOKENS) return VQ_ERR_UNSUPPORTED;
    if (tokens == 0) return VQ_OK;
    const uintptr_t es = dtype == VQ_F32 ? 4 : 2;
    if (!q || !cu_new || !k_centroids || !v_centroids || !out || !workspace) return VQ_ERR_INVALID_ARG;
    if (requests > 0 && (!lens || (max_blocks > 0 && !block_table))) return VQ_ERR_INVALID_ARG;
    if (num_pages > 0 && (!k_codes || !v_codes || !k_scales || !v_scales)) return VQ_ERR_INVALID_ARG;
    if ((uintptr_t)q % es || (uintptr_t)k_scales % es || (uintptr_t)v_scales % es || (uintptr_t)out % es ||
        !aligned4(k_centroids) || !aligned4(v_centroids) || !aligned4(cu_new) || !aligned4(lens) ||
        !aligned4(block_table) || !aligned4(lse) || (uintptr_t)slots % 8 || (uintptr_t)workspace % 16)
        return VQ_ERR_INVALID_ARG;
    if (workspace_bytes <
        vq_paged_scalar_attention_workspace_bytes(requests, tokens, max_new, heads_q, heads_kv, head_dim, page_size))
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
    a.k_scales = k_scales;
    a.v_scales = v_scales;
    a.k_cent = k_centroids;
    a.v_cent = v_centroids;
    a.out = out;
    a.lse = lse;
    a.cu = cu_new;
    a.lens = lens;
    a.slots = slots;
    a.table = block_table;
    a.tokens = tokens;
    a.q_stride = q_stride;
    a.page_stride = page_stride;
    a.scale_stride = scale_stride;
    a.num_pages = num_pages;
    a.requests = (int32_t)requests;
    a.max_blocks = (int32_t)max_blocks;
    a.page_shift = page_shift(page_size);
    a.hq = heads_q;
    a.hkv = heads_kv;
    a.group = heads_q / heads_kv;
    a.dim = head_dim;
    a.sub = 2;
    a.ns = head_dim / 2;
    a.nc = n_centroids;
    a.window = window >= INT32_MAX ? 0 : (int32_t)window;
    a.kappa = (scale > 0.f ? scale : 1.0f / sqrtf((float)head_dim)) * 1.4426950408889634f;

    unsigned char *ws = static_cast<unsigned char *>(workspace);
    if (tensor_shape(dtype, head_dim, page_size) && tensor_layout(a)) return launch_tensor(c, tensor_kernels(head_dim, a.group, max_new), ws);
    const AttnPart p = simple_part(c.sms, a.group, head_dim, 0);
    switch (dtype) {
    case VQ_F16: return launch_simple<__half>(c, p, ws);
    case VQ_BF16: return launch_simple<__nv_bfloat16>(c, p, ws);
    case VQ_F32: return launch_simple<float>(c, p, ws);
    }
    return VQ_ERR_INTERNAL;
}

}  // extern "C"
