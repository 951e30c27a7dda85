// vq_append.cu -- C ABI entry point of the append to the paged code cache
// (see include/vq_encode.h for its contract).  Host side only.

#include <cuda_runtime.h>

#include <cstdint>

#include "vq_encode.h"
#include "vq_append.cuh"
#include "vq_host.h"
#include "vq_status.cuh"
#include "vq_tc_host.h"

VQH_STATUS_READER(vqh_status_append)

namespace {

template <typename T>
vq_status launch_general(const vqk::AppendArgs &a, int kv0, int n, cudaStream_t st)
{
    const int64_t rows = a.tokens * a.heads * a.ns;
    const int64_t blocks = (rows + 127) / 128;
    if (blocks > 0x7fffffffLL) return VQ_ERR_UNSUPPORTED;
    vqk::append_general<T><<<dim3((unsigned)blocks, (unsigned)n), 128, 0, st>>>(a, kv0, 1.0f);
    return vqh_launched(st, vqh_status_append);
}

template <typename T, int SUB, bool SMOOTH>
vq_status launch_tc(const vqk::AppendArgs &a, vq_dtype dtype, int kv0, int kinds, cudaStream_t st)
{
    constexpr bool kSplit = vqh::tc_split<T, SMOOTH>();
    using C = vqk::TcConfig<SUB, kSplit>;
    const size_t smem = vqh::tc_smem<SUB, SMOOTH>(a.nc, dtype);
    int64_t per_group = 0;
    int32_t tiles = 0;
    const int64_t groups = (int64_t)kinds * a.heads;
    vqh::tc_shape(groups, a.tokens * a.ns, vqh::tc_slots(SUB, kSplit, smem), vqh::tc_tps(SUB, kSplit), &per_group, &tiles);
    if (groups * per_group > 0x7fffffffLL) return VQ_ERR_UNSUPPORTED;
    auto kernel = vqk::append_tc<T, SUB, C::kCols, C::kGroup, C::kMinBlocks, SMOOTH, C::kTps>;
    if (!vqh_allow_smem(kernel, vqh::tc_smem<SUB, SMOOTH>(vqh::kTcMaxCentroids, dtype))) return vqh_failed();
    kernel<<<(unsigned)(groups * per_group), 128 * C::kTps, smem, st>>>(a, kv0, (int32_t)per_group, tiles, 1.0f);
    return vqh_launched(st, vqh_status_append);
}

// Rows aligned for the vector loads, codebooks that screening pays for, rows
// counted in 31 bits: the tensor-core encode.  Otherwise the general kernel.
template <typename T>
bool tc_takes(const vqk::AppendArgs &a)
{
    const int64_t row = (int64_t)a.sub * sizeof(T), align = row < 16 ? row : 16;
    for (int kv = 0; kv < 2; ++kv)
        if ((uintptr_t)a.x[kv] % align || a.stride[kv] * (int64_t)sizeof(T) % align) return false;
    return (a.sub == 4 || a.sub == 8) && a.nc >= vqh::kFilterMinCentroids && a.tokens * a.ns < 0x7fffffffLL - 128;
}

template <typename T, int SUB>
vq_status launch_sub(const vqk::AppendArgs &a, vq_dtype dtype, cudaStream_t st)
{
    if (!a.smooth) return launch_tc<T, SUB, false>(a, dtype, 0, 2, st);
    const vq_status s = launch_tc<T, SUB, true>(a, dtype, 0, 1, st);  // smoothed keys: rows in two pieces
    return s != VQ_OK ? s : launch_tc<T, SUB, false>(a, dtype, 1, 1, st);
}

template <typename T>
vq_status launch(const vqk::AppendArgs &a, vq_dtype dtype, cudaStream_t st)
{
    if (!tc_takes<T>(a)) return launch_general<T>(a, 0, 2, st);
    return a.sub == 4 ? launch_sub<T, 4>(a, dtype, st) : launch_sub<T, 8>(a, dtype, st);
}

}  // namespace

extern "C" {

vq_status vq_paged_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                          const int64_t *slots, int64_t tokens, int32_t heads, int32_t head_dim,
                          int32_t sub_dim, int32_t n_centroids, const void *k_codebooks,
                          const void *v_codebooks, const float *k_smooth, uint8_t *k_codes,
                          uint8_t *v_codes, int64_t num_pages, int32_t page_size,
                          int64_t page_stride, vq_dtype dtype, vq_stream_t stream)
{
    if (dtype != VQ_F16 && dtype != VQ_BF16 && dtype != VQ_F32) return VQ_ERR_INVALID_ARG;
    if (tokens < 0 || num_pages < 0 || heads < 1 || sub_dim < 1 || head_dim < 1 || head_dim % sub_dim)
        return VQ_ERR_INVALID_ARG;
    if (sub_dim > vqk::kAppendMaxSub || head_dim > VQ_PAGED_MAX_HEAD_DIM || heads > VQ_PAGED_MAX_HEADS ||
        n_centroids < 1 || n_centroids > 256)
        return VQ_ERR_UNSUPPORTED;
    if (page_size < 1 || (page_size & (page_size - 1))) return VQ_ERR_INVALID_ARG;
    if (page_size > VQ_PAGED_MAX_PAGE) return VQ_ERR_UNSUPPORTED;
    const int32_t ns = head_dim / sub_dim;
    const int64_t page_bytes = (int64_t)heads * page_size * ns;
    if (page_stride < page_bytes || num_pages > (INT64_MAX >> 20) / page_size) return VQ_ERR_INVALID_ARG;
    if (num_pages > 1 && page_stride > INT64_MAX / num_pages) return VQ_ERR_INVALID_ARG;
    const int64_t row = (int64_t)heads * head_dim;
    if (k_stride < row || v_stride < row) return VQ_ERR_INVALID_ARG;
    if (tokens > VQ_PAGED_MAX_TOKENS || k_stride > INT64_MAX / 8 / VQ_PAGED_MAX_TOKENS ||
        v_stride > INT64_MAX / 8 / VQ_PAGED_MAX_TOKENS)
        return VQ_ERR_UNSUPPORTED;
    if (tokens == 0) return VQ_OK;
    const uintptr_t es = dtype == VQ_F32 ? 4 : 2;
    if (!k || !v || !slots || !k_codebooks || !v_codebooks || (num_pages > 0 && (!k_codes || !v_codes)))
        return VQ_ERR_INVALID_ARG;
    if ((uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)k_codebooks % es || (uintptr_t)v_codebooks % es ||
        (uintptr_t)slots % 8 || (uintptr_t)k_smooth % 4)
        return VQ_ERR_INVALID_ARG;
    if (num_pages == 0) return VQ_OK;  // no slot exists
    vqk::AppendArgs a{};
    a.x[0] = k;
    a.x[1] = v;
    a.codebooks[0] = k_codebooks;
    a.codebooks[1] = v_codebooks;
    a.codes[0] = k_codes;
    a.codes[1] = v_codes;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.smooth = k_smooth;
    a.slots = slots;
    a.tokens = tokens;
    a.num_pages = num_pages;
    a.page_stride = page_stride;
    a.heads = heads;
    a.ns = ns;
    a.sub = sub_dim;
    a.nc = n_centroids;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
    case VQ_F16: return launch<__half>(a, dtype, st);
    case VQ_BF16: return launch<__nv_bfloat16>(a, dtype, st);
    case VQ_F32: return launch<float>(a, dtype, st);
    }
    return VQ_ERR_INTERNAL;
}

}  // extern "C"
