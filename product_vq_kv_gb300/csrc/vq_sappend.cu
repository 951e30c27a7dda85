// vq_sappend.cu -- C ABI entry point of the append to the paged cache of 4-bit scalar
// codes (see include/vq_encode.h for its contract).  Host side only.

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "vq_encode.h"
#include "vq_host.h"
#include "vq_sappend.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_sappend)

namespace {

template <typename T, int LANES, bool CUTS>
vq_status launch(const vqk::ScalarAppendArgs &a, cudaStream_t st)
{
    constexpr int kRows = vqk::kSAppendThreads / LANES;  // of a block
    const int64_t want = (a.tokens * a.heads + kRows - 1) / kRows;
    // three blocks an SM, keys and values: a block's set-up is worth several rows a warp
    const int64_t most = 3 * (int64_t)(vqh_device_sms() > 0 ? vqh_device_sms() : 152) / 2;
    vqk::scalar_append<T, LANES, CUTS><<<dim3((unsigned)(want < most ? want : most), 2), vqk::kSAppendThreads, 0, st>>>(a);
    return vqh_launched(st, vqh_status_sappend);
}

template <typename T, int LANES>
vq_status launch_nc(const vqk::ScalarAppendArgs &a, cudaStream_t st)
{
    return a.nc == 16 ? launch<T, LANES, true>(a, st) : launch<T, LANES, false>(a, st);
}

template <typename T>
vq_status launch_dim(const vqk::ScalarAppendArgs &a, cudaStream_t st)
{
    if (a.dim <= 16) return launch_nc<T, 1>(a, st);
    if (a.dim <= 32) return launch_nc<T, 2>(a, st);
    if (a.dim <= 64) return launch_nc<T, 4>(a, st);
    if (a.dim <= 128) return launch_nc<T, 8>(a, st);
    if (a.dim <= 256) return launch_nc<T, 16>(a, st);
    return launch_nc<T, 32>(a, st);
}

}  // namespace

extern "C" {

vq_status vq_paged_scalar_append(const void *k, const void *v, int64_t k_stride, int64_t v_stride,
                                 const int64_t *slots, int64_t tokens, int32_t heads, int32_t head_dim,
                                 int32_t n_centroids, const float *k_centroids, const float *v_centroids,
                                 const float *k_signs, uint8_t *k_codes, uint8_t *v_codes, void *k_scales,
                                 void *v_scales, int64_t num_pages, int32_t page_size, int64_t page_stride,
                                 int64_t scale_stride, vq_dtype dtype, vq_stream_t stream)
{
    if (dtype != VQ_F16 && dtype != VQ_BF16 && dtype != VQ_F32) return VQ_ERR_INVALID_ARG;
    if (tokens < 0 || num_pages < 0 || heads < 1 || head_dim < 2 || head_dim % 2) return VQ_ERR_INVALID_ARG;
    if (head_dim > VQ_PAGED_MAX_HEAD_DIM || heads > VQ_PAGED_MAX_HEADS || n_centroids < 1 ||
        n_centroids > VQ_PAGED_SCALAR_MAX_CENTROIDS)
        return VQ_ERR_UNSUPPORTED;
    if (k_signs && (head_dim & (head_dim - 1))) return VQ_ERR_UNSUPPORTED;
    if (page_size < 1 || (page_size & (page_size - 1))) return VQ_ERR_INVALID_ARG;
    if (page_size > VQ_PAGED_MAX_PAGE) return VQ_ERR_UNSUPPORTED;
    const int64_t page_rows = (int64_t)heads * page_size;
    if (page_stride < page_rows * (head_dim / 2) || scale_stride < page_rows || num_pages > (INT64_MAX >> 20) / page_size)
        return VQ_ERR_INVALID_ARG;
    if (num_pages > 1 && (page_stride > INT64_MAX / num_pages || scale_stride > INT64_MAX / 4 / num_pages))
        return VQ_ERR_INVALID_ARG;
    const int64_t row = (int64_t)heads * head_dim;
    if (k_stride < row || v_stride < row) return VQ_ERR_INVALID_ARG;
    if (tokens > VQ_PAGED_MAX_TOKENS || k_stride > INT64_MAX / 8 / VQ_PAGED_MAX_TOKENS ||
        v_stride > INT64_MAX / 8 / VQ_PAGED_MAX_TOKENS)
        return VQ_ERR_UNSUPPORTED;
    if (tokens == 0) return VQ_OK;
    const uintptr_t es = dtype == VQ_F32 ? 4 : 2;
    if (!k || !v || !slots || !k_centroids || !v_centroids ||
        (num_pages > 0 && (!k_codes || !v_codes || !k_scales || !v_scales)))
        return VQ_ERR_INVALID_ARG;
    if ((uintptr_t)k % es || (uintptr_t)v % es || (uintptr_t)k_scales % es || (uintptr_t)v_scales % es ||
        (uintptr_t)slots % 8 || (uintptr_t)k_centroids % 4 || (uintptr_t)v_centroids % 4 || (uintptr_t)k_signs % 4)
        return VQ_ERR_INVALID_ARG;
    if (num_pages == 0) return VQ_OK;  // no slot exists
    vqk::ScalarAppendArgs a{};
    a.x[0] = k;
    a.x[1] = v;
    a.centroids[0] = k_centroids;
    a.centroids[1] = v_centroids;
    a.codes[0] = k_codes;
    a.codes[1] = v_codes;
    a.scales[0] = k_scales;
    a.scales[1] = v_scales;
    a.stride[0] = k_stride;
    a.stride[1] = v_stride;
    a.signs = k_signs;
    a.slots = slots;
    a.tokens = tokens;
    a.num_pages = num_pages;
    a.page_stride = page_stride;
    a.scale_stride = scale_stride;
    a.heads = heads;
    a.dim = head_dim;
    a.nc = n_centroids;
    while ((1 << a.page_shift) < page_size) ++a.page_shift;
    a.norm = (float)(1.0 / std::sqrt((double)head_dim));
    a.over_dim = (float)(1.0 / head_dim);
    a.exact = (head_dim & (head_dim - 1)) == 0;
    // rows of whole runs, each 16-byte aligned
    const bool runs = head_dim >= vqk::kRowRun && a.exact;
    for (int kv = 0; kv < 2; ++kv)
        a.vec[kv] = runs && (uintptr_t)a.x[kv] % 16 == 0 && a.stride[kv] * (int64_t)es % 16 == 0;
    a.vec_codes = head_dim % vqk::kRowRun == 0 && (uintptr_t)k_codes % 8 == 0 && (uintptr_t)v_codes % 8 == 0 &&
                  page_stride % 8 == 0;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    switch (dtype) {
    case VQ_F16: return launch_dim<__half>(a, st);
    case VQ_BF16: return launch_dim<__nv_bfloat16>(a, st);
    case VQ_F32: return launch_dim<float>(a, st);
    }
    return VQ_ERR_INTERNAL;
}

}  // extern "C"
