// vq_sfew.cu -- launches of the paged attention of a few rows over 4-bit scalar codes
// (vq_sfew.cuh).

#include <cuda_runtime.h>

#include "vq_host.h"
#include "vq_paged_host.h"
#include "vq_sfew.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_sfew)

namespace {

template <typename T, int D, bool PAIR>
vq_status launch_rows(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    auto kernel = vqk::paged_attn_sfew<T, D, PAIR>;
    using S = vqk::SFewShape<D>;
    if (!vqh_allow_smem(kernel, S::kSmem)) return vqh_failed();
    kernel<<<(unsigned)blocks, S::kWarps * 32, S::kSmem, st>>>(a);
    return vqh_launched(st, vqh_status_sfew);
}

template <typename T, int D>
vq_status launch(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    return a.tile_rows <= 4 ? launch_rows<T, D, true>(a, blocks, st) : launch_rows<T, D, false>(a, blocks, st);
}

template <typename T>
vq_status launch_dim(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    switch (a.dim) {
    case 64: return launch<T, 64>(a, blocks, st);
    case 128: return launch<T, 128>(a, blocks, st);
    case 256: return launch<T, 256>(a, blocks, st);
    }
    return VQ_ERR_INTERNAL;
}

}  // namespace

vq_status vqh_paged_sfew(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st)
{
    return dtype == VQ_F16 ? launch_dim<__half>(a, blocks, st) : launch_dim<__nv_bfloat16>(a, blocks, st);
}
