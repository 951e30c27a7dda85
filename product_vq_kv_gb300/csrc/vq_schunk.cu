// vq_schunk.cu -- launches of the paged attention of chunks over 4-bit scalar codes
// (vq_pchunk.cuh with SUB = 2).

#include <cuda_runtime.h>

#include "vq_host.h"
#include "vq_paged_host.h"
#include "vq_pchunk.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_schunk)

namespace {

template <typename T, int D>
vq_status launch(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    auto kernel = vqk::paged_attn_chunk<T, D, 2>;
    const size_t smem = vqk::ScalarChunk<D>::kSmem;
    if (!vqh_allow_smem(kernel, smem)) return vqh_failed();
    kernel<<<(unsigned)blocks, vqk::kChunkThreads, smem, st>>>(a);
    return vqh_launched(st, vqh_status_schunk);
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

vq_status vqh_paged_schunk(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st)
{
    return dtype == VQ_F16 ? launch_dim<__half>(a, blocks, st) : launch_dim<__nv_bfloat16>(a, blocks, st);
}
