// vq_pfew.cu -- launches of the paged attention of a few rows (vq_pfew.cuh).

#include <cuda_runtime.h>

#include "vq_host.h"
#include "vq_paged_host.h"
#include "vq_pfew.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_pfew)

namespace {

template <typename T, int D, int SUB, int NT>
vq_status launch(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    auto kernel = vqk::paged_attn_few<T, D, SUB, NT>;
    using S = vqk::FewShape<D, NT>;
    const size_t smem = S::kSmem;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return VQ_ERR_CUDA;
    kernel<<<(unsigned)blocks, S::kWarps * 32, smem, st>>>(a);
    return vqh_launched(st, vqh_status_pfew);
}

template <typename T, int SUB>
vq_status launch_dim(const vqk::PagedArgs &a, int nt, int blocks, cudaStream_t st)
{
    switch (a.dim) {
    case 64: return nt == 1 ? launch<T, 64, SUB, 1>(a, blocks, st) : launch<T, 64, SUB, 2>(a, blocks, st);
    case 128: return nt == 1 ? launch<T, 128, SUB, 1>(a, blocks, st) : launch<T, 128, SUB, 2>(a, blocks, st);
    case 256: return launch<T, 256, SUB, 1>(a, blocks, st);
    }
    return VQ_ERR_INTERNAL;
}

}  // namespace

int vqh_few_blocks_per_sm(int32_t dim, int nt)
{
    switch (dim) {
    case 64: return nt == 1 ? vqk::FewShape<64, 1>::kBlocks : vqk::FewShape<64, 2>::kBlocks;
    case 128: return nt == 1 ? vqk::FewShape<128, 1>::kBlocks : vqk::FewShape<128, 2>::kBlocks;
    }
    return vqk::FewShape<256, 1>::kBlocks;
}

vq_status vqh_paged_few(const vqk::PagedArgs &a, vq_dtype dtype, int nt, int blocks, cudaStream_t st)
{
    if (dtype == VQ_F16)
        return a.sub == 4 ? launch_dim<__half, 4>(a, nt, blocks, st) : launch_dim<__half, 8>(a, nt, blocks, st);
    return a.sub == 4 ? launch_dim<__nv_bfloat16, 4>(a, nt, blocks, st)
                      : launch_dim<__nv_bfloat16, 8>(a, nt, blocks, st);
}
