// vq_pchunk.cu -- launches of the paged attention of chunks (vq_pchunk.cuh).

#include <cuda_runtime.h>

#include "vq_host.h"
#include "vq_paged_host.h"
#include "vq_pchunk.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_pchunk)

// The waits of a segment outlast the longest one: 2 us a unit (1.9 at dim 128), at 3.5
// us a poll.
static_assert(vqk::kSegmentPolls / 2 * 7 > VQ_PAGED_MAX_TOKENS / vqk::kUnit * 2, "a segment's waits would give up");

namespace {

template <typename T, int D, int SUB>
vq_status launch(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    auto kernel = vqk::paged_attn_chunk<T, D, SUB>;
    const size_t smem = vqk::ChunkShape<D>::kSmem;
    if (!vqh_allow_smem(kernel, smem)) return vqh_failed();
    kernel<<<(unsigned)blocks, vqk::kChunkThreads, smem, st>>>(a);
    return vqh_launched(st, vqh_status_pchunk);
}

template <typename T, int SUB>
vq_status launch_dim(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    switch (a.dim) {
    case 64: return launch<T, 64, SUB>(a, blocks, st);
    case 128: return launch<T, 128, SUB>(a, blocks, st);
    case 256: return launch<T, 256, SUB>(a, blocks, st);
    }
    return VQ_ERR_INTERNAL;
}

}  // namespace

int vqh_chunk_tiles(int32_t dim) { return dim == 256 ? vqk::ChunkShape<256>::kTiles : vqk::ChunkShape<128>::kTiles; }

vq_status vqh_paged_chunk(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st)
{
    if (dtype == VQ_F16)
        return a.sub == 4 ? launch_dim<__half, 4>(a, blocks, st) : launch_dim<__half, 8>(a, blocks, st);
    return a.sub == 4 ? launch_dim<__nv_bfloat16, 4>(a, blocks, st) : launch_dim<__nv_bfloat16, 8>(a, blocks, st);
}
