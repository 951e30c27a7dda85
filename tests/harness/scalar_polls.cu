// scalar_polls.cu -- test-only: the attention over 4-bit scalar codes with the library's chunk
// kernel (vq_pchunk.cuh, SUB = 2) at 0 or 1 polls a wait, as paged_polls.cu does it for
// product-VQ codes.  Built by the tests; not part of libvqenc.so.

// the entry points under names of their own; what paged_polls.cu defines is used from there
#define vq_paged_scalar_attention polls_scalar_attention
#define vq_paged_scalar_attention_workspace_bytes polls_scalar_attention_workspace_bytes
#define vqh_status_scache polls_status_scache
#define vqh_device_sms polls_device_sms
#define vqh_few_rows polls_few_rows
#define vqh_chunk_tiles polls_chunk_tiles
#define vqh_paged_sfew polls_paged_sfew
#define vqh_paged_schunk polls_paged_schunk

#include "vq_scache.cu"
#include "vq_pchunk.cuh"

namespace {

int scalar_polls = 0;

template <int D, int POLLS>
vq_status launch_polls(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    auto kernel = vqk::paged_attn_chunk<__half, D, 2, POLLS>;
    const size_t smem = vqk::ScalarChunk<D>::kSmem;
    if (!vqh_allow_smem(kernel, smem)) return vqh_failed();
    kernel<<<(unsigned)blocks, vqk::kChunkThreads, smem, st>>>(a);
    return vqh_launched(st, vqh_status_scache);
}

}  // namespace

vq_status vqh_paged_sfew(const vqk::PagedArgs &, vq_dtype, int, cudaStream_t) { return VQ_ERR_UNSUPPORTED; }

// fp16, head size 128 (0 or 1 polls) or 256 (1)
vq_status vqh_paged_schunk(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st)
{
    if (dtype != VQ_F16) return VQ_ERR_UNSUPPORTED;
    if (a.dim == 128) return scalar_polls == 0 ? launch_polls<128, 0>(a, blocks, st) : launch_polls<128, 1>(a, blocks, st);
    return a.dim == 256 && scalar_polls == 1 ? launch_polls<256, 1>(a, blocks, st) : VQ_ERR_UNSUPPORTED;
}

extern "C" void polls_scalar_set(int n) { scalar_polls = n; }

// This unit's device status word, optionally cleared.
extern "C" int polls_scalar_status(uint32_t *bits, int clear)
{
    *bits = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return 1;
    return vqh_status_scache(bits, clear != 0) != cudaSuccess;
}
