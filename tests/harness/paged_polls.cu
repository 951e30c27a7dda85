// paged_polls.cu -- test-only: the paged attention's entry point over the library's
// chunk kernel (vq_pchunk.cuh) with 0 or 1 polls a wait, so that waits give up while
// every product still completes: the path that marks the rows not written, records
// kStatusWaitGaveUp and frees tensor memory only after the last product.  That last wait
// keeps its full limit.  Built by the tests; not part of libvqenc.so.

// the entry points under names of their own
#define vq_paged_reserve polls_paged_reserve
#define vq_paged_trim polls_paged_trim
#define vq_paged_attention polls_paged_attention
#define vq_paged_attention_slots polls_paged_attention_slots
#define vq_paged_attention_workspace_bytes polls_paged_attention_workspace_bytes
#define vqh_status_paged polls_status_paged
#define vqh_device_sms polls_device_sms
#define vqh_few_rows polls_few_rows
#define vqh_few_blocks_per_sm polls_few_blocks_per_sm
#define vqh_chunk_tiles polls_chunk_tiles
#define vqh_paged_few polls_paged_few
#define vqh_paged_chunk polls_paged_chunk

#include "vq_paged.cu"
#include "vq_pchunk.cuh"

namespace {

int polls = 0;

template <int D, int POLLS>
vq_status launch(const vqk::PagedArgs &a, int blocks, cudaStream_t st)
{
    auto kernel = vqk::paged_attn_chunk<__half, D, 8, POLLS>;
    const size_t smem = vqk::ChunkShape<D>::kSmem;
    if (!vqh_allow_smem(kernel, smem)) return vqh_failed();
    kernel<<<(unsigned)blocks, vqk::kChunkThreads, smem, st>>>(a);
    return vqh_launched(st, vqh_status_paged);
}

}  // namespace

int vqh_device_sms()
{
    int dev = 0, sms = 0;
    (void)cudaGetDevice(&dev);
    (void)cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return sms;
}
int vqh_few_rows() { return vqk::kFewRows; }
int vqh_few_blocks_per_sm(int32_t dim) { return dim == 256 ? 1 : 2; }
int vqh_chunk_tiles(int32_t dim) { return dim == 256 ? 1 : 2; }
vq_status vqh_paged_few(const vqk::PagedArgs &, vq_dtype, int, cudaStream_t) { return VQ_ERR_UNSUPPORTED; }

// fp16, sub-vectors of 8, head size 128 (0 or 1 polls) or 256 (1)
vq_status vqh_paged_chunk(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st)
{
    if (dtype != VQ_F16 || a.sub != 8) return VQ_ERR_UNSUPPORTED;
    if (a.dim == 128) return polls == 0 ? launch<128, 0>(a, blocks, st) : launch<128, 1>(a, blocks, st);
    return a.dim == 256 && polls == 1 ? launch<256, 1>(a, blocks, st) : VQ_ERR_UNSUPPORTED;
}

extern "C" void polls_paged_set(int n) { polls = n; }

// This unit's device status word, optionally cleared.
extern "C" int polls_paged_status(uint32_t *bits, int clear)
{
    *bits = 0;
    if (cudaDeviceSynchronize() != cudaSuccess) return 1;
    return vqh_status_paged(bits, clear != 0) != cudaSuccess;
}
