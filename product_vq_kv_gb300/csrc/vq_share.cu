// vq_share.cu -- C ABI entry points of shared pages: fork, compact and copy (see
// include/vq_encode.h for the contract of each).  Host side only.

#include <cuda_runtime.h>

#include <cstdint>

#include "vq_encode.h"
#include "vq_host.h"
#include "vq_paged_plan.h"
#include "vq_share.cuh"
#include "vq_status.cuh"

VQH_STATUS_READER(vqh_status_share)

namespace {

using namespace vqp;

// A launch that may start while the one before it ends (the kernel waits for that).
template <typename Kernel, typename Args>
bool launch_after(Kernel *kernel, int blocks, int threads, size_t smem, int cluster, cudaStream_t st, const Args &args)
{
    cudaLaunchAttribute attr[2];
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, args) == cudaSuccess;
}

// Blocks of `per` items that cover `items`, at most four an SM.
int spread(int64_t items, int per)
{
    const int sms = vqh_device_sms() > 0 ? vqh_device_sms() : 152;
    const int64_t want = (items + per - 1) / per;
    return (int)(want < 1 ? 1 : want > 4 * sms ? 4 * sms : want);
}

// Blocks of the cluster that goes through the pages: one for up to per_block.
int page_cluster(int64_t num_pages, int per_block)
{
    int blocks = 1;
    while (blocks < 8 && num_pages > (int64_t)blocks * per_block) blocks *= 2;
    return blocks;
}

}  // namespace

extern "C" {

size_t vq_paged_fork_workspace_bytes(int64_t num_pages)
{
    if (num_pages < 0 || num_pages > INT32_MAX) return 0;
    const size_t padded = up256((size_t)num_pages);  // (the flags are cleared 16 at a time)
    return 2 * padded + padded * 4;
}

vq_status vq_paged_fork(const int32_t *lens, const int32_t *parents, const int32_t *keep_lens, int64_t seats,
                        const int32_t *block_table, int64_t max_blocks, int32_t page_size, int32_t *free_pages,
                        const int32_t *free_count, int64_t num_pages, int32_t *lens_out, int32_t *table_out,
                        int32_t *free_count_out, int32_t *copies, void *workspace, size_t workspace_bytes,
                        vq_stream_t stream)
{
    vq_status s = check_pool(seats, max_blocks, page_size, num_pages);
    if (s != VQ_OK) return s;
    if (!free_count || !free_count_out || (num_pages > 0 && (!free_pages || !workspace))) return VQ_ERR_INVALID_ARG;
    if (seats > 0 && (!lens || !parents || !lens_out || !copies || (max_blocks > 0 && (!block_table || !table_out))))
        return VQ_ERR_INVALID_ARG;
    for (const void *p : {(const void *)lens, (const void *)parents, (const void *)keep_lens, (const void *)block_table,
                          (const void *)free_pages, (const void *)free_count, (const void *)lens_out,
                          (const void *)table_out, (const void *)free_count_out, (const void *)copies})
        if (!aligned4(p)) return VQ_ERR_INVALID_ARG;
    if ((uintptr_t)workspace % 16 || workspace_bytes < vq_paged_fork_workspace_bytes(num_pages)) return VQ_ERR_INVALID_ARG;
    // rows are read while others are written
    const int64_t entries = seats * max_blocks;
    if (entries > 0 && block_table < table_out + entries && table_out < block_table + entries) return VQ_ERR_INVALID_ARG;

    vqk::ForkArgs a{};
    a.lens = lens;
    a.parents = parents;
    a.keep = keep_lens;
    a.table = block_table;
    a.table_out = table_out;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.lens_out = lens_out;
    a.free_count_out = free_count_out;
    a.copies = copies;
    a.before = static_cast<uint8_t *>(workspace);
    a.whole = a.before + up256((size_t)num_pages);
    a.first = reinterpret_cast<int32_t *>(a.whole + up256((size_t)num_pages));
    a.seats = (int32_t)seats;
    a.max_blocks = (int32_t)max_blocks;
    a.page_shift = page_shift(page_size);
    a.num_pages = (int32_t)num_pages;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const size_t smem = vqk::fork_finish_smem(seats);
    const int64_t segments = seats * ((max_blocks + vqk::kForkSegment - 1) / vqk::kForkSegment);
    vqk::fork_clear<<<(unsigned)spread((num_pages + 15) / 16, vqk::kForkThreads), vqk::kForkThreads, 0, st>>>(a);
    if ((s = vqh_launched(st, vqh_status_share)) != VQ_OK) return s;
    if (!launch_after(vqk::fork_mark, spread(segments, vqk::kForkThreads / 32), vqk::kForkThreads, 0, 1, st, a))
        return vqh_failed();
    if ((s = vqh_launched(st, vqh_status_share)) != VQ_OK) return s;
    const int blocks = page_cluster(num_pages, 16 * vqk::kPageThreads);
    if (!launch_after(vqk::fork_finish, blocks, vqk::kPageThreads, smem, blocks, st, a)) return vqh_failed();
    return vqh_launched(st, vqh_status_share);
}

size_t vq_paged_compact_workspace_bytes(int64_t num_pages)
{
    return num_pages < 0 || num_pages > INT32_MAX ? 0 : up256((size_t)(num_pages + 31) / 32 * 4);
}

vq_status vq_paged_compact(const int32_t *lens, int64_t requests, const int32_t *block_table, int64_t max_blocks,
                           int32_t page_size, const int32_t *free_pages, const int32_t *free_count,
                           int64_t num_pages, int32_t *table_out, int32_t *free_pages_out,
                           int32_t *free_count_out, int32_t *moves, int32_t *page_map, void *workspace,
                           size_t workspace_bytes, vq_stream_t stream)
{
    vq_status s = check_pool(requests, max_blocks, page_size, num_pages);
    if (s != VQ_OK) return s;
    if (!free_count || !free_count_out || (num_pages > 0 && (!free_pages || !free_pages_out || !page_map)))
        return VQ_ERR_INVALID_ARG;
    if ((num_pages > 1 && !moves) || (num_pages > 0 && !workspace)) return VQ_ERR_INVALID_ARG;
    if ((uintptr_t)workspace % 16 || workspace_bytes < vq_paged_compact_workspace_bytes(num_pages)) return VQ_ERR_INVALID_ARG;
    if (requests > 0 && (!lens || (max_blocks > 0 && (!block_table || !table_out)))) return VQ_ERR_INVALID_ARG;
    for (const void *p : {(const void *)lens, (const void *)block_table, (const void *)free_pages,
                          (const void *)free_count, (const void *)table_out, (const void *)free_pages_out,
                          (const void *)free_count_out, (const void *)moves, (const void *)page_map})
        if (!aligned4(p)) return VQ_ERR_INVALID_ARG;
    vqk::CompactArgs a{};
    a.lens = lens;
    a.table = block_table;
    a.table_out = table_out;
    a.free_pages = free_pages;
    a.free_count = free_count;
    a.free_out = free_pages_out;
    a.free_count_out = free_count_out;
    a.moves = moves;
    a.map = page_map;
    a.idle = static_cast<uint32_t *>(workspace);
    a.requests = (int32_t)requests;
    a.max_blocks = (int32_t)max_blocks;
    a.page_shift = page_shift(page_size);
    a.num_pages = (int32_t)num_pages;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    const int blocks = page_cluster(num_pages, 4 * vqk::kPageThreads);  // (for the lists: the bits would take fewer)
    cudaLaunchConfig_t cfg = cluster_launch(blocks, vqk::kPageThreads, 0, st, attr);
    if (cudaLaunchKernelEx(&cfg, vqk::compact_plan, a) != cudaSuccess) return vqh_failed();
    if ((s = vqh_launched(st, vqh_status_share)) != VQ_OK) return s;
    const int64_t entries = requests * max_blocks;
    if (entries == 0) return VQ_OK;
    if (!launch_after(vqk::compact_table, spread(entries, vqk::kForkThreads), vqk::kForkThreads, 0, 1, st, a))
        return vqh_failed();
    return vqh_launched(st, vqh_status_share);
}

vq_status vq_paged_copy(const int32_t *pairs, int64_t n_pairs, const vq_page_pool *pools, int32_t n_pools,
                        int64_t num_pages, vq_stream_t stream)
{
    if (n_pairs < 0 || n_pools < 0 || num_pages < 0) return VQ_ERR_INVALID_ARG;
    if (n_pools > VQ_PAGED_MAX_POOLS || num_pages > INT32_MAX || n_pairs > VQ_PAGED_MAX_TOKENS) return VQ_ERR_UNSUPPORTED;
    if (n_pairs == 0 || n_pools == 0 || num_pages == 0) return VQ_OK;
    if (!pairs || !pools || !aligned4(pairs)) return VQ_ERR_INVALID_ARG;
    static_assert(VQ_PAGED_MAX_POOLS == vqk::kCopyPools, "pools of a copy");
    vqk::CopyArgs a{};
    a.pairs = pairs;
    a.n_pairs = n_pairs;
    a.num_pages = num_pages;
    int64_t total = 0;
    for (int32_t i = 0; i < n_pools; ++i) {
        const vq_page_pool &p = pools[i];
        if (p.layers < 0 || p.page_bytes < 0) return VQ_ERR_INVALID_ARG;
        if (p.layers == 0 || p.page_bytes == 0) continue;
        if (!p.base) return VQ_ERR_INVALID_ARG;
        // pages of a layer do not overlap, nor do layers
        if ((num_pages > 1 && p.page_stride < p.page_bytes) || p.page_stride > INT64_MAX / 4 / num_pages ||
            p.layer_stride > INT64_MAX / 4 / p.layers)
            return VQ_ERR_INVALID_ARG;
        const int64_t span = (num_pages - 1) * p.page_stride + p.page_bytes;
        // layers behind one another, or inside one another's pages (pool[page][layer])
        if (p.layers > 1 && p.layer_stride < span &&
            (p.layer_stride < p.page_bytes || (num_pages > 1 && p.page_stride < (p.layers - 1) * p.layer_stride + p.page_bytes)))
            return VQ_ERR_INVALID_ARG;
        vqk::CopyPool &to = a.pool[a.n_pools++];
        to.base = static_cast<unsigned char *>(p.base);
        to.page_stride = p.page_stride;
        to.page_bytes = p.page_bytes;
        to.layer_stride = p.layer_stride;
        to.layers = p.layers;
        const uint64_t low = (uint64_t)(uintptr_t)p.base | (uint64_t)p.page_bytes |
                             (num_pages > 1 ? (uint64_t)p.page_stride : 0) | (p.layers > 1 ? (uint64_t)p.layer_stride : 0);
        to.vec = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : 1;
        const int64_t pieces = (p.page_bytes + vqk::kCopyPiece - 1) / vqk::kCopyPiece;
        if (pieces > INT32_MAX / p.layers || total + pieces * p.layers > INT32_MAX) return VQ_ERR_UNSUPPORTED;
        to.pieces = (int32_t)pieces;
        to.first = (int32_t)total;
        total += pieces * p.layers;
    }
    if (a.n_pools == 0) return VQ_OK;
    a.total = (int32_t)total;
    const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    const int sms = vqh_device_sms() > 0 ? vqh_device_sms() : 152;
    // a warp a piece, up to what an SM holds
    const int64_t most = total < INT64_MAX / n_pairs ? total * n_pairs : INT64_MAX;
    const int64_t want = (most - 1) / (vqk::kCopyThreads / 32) + 1;
    const int blocks = (int)(want < 4 * (int64_t)sms ? want : 4 * (int64_t)sms);
    vqk::copy_pages<<<(unsigned)blocks, vqk::kCopyThreads, 0, st>>>(a);
    return vqh_launched(st, vqh_status_share);
}

}  // extern "C"
