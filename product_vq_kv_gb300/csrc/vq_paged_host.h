// vq_paged_host.h -- launches of the paged attention's tensor kernels, one
// translation unit each (internal; not part of the C ABI).
#pragma once

#include <cuda_runtime.h>

#include "vq_encode.h"

namespace vqk {
struct PagedArgs;
}

// A few rows (vq_pfew.cuh): items of vqh_few_rows rows; dim 64, 128 or 256, sub 4
// or 8, fp16 or bf16.
int vqh_few_rows();
int vqh_few_blocks_per_sm(int32_t dim);
vq_status vqh_paged_few(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st);

// Chunks (vq_pchunk.cuh): items of vqh_chunk_tiles tiles of 128 rows; one block
// an SM; dim 64, 128 or 256, sub 4 or 8, fp16 or bf16.
int vqh_chunk_tiles(int32_t dim);
vq_status vqh_paged_chunk(const vqk::PagedArgs &a, vq_dtype dtype, int blocks, cudaStream_t st);
