// vq_pagescan.cuh -- what the kernels over pages share: their limits, and prefix sums
// over a block's threads.
#pragma once

#include <stdint.h>

namespace vqk {

constexpr int kPageThreads = 1024;     // of a block; 256 for a small step
constexpr int kPageFewThreads = 256;
constexpr int kPageMaxRequests = 8192;  // three scanned arrays of it fit in shared memory

// Inclusive sums of (a, b) over the block's threads; every thread calls.
// `scratch` holds 2 * 32 values.
__device__ __forceinline__ void block_scan2(int64_t &a, int64_t &b, int64_t *scratch)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t pa = __shfl_up_sync(0xffffffffu, a, off), pb = __shfl_up_sync(0xffffffffu, b, off);
        if (lane >= off) {
            a += pa;
            b += pb;
        }
    }
    if (lane == 31) {
        scratch[warp] = a;
        scratch[32 + warp] = b;
    }
    __syncthreads();
    if (warp == 0) {
        int64_t wa = lane < warps ? scratch[lane] : 0, wb = lane < warps ? scratch[32 + lane] : 0;  // totals in 31 and 63
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int64_t pa = __shfl_up_sync(0xffffffffu, wa, off), pb = __shfl_up_sync(0xffffffffu, wb, off);
            if (lane >= off) {
                wa += pa;
                wb += pb;
            }
        }
        scratch[lane] = wa;
        scratch[32 + lane] = wb;
    }
    __syncthreads();
    if (warp > 0) {
        a += scratch[warp - 1];
        b += scratch[32 + warp - 1];
    }
}

__device__ __forceinline__ int32_t clamp_i32(int64_t v) { return (int32_t)(v > INT32_MAX ? INT32_MAX : v); }

}  // namespace vqk
