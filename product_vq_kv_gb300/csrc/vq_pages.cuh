// vq_pages.cuh -- pages of the paged code cache: the block table and the slot
// map of new tokens from request lengths (reserve), and the way back (trim).
//
// With P = page_size, L_r the tokens request r holds and n_r its new ones:
//   need_r = ceil((L_r + n_r) / P) - ceil(L_r / P)     (0 if the table is too narrow)
//   c_r    = need_0 + .. + need_r
//   r is granted iff L_r + n_r <= max_blocks P and (need_r = 0 or c_r <= free)
// and page number k of the sequence (request order, then block order) is
// free_pages[free - 1 - k]: the free list is a stack.  A trim of r to keep_r
// tokens pushes pages ceil(keep_r / P) .. ceil(L_r / P) - 1 back in the same
// order.  Every result is fixed by these sums: no atomics, no order of arrival.
//
// What bounds it: latency.  A decode step of 64 requests moves 1.6 KB and takes 6.2
// us on the device (a graph's replay; 8.3 with 1024 threads where 256 do); a burst
// of 257 prompts moves 1.1 MB, a fifth of a microsecond of HBM time.  So one launch does
// everything: a cluster of 1 to 8 blocks, each of which scans all the requests
// by itself (two 64-bit sums a request: warp shuffles, then one over the warps)
// and keeps the scanned arrays in shared memory; then the blocks share out the
// table entries (one warp per request) and the slots (one thread per token, a
// binary search in shared memory).  The cluster barrier between the last read
// of lens / free_count and the first write lets the caller update both in
// place.
#pragma once

#include <cooperative_groups.h>
#include <stdint.h>

#include "vq_check.cuh"

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

// Launch: one cluster (gridDim.x = cluster size), up to kPageThreads threads,
// dynamic shared memory page_reserve_smem(requests).
__host__ __device__ inline size_t page_reserve_smem(int64_t requests)
{
    return 64 * 8 + (size_t)(3 * requests + 1) * 4;
}

__global__ void __launch_bounds__(kPageThreads)
    page_reserve(const int32_t *lens, const int32_t *new_lens, int32_t requests,
                 const int32_t *__restrict__ free_pages, const int32_t *free_count, int32_t num_pages,
                 int32_t *__restrict__ table, int32_t max_blocks, int32_t page_shift, int64_t total_new,
                 int32_t *lens_out, int32_t *free_count_out, int32_t *__restrict__ cu_new,
                 int64_t *__restrict__ slots)
{
    extern __shared__ __align__(16) unsigned char page_smem[];
    int64_t *scratch = reinterpret_cast<int64_t *>(page_smem);
    int32_t *cu = reinterpret_cast<int32_t *>(scratch + 64);  // [requests + 1]: first token of each request
    int32_t *held = cu + requests + 1;                        // [requests]: L_r
    int32_t *take = held + requests;                          // [requests]: pages taken before r; -1: refused
    auto cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x;
    const int rank = blockIdx.x, blocks = gridDim.x, threads = blockDim.x;
    const int64_t page = (int64_t)1 << page_shift, cap = (int64_t)max_blocks << page_shift;
    const int32_t fc = *free_count;
    const int64_t avail = fc < 0 ? 0 : fc > num_pages ? num_pages : fc;

    int64_t tok_base = 0, need_base = 0;
    for (int base = 0; base < requests; base += threads) {
        const int r = base + tid;
        int64_t l = 0, n = 0, need = 0;
        bool fits = false;
        if (r < requests) {
            l = lens[r] > 0 ? lens[r] : 0;
            n = new_lens[r] > 0 ? new_lens[r] : 0;
            fits = l + n <= cap;
            need = fits ? ((l + n + page - 1) >> page_shift) - ((l + page - 1) >> page_shift) : 0;
        }
        int64_t ts = n, ns = need;
        block_scan2(ts, ns, scratch);
        if (r < requests) {
            const bool granted = fits && (need == 0 || need_base + ns <= avail);
            cu[r] = clamp_i32(tok_base + ts - n);
            held[r] = (int32_t)l;
            // a granted request with need has c_r <= avail, so its start fits; one without needs none
            take[r] = granted ? (need ? (int32_t)(need_base + ns - need) : 0) : -1;
        }
        tok_base += scratch[31];
        need_base += scratch[63];
        __syncthreads();  // before the next pass writes scratch
    }
    if (tid == 0) cu[requests] = clamp_i32(tok_base);
    __syncthreads();

    auto new_of = [&](int r) { return (int64_t)(cu[r + 1] - cu[r]); };
    // the pages of the granted requests are a prefix of the sequence: its length
    // (at most free_count, so 32 bits hold it)
    uint32_t mine = 0;
    for (int r = tid; r < requests; r += threads) {
        if (take[r] < 0) continue;
        const int64_t l = held[r];
        const int64_t need = ((l + new_of(r) + page - 1) >> page_shift) - ((l + page - 1) >> page_shift);
        if (need && take[r] + need > mine) mine = (uint32_t)(take[r] + need);
    }
    mine = __reduce_max_sync(0xffffffffu, mine);
    if ((tid & 31) == 0) scratch[tid >> 5] = mine;
    __syncthreads();
    const int64_t taken = __reduce_max_sync(0xffffffffu, (tid & 31) < (threads >> 5) ? (uint32_t)scratch[tid & 31] : 0u);

    // table entries of the new pages: a warp per request (new entries only, so
    // no other thread's read of a held page meets a write)
    const int warps = blocks * (threads >> 5), lane = tid & 31;
    for (int r = rank * (threads >> 5) + (tid >> 5); r < requests; r += warps) {
        if (take[r] < 0) continue;
        const int64_t l = held[r];
        const int64_t b0 = (l + page - 1) >> page_shift, b1 = (l + new_of(r) + page - 1) >> page_shift;
        for (int64_t b = b0 + lane; b < b1; b += 32) {
            const int64_t at = avail - 1 - take[r] - (b - b0);
            int32_t *dst = table + (int64_t)r * max_blocks + b;
            if (VQ_SPAN(free_pages + at, 1, free_pages, num_pages) &&
                VQ_SPAN(dst, 1, table, (int64_t)requests * max_blocks))
                *dst = free_pages[at];
        }
    }

    // slots: a thread per token
    for (int64_t t = (int64_t)rank * threads + tid; t < total_new; t += (int64_t)blocks * threads) {
        int64_t slot = -1;
        if (t < cu[requests]) {
            int lo = 0, hi = requests - 1;  // the last r with cu[r] <= t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (cu[mid] <= t) lo = mid;
                else hi = mid - 1;
            }
            if (take[lo] >= 0) {
                const int64_t l = held[lo], p = l + (t - cu[lo]);
                const int64_t b = p >> page_shift, b0 = (l + page - 1) >> page_shift;
                int32_t pg = -1;
                if (b < b0) {
                    if (VQ_SPAN(table + (int64_t)lo * max_blocks + b, 1, table, (int64_t)requests * max_blocks))
                        pg = table[(int64_t)lo * max_blocks + b];
                } else {
                    const int64_t at = avail - 1 - take[lo] - (b - b0);
                    if (VQ_SPAN(free_pages + at, 1, free_pages, num_pages)) pg = free_pages[at];
                }
                if (pg >= 0) slot = ((int64_t)pg << page_shift) + (p & (page - 1));
            }
        }
        if (VQ_SPAN(slots + t, 1, slots, total_new)) slots[t] = slot;
    }

    cluster.sync();  // lens and free_count have been read by every block
    for (int r = rank * threads + tid; r < requests; r += blocks * threads) {
        lens_out[r] = (int32_t)(held[r] + (take[r] >= 0 ? new_of(r) : 0));
        cu_new[r] = cu[r];
    }
    if (rank == 0 && tid == 0) {
        cu_new[requests] = cu[requests];
        *free_count_out = (int32_t)(avail - taken);
    }
}

// Launch: one cluster, up to kPageThreads threads, dynamic shared memory
// page_trim_smem(requests).
__host__ __device__ inline size_t page_trim_smem(int64_t requests)
{
    return 64 * 8 + (size_t)(3 * requests) * 4;
}

__global__ void __launch_bounds__(kPageThreads)
    page_trim(const int32_t *lens, const int32_t *keep_lens, int32_t requests,
              const int32_t *__restrict__ table, int32_t max_blocks, int32_t page_shift,
              int32_t *__restrict__ free_pages, const int32_t *free_count, int32_t num_pages,
              int32_t *lens_out, int32_t *free_count_out)
{
    extern __shared__ __align__(16) unsigned char page_smem[];
    int64_t *scratch = reinterpret_cast<int64_t *>(page_smem);
    int32_t *first = reinterpret_cast<int32_t *>(scratch + 64);  // pages returned before r
    int32_t *kept = first + requests;                            // tokens kept
    int32_t *back = kept + requests;                             // pages returned
    auto cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x;
    const int rank = blockIdx.x, blocks = gridDim.x, threads = blockDim.x;
    const int64_t page = (int64_t)1 << page_shift, cap = (int64_t)max_blocks << page_shift;
    const int32_t fc = *free_count;
    const int64_t avail = fc < 0 ? 0 : fc > num_pages ? num_pages : fc;

    int64_t base_pages = 0;
    for (int base = 0; base < requests; base += threads) {
        const int r = base + tid;
        int64_t l = 0, k = 0, n = 0, unused = 0;
        if (r < requests) {
            l = lens[r] > 0 ? lens[r] : 0;
            if (l > cap) l = cap;
            k = keep_lens[r] > 0 ? keep_lens[r] : 0;
            if (k > l) k = l;
            n = ((l + page - 1) >> page_shift) - ((k + page - 1) >> page_shift);
        }
        int64_t s = n;
        block_scan2(s, unused, scratch);
        if (r < requests) {
            first[r] = clamp_i32(base_pages + s - n);
            kept[r] = (int32_t)k;
            back[r] = (int32_t)n;
        }
        base_pages += scratch[31];
        __syncthreads();
    }

    const int warps = blocks * (threads >> 5), lane = tid & 31;
    for (int r = rank * (threads >> 5) + (tid >> 5); r < requests; r += warps) {
        const int64_t b0 = (kept[r] + page - 1) >> page_shift;
        for (int i = lane; i < back[r]; i += 32) {
            const int64_t at = avail + first[r] + i;
            const int32_t *src = table + (int64_t)r * max_blocks + b0 + i;
            // a list that would overflow (more pages held than the pool has) drops the rest
            if (at < num_pages && VQ_SPAN(src, 1, table, (int64_t)requests * max_blocks) &&
                VQ_SPAN(free_pages + at, 1, free_pages, num_pages))
                free_pages[at] = *src;
        }
    }

    cluster.sync();  // lens and free_count have been read by every block
    for (int r = rank * threads + tid; r < requests; r += blocks * threads) lens_out[r] = kept[r];
    if (rank == 0 && tid == 0) {
        const int64_t n = avail + base_pages;
        *free_count_out = (int32_t)(n > num_pages ? num_pages : n);
    }
}

}  // namespace vqk
