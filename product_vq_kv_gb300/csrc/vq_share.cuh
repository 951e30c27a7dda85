// vq_share.cuh -- pages held by several requests: forking (beams, samples of one
// prompt), bringing a pool together, and the copies of pages that both ask for.
//
// Fork.  With P = page_size, seat d takes the first
//   k_d = min(keep_d, L_p) tokens of its parent p (none if p is no seat),
// that is pages table[p][0 .. ceil(k_d / P)).  A page counts as whole for a seat
// whose tokens fill it, as a part for the seat that ends inside it.  Then
//   freed = pages of the old rows that no new row holds, pushed on the free list
//           in ascending order;
//   a seat that holds a page as a part gives it up for a copy if any seat holds
//   it whole, or a lower seat holds it as a part: copy number i (in seat order)
//   goes to the i-th page from the top of the list, if there is one, else the seat
//   is cut to its whole pages.
// So the page that a seat writes its next token to is its own.  Every result is
// fixed by flags (set by anyone, in any order), a minimum over seats and prefix
// sums: no order of arrival.
//
// What bounds it: the table is read twice and written once, at scattered flags of
// one byte a page.  256 seats of 150 pages move 0.2 MB, so launches and their
// dependent loads count: three launches, each started while the one before ends (26 us on the
// device with a cold cache, 30 us for 800 seats of up to 577 pages; one launch of a cluster of
// eight blocks took 13 us where three take 15 for four seats, but 30 and 75 us here).
//
// Compact.  used = pages that are not on the free list.  The i-th held page at or
// past `used` moves to the i-th free page below it.  Bound by latency too: a bit a page, so that
// 200,000 pages are one word for each thread of a cluster, and counts of bits (4,096 pages 19 us
// on the device with a cold cache, 200,000 of 1000 requests 34; with a byte a page 49).
//
// Copy.  Pairs of pages in up to kCopyPools pools, each of any number of layers.
// Bound by HBM: every byte is read and written once; a warp takes 4 KiB of one page
// at a time, eight 16-byte loads in flight a lane (2047 pages of eight layers, 278 MB: 92 us, 89 % of
// the rate of a plain copy; pieces of 2 and 8 KiB and two to eight blocks an SM are no faster).
#pragma once

#include <cooperative_groups.h>
#include <stdint.h>

#include "vq_check.cuh"
#include "vq_pagescan.cuh"

namespace vqk {

struct ForkArgs {
    const int32_t *lens, *parents, *keep;  // keep: or null
    const int32_t *table;
    int32_t *table_out;
    int32_t *free_pages;
    const int32_t *free_count;
    int32_t *lens_out, *free_count_out;
    int32_t *copies;  // [seats][2]
    uint8_t *before;  // [num_pages] 1: an old row holds it
    uint8_t *whole;   // [num_pages] 1: a new row holds it whole
    int32_t *first;   // [num_pages] the lowest seat that holds it as a part, else kNoSeat
    int32_t seats, max_blocks, page_shift, num_pages;
};

constexpr int32_t kNoSeat = INT32_MAX;
constexpr int kForkThreads = 256;
constexpr int kForkSegment = 128;  // entries of a row that a warp takes at a time

__device__ __forceinline__ int32_t fork_held(const ForkArgs &a, int32_t seat)
{
    const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
    if (!VQ_SPAN(a.lens + seat, 1, a.lens, a.seats)) return 0;
    const int64_t l = a.lens[seat];
    return (int32_t)(l < 0 ? 0 : l > cap ? cap : l);
}

// The parent of a seat, -1 if it has none, and the tokens it takes.
__device__ __forceinline__ int32_t fork_parent(const ForkArgs &a, int32_t seat, int32_t *take)
{
    *take = 0;
    if (!VQ_SPAN(a.parents + seat, 1, a.parents, a.seats)) return -1;
    const int32_t p = a.parents[seat];
    if (p < 0 || p >= a.seats) return -1;
    int32_t k = fork_held(a, p);
    if (a.keep && VQ_SPAN(a.keep + seat, 1, a.keep, a.seats)) {
        const int32_t most = a.keep[seat] > 0 ? a.keep[seat] : 0;
        if (k > most) k = most;
    }
    *take = k;
    return p;
}

__device__ __forceinline__ int32_t fork_blocks(const ForkArgs &a, int32_t tokens)
{
    return (int32_t)(((int64_t)tokens + ((int64_t)1 << a.page_shift) - 1) >> a.page_shift);
}

__device__ __forceinline__ bool fork_page(const ForkArgs &a, int32_t pg) { return pg >= 0 && pg < a.num_pages; }

// The flags of all pages, 16 at a time (they are padded to that).
__global__ void __launch_bounds__(kForkThreads) fork_clear(const __grid_constant__ ForkArgs a)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int64_t tiles = ((int64_t)a.num_pages + 15) / 16, threads = (int64_t)gridDim.x * kForkThreads;
    for (int64_t t = (int64_t)blockIdx.x * kForkThreads + threadIdx.x; t < tiles; t += threads) {
        if (VQ_VSPAN(a.before + 16 * t, 16, a.before, 16 * tiles, 16)) reinterpret_cast<uint4 *>(a.before)[t] = make_uint4(0, 0, 0, 0);
        if (VQ_VSPAN(a.whole + 16 * t, 16, a.whole, 16 * tiles, 16)) reinterpret_cast<uint4 *>(a.whole)[t] = make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (VQ_VSPAN(a.first + 16 * t + 4 * k, 4, a.first, 16 * tiles, 16))
                reinterpret_cast<int4 *>(a.first)[4 * t + k] = make_int4(kNoSeat, kNoSeat, kNoSeat, kNoSeat);
    }
}

// Flags of the old rows, the new rows and their flags: a warp takes a seat and kForkSegment
// entries at a time.
__global__ void __launch_bounds__(kForkThreads) fork_mark(const __grid_constant__ ForkArgs a)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t me = (int64_t)blockIdx.x * (kForkThreads / 32) + (threadIdx.x >> 5), warps = (int64_t)gridDim.x * (kForkThreads / 32);
    const int lane = threadIdx.x & 31;
    const int32_t per = (a.max_blocks + kForkSegment - 1) / kForkSegment;
    const int64_t entries = (int64_t)a.seats * a.max_blocks;
    const int64_t all = (int64_t)a.seats * per;
    for (int64_t i = me; i < all; i += warps) {
        const int32_t seat = (int32_t)(i / per);
        const int32_t b0 = (int32_t)(i - (int64_t)seat * per) * kForkSegment + lane;
        const int32_t old = fork_blocks(a, fork_held(a, seat));
        int32_t take;
        const int32_t parent = fork_parent(a, seat, &take);
        const int32_t upto = fork_blocks(a, take), whole = take >> a.page_shift;
        const int32_t *from = a.table + (int64_t)seat * a.max_blocks;
        const int32_t *src = a.table + (int64_t)(parent < 0 ? 0 : parent) * a.max_blocks;
        int32_t *dst = a.table_out + (int64_t)seat * a.max_blocks;
        int32_t was[kForkSegment / 32], is[kForkSegment / 32];
#pragma unroll
        for (int k = 0; k < kForkSegment / 32; ++k) {
            const int32_t b = b0 + k * 32;
            was[k] = b < old && VQ_SPAN(from + b, 1, a.table, entries) ? __ldg(from + b) : -1;
            is[k] = b < upto && VQ_SPAN(src + b, 1, a.table, entries) ? __ldg(src + b) : -1;
        }
#pragma unroll
        for (int k = 0; k < kForkSegment / 32; ++k) {
            const int32_t b = b0 + k * 32;
            if (fork_page(a, was[k]) && VQ_SPAN(a.before + was[k], 1, a.before, a.num_pages)) a.before[was[k]] = 1;
            if (fork_page(a, is[k])) {
                if (b < whole) {
                    if (VQ_SPAN(a.whole + is[k], 1, a.whole, a.num_pages)) a.whole[is[k]] = 1;
                } else if (VQ_SPAN(a.first + is[k], 1, a.first, a.num_pages)) {
                    atomicMin(a.first + is[k], seat);  // the same whatever the order
                }
            }
            if (b < a.max_blocks && VQ_SPAN(dst + b, 1, a.table_out, entries)) dst[b] = is[k];
        }
    }
}

// Launch: one cluster, kPageThreads threads, dynamic shared memory
// fork_finish_smem(seats).
__host__ __device__ inline size_t fork_finish_smem(int64_t seats) { return 64 * 8 + 16 * 8 + (size_t)seats * 4; }

__global__ void __launch_bounds__(kPageThreads) fork_finish(const __grid_constant__ ForkArgs a)
{
    extern __shared__ __align__(16) unsigned char share_smem[];
    int64_t *scratch = reinterpret_cast<int64_t *>(share_smem);
    int64_t *mine = scratch + 64;                             // pages freed in this block's range
    int32_t *take = reinterpret_cast<int32_t *>(scratch + 80);  // [seats]
    auto cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x, rank = blockIdx.x, blocks = gridDim.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int32_t fc = *a.free_count;
    const int64_t avail = fc < 0 ? 0 : fc > a.num_pages ? a.num_pages : fc;
    // this block's pages, 16 to a thread and pass
    const int64_t tiles = ((int64_t)a.num_pages + 15) / 16;
    const int64_t t0 = tiles * rank / blocks, t1 = tiles * (rank + 1) / blocks;
    // bit i: page 16 t + i goes back
    auto freed_of = [&](int64_t t) -> uint32_t {
        if (!VQ_VSPAN(a.before + 16 * t, 16, a.before, (a.num_pages + 15) / 16 * 16, 16) ||
            !VQ_VSPAN(a.whole + 16 * t, 16, a.whole, (a.num_pages + 15) / 16 * 16, 16))
            return 0;
        const uint4 b = __ldcg(reinterpret_cast<const uint4 *>(a.before) + t);
        const uint4 w = __ldcg(reinterpret_cast<const uint4 *>(a.whole) + t);
        const uint32_t c[4] = {b.x & ~w.x, b.y & ~w.y, b.z & ~w.z, b.w & ~w.w};
        uint32_t bits = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i) bits |= (c[k] >> (8 * i) & 1u) << (4 * k + i);
        if (t == tiles - 1 && a.num_pages % 16) bits &= (1u << (a.num_pages % 16)) - 1u;  // the flags' padding
        for (uint32_t left = bits; left; left &= left - 1) {
            const int i = __ffs((int)left) - 1;
            if (VQ_SPAN(a.first + 16 * t + i, 1, a.first, a.num_pages) && __ldcg(a.first + 16 * t + i) != kNoSeat)
                bits &= ~(1u << i);
        }
        return bits;
    };
    int64_t n = 0, unused = 0;
    for (int64_t t = t0 + tid; t < t1; t += kPageThreads) n += __popc(freed_of(t));
    block_scan2(n, unused, scratch);
    if (tid == 0) mine[0] = scratch[31];
    cluster.sync();
    int64_t before = 0, freed = 0;
    for (int b = 0; b < blocks; ++b) {
        const int64_t c = *cluster.map_shared_rank(mine, b);
        if (b < rank) before += c;
        freed += c;
    }
    for (int64_t base = t0; base < t1; base += kPageThreads) {
        const int64_t t = base + tid;
        const uint32_t bits = t < t1 ? freed_of(t) : 0;
        int64_t s = __popc(bits);
        const int64_t own = s;
        block_scan2(s, unused, scratch);
        int64_t at = avail + before + s - own;
        for (uint32_t left = bits; left; left &= left - 1) {
            // (a list that would overflow, more pages held than the pool has, drops the rest)
            if (at < a.num_pages && VQ_SPAN(a.free_pages + at, 1, a.free_pages, a.num_pages))
                a.free_pages[at] = (int32_t)(16 * t) + __ffs((int)left) - 1;
            ++at;
        }
        before += scratch[31];
        __syncthreads();  // before the next pass writes scratch
    }
    cluster.sync();  // the list is written, every block's count read
    if (rank != 0) return;
    const int64_t have = avail + freed < a.num_pages ? avail + freed : a.num_pages;
    int64_t base_copies = 0;
    for (int base = 0; base < a.seats; base += kPageThreads) {
        const int seat = base + tid;
        int32_t k = 0, tail = -1;
        int64_t copy = 0;
        if (seat < a.seats) {
            (void)fork_parent(a, seat, &k);
            if (k & ((1 << a.page_shift) - 1)) {
                const int32_t *e = a.table_out + (int64_t)seat * a.max_blocks + (k >> a.page_shift);
                if (VQ_SPAN(e, 1, a.table_out, (int64_t)a.seats * a.max_blocks)) tail = __ldcg(e);
                if (fork_page(a, tail) && VQ_SPAN(a.whole + tail, 1, a.whole, a.num_pages) &&
                    VQ_SPAN(a.first + tail, 1, a.first, a.num_pages))
                    copy = __ldcg(a.whole + tail) || __ldcg(a.first + tail) < seat;
            }
        }
        int64_t s = copy;
        block_scan2(s, unused, scratch);
        if (seat < a.seats) {
            int32_t to = -1;
            if (copy) {
                int32_t *e = a.table_out + (int64_t)seat * a.max_blocks + (k >> a.page_shift);
                const int64_t at = have - (base_copies + s);
                if (at >= 0 && VQ_SPAN(a.free_pages + at, 1, a.free_pages, a.num_pages)) to = __ldcg(a.free_pages + at);
                if (!fork_page(a, to)) {  // no page for it (or an entry of the list that is none)
                    to = -1;
                    k = k >> a.page_shift << a.page_shift;
                }
                if (VQ_SPAN(e, 1, a.table_out, (int64_t)a.seats * a.max_blocks)) *e = to;
            }
            int32_t *pair = a.copies + 2 * (int64_t)seat;
            if (VQ_SPAN(pair, 2, a.copies, 2 * (int64_t)a.seats)) {
                pair[0] = to >= 0 ? tail : -1;
                pair[1] = to;
            }
            take[seat] = k;
        }
        base_copies += scratch[31];
        __syncthreads();
    }
    // (lens_out may be lens, which the loop above reads for every seat's parent)
    for (int seat = tid; seat < a.seats; seat += kPageThreads)
        if (VQ_SPAN(a.lens_out + seat, 1, a.lens_out, a.seats)) a.lens_out[seat] = take[seat];
    if (tid == 0) *a.free_count_out = (int32_t)(have - (base_copies < have ? base_copies : have));
}

// ------------------------------------------------------------------ compact

struct CompactArgs {
    const int32_t *lens, *table;
    int32_t *table_out;
    const int32_t *free_pages, *free_count;
    int32_t *free_out, *free_count_out;
    int32_t *moves;  // [num_pages / 2][2]
    int32_t *map;    // [num_pages]
    uint32_t *idle;  // a bit a page: on the free list
    int32_t requests, max_blocks, page_shift, num_pages;
};

// Launch: one cluster, kPageThreads threads, static shared memory only.
__global__ void __launch_bounds__(kPageThreads) compact_plan(const __grid_constant__ CompactArgs a)
{
    __shared__ int64_t scratch[64];
    __shared__ int64_t mine[2];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    auto cluster = cooperative_groups::this_cluster();
    const int tid = threadIdx.x, rank = blockIdx.x, blocks = gridDim.x;
    const int64_t P = a.num_pages, all = (int64_t)blocks * kPageThreads, me = (int64_t)rank * kPageThreads + tid;
    const int64_t words = (P + 31) / 32;
    const int32_t fc = *a.free_count;
    const int64_t avail = fc < 0 ? 0 : fc > P ? P : fc;
    for (int64_t w = me; w < words; w += all)
        if (VQ_SPAN(a.idle + w, 1, a.idle, words)) a.idle[w] = 0;
    cluster.sync();
    for (int64_t i = me; i < avail; i += all) {
        if (!VQ_SPAN(a.free_pages + i, 1, a.free_pages, P)) continue;
        const int32_t p = a.free_pages[i];
        if (p >= 0 && p < P && VQ_SPAN(a.idle + (p >> 5), 1, a.idle, words)) atomicOr(a.idle + (p >> 5), 1u << (p & 31));
    }
    cluster.sync();
    // this block's words, one to a thread and pass
    const int64_t w0 = words * rank / blocks, w1 = words * (rank + 1) / blocks;
    auto held_of = [&](int64_t w) -> uint32_t {  // bit i: page 32 w + i is held
        if (!VQ_SPAN(a.idle + w, 1, a.idle, words)) return 0;
        const uint32_t bits = ~__ldcg(a.idle + w);
        return w == words - 1 && P % 32 ? bits & ((1u << (P % 32)) - 1u) : bits;
    };
    int64_t held = 0, unused = 0;
    for (int64_t w = w0 + tid; w < w1; w += kPageThreads) held += __popc(held_of(w));
    block_scan2(held, unused, scratch);
    if (tid == 0) mine[0] = scratch[31];
    cluster.sync();
    int64_t used = 0, held_before = 0;
    for (int b = 0; b < blocks; ++b) {
        const int64_t c = *cluster.map_shared_rank(mine, b);
        if (b < rank) held_before += c;
        used += c;
    }
    // Page p has h held pages before it.  A hole below `used` is number p - h; a held page
    // at or past it is number h - (held pages below `used`), and there are as many holes as
    // such pages.
    int64_t below = 0;  // held pages below `used`, of this block
    for (int64_t w = w0 + tid; w < w1; w += kPageThreads) {
        const int64_t left = used - 32 * w;
        if (left > 0) below += __popc(held_of(w) & (left < 32 ? (1u << left) - 1u : 0xffffffffu));
    }
    __syncthreads();  // scratch is read
    block_scan2(below, unused, scratch);
    if (tid == 0) mine[1] = scratch[31];
    cluster.sync();
    int64_t kept = 0;  // held pages below `used`
    for (int b = 0; b < blocks; ++b) kept += *cluster.map_shared_rank(mine + 1, b);
    const int64_t moving = used - kept;
    const int64_t rows = P / 2;
    const int lane = tid & 31;
    for (int64_t base = w0; base < w1; base += kPageThreads) {
        const uint32_t bits = base + tid < w1 ? held_of(base + tid) : 0;
        int64_t s = __popc(bits);
        const int64_t own = s;
        __syncthreads();  // scratch is read
        block_scan2(s, unused, scratch);
        // the pages of the warp's words, a word at a time: a lane a page
        const int64_t h0 = held_before + s - own;
        for (int k = 0; k < 32; ++k) {
            const int64_t w = base + (tid & ~31) + k;
            if (w >= w1) break;  // warp-uniform
            const uint32_t word = __shfl_sync(0xffffffffu, bits, k);
            const int64_t h = __shfl_sync(0xffffffffu, h0, k) + __popc(word & ((1u << lane) - 1u));
            const int64_t p = 32 * w + lane;
            const bool is_held = word >> lane & 1u;
            if (p >= P) continue;
            if (is_held != (p >= used)) {  // it stays, or is free past the held ones
                if (VQ_SPAN(a.map + p, 1, a.map, P)) a.map[p] = is_held ? (int32_t)p : -1;
            } else {
                const int64_t nth = is_held ? h - kept : p - h;
                int32_t *m = a.moves + 2 * nth + (is_held ? 0 : 1);
                if (nth < rows && VQ_SPAN(m, 1, a.moves, 2 * rows)) *m = (int32_t)p;
                if (!is_held && VQ_SPAN(a.map + p, 1, a.map, P)) a.map[p] = -1;
            }
        }
        held_before += scratch[31];
    }
    for (int64_t i = moving + me; i < rows; i += all)
        if (VQ_SPAN(a.moves + 2 * i, 2, a.moves, 2 * rows)) {
            a.moves[2 * i] = -1;
            a.moves[2 * i + 1] = -1;
        }
    cluster.sync();  // the moves are written; the free list has been read long since
    for (int64_t i = me; i < moving; i += all) {
        if (!VQ_SPAN(a.moves + 2 * i, 2, a.moves, 2 * rows)) continue;
        const int32_t from = __ldcg(a.moves + 2 * i), to = __ldcg(a.moves + 2 * i + 1);
        if (VQ_SPAN(a.map + from, 1, a.map, P)) a.map[from] = to;
    }
    for (int64_t i = me; i < P; i += all)
        if (VQ_SPAN(a.free_out + i, 1, a.free_out, P)) a.free_out[i] = i < P - used ? (int32_t)(P - 1 - i) : -1;
    if (me == 0) *a.free_count_out = (int32_t)(P - used);
}

// The table through the map: entries of tokens a request holds.
__global__ void __launch_bounds__(kForkThreads) compact_table(const __grid_constant__ CompactArgs a)
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t entries = (int64_t)a.requests * a.max_blocks, stride = (int64_t)gridDim.x * kForkThreads;
    for (int64_t i = (int64_t)blockIdx.x * kForkThreads + threadIdx.x; i < entries; i += stride) {
        const int32_t r = entries <= 0x7fffffff ? (int32_t)i / a.max_blocks : (int32_t)(i / a.max_blocks);
        if (!VQ_SPAN(a.table + i, 1, a.table, entries) || !VQ_SPAN(a.lens + r, 1, a.lens, a.requests)) continue;
        int32_t pg = a.table[i];
        const int64_t b = i - (int64_t)r * a.max_blocks;
        if (b << a.page_shift < __ldg(a.lens + r) && pg >= 0 && pg < a.num_pages &&
            VQ_SPAN(a.map + pg, 1, a.map, a.num_pages))
            pg = __ldcg(a.map + pg);
        if (VQ_SPAN(a.table_out + i, 1, a.table_out, entries)) a.table_out[i] = pg;
    }
}

// ------------------------------------------------------------------ copy

constexpr int kCopyPools = 8;
constexpr int kCopyThreads = 256;
constexpr int kCopyPiece = 4096;   // bytes that a warp copies at a time
constexpr int kCopyWindow = 2048;  // pairs looked through at a time

struct CopyPool {
    unsigned char *base;
    int64_t page_stride, page_bytes, layer_stride;
    int32_t pieces;     // of a page
    int32_t first;      // pieces of a pair in the pools before
    int32_t layers;
    int32_t vec;        // width of the accesses: 16, 4 or 1
};

struct CopyArgs {
    const int32_t *pairs;
    int64_t n_pairs, num_pages;
    int32_t n_pools;
    int32_t total;  // pieces of a pair in all pools
    CopyPool pool[kCopyPools];
};

template <typename V, int N>
__device__ __forceinline__ void copy_piece(const unsigned char *from, unsigned char *to, int64_t bytes,
                                           const CopyPool &p, int64_t region)
{
    const int lane = threadIdx.x & 31;
    const int64_t n = bytes / (int64_t)sizeof(V);
    for (int64_t i0 = 0; i0 < n; i0 += 32 * N) {
        V v[N];
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t i = i0 + k * 32 + lane;
            if (i < n && span_ok(from + i * sizeof(V), sizeof(V), p.base, region, sizeof(V)))
                v[k] = __ldcs(reinterpret_cast<const V *>(from) + i);
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int64_t i = i0 + k * 32 + lane;
            if (i < n && span_ok(to + i * sizeof(V), sizeof(V), p.base, region, sizeof(V)))
                __stcs(reinterpret_cast<V *>(to) + i, v[k]);
        }
    }
}

// Every block goes through the list window by window: the window's pairs that name two
// pages are gathered in shared memory, in list order, and their pieces shared out over
// the warps of the grid.
__global__ void __launch_bounds__(kCopyThreads) copy_pages(const __grid_constant__ CopyArgs a)
{
    __shared__ int2 live[kCopyWindow];
    __shared__ int32_t counts[kCopyThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = kCopyWindow / kCopyThreads;
    const int64_t warps = (int64_t)gridDim.x * (kCopyThreads / 32);
    int64_t turn = (int64_t)blockIdx.x * (kCopyThreads / 32) + warp;  // this warp's next piece, of the window
    for (int64_t w0 = 0; w0 < a.n_pairs; w0 += kCopyWindow) {
        int2 pair[kPer];
        uint32_t has = 0;
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const int64_t i = w0 + warp * (32 * kPer) + k * 32 + lane;
            pair[k] = make_int2(-1, -1);
            if (i < a.n_pairs && VQ_SPAN(a.pairs + 2 * i, 2, a.pairs, 2 * a.n_pairs))
                pair[k] = make_int2(__ldg(a.pairs + 2 * i), __ldg(a.pairs + 2 * i + 1));
            if (pair[k].x >= 0 && pair[k].x < a.num_pages && pair[k].y >= 0 && pair[k].y < a.num_pages &&
                pair[k].x != pair[k].y)
                has |= 1u << k;
        }
        int n = 0, at[kPer];
#pragma unroll
        for (int k = 0; k < kPer; ++k) {
            const uint32_t all = __ballot_sync(0xffffffffu, has >> k & 1u);
            at[k] = n + __popc(all & ((1u << lane) - 1u));
            n += __popc(all);
        }
        __syncthreads();  // the last window's pairs are read
        if (lane == 0) counts[warp] = n;
        __syncthreads();
        int before = 0, total = 0;
#pragma unroll
        for (int k = 0; k < kCopyThreads / 32; ++k) {
            before += k < warp ? counts[k] : 0;
            total += counts[k];
        }
#pragma unroll
        for (int k = 0; k < kPer; ++k)
            if (has >> k & 1u) live[before + at[k]] = pair[k];
        __syncthreads();
        const int64_t pieces = (int64_t)total * a.total;
        for (; turn < pieces; turn += warps) {
            const int32_t j = (int32_t)(turn / a.total);
            int32_t c = (int32_t)(turn - (int64_t)j * a.total);
            int k = 0;
            while (k + 1 < a.n_pools && c >= a.pool[k + 1].first) ++k;
            const CopyPool &p = a.pool[k];
            c -= p.first;
            const int32_t layer = c / p.pieces;
            const int64_t off = (int64_t)(c - layer * p.pieces) * kCopyPiece;
            const int64_t bytes = p.page_bytes - off < kCopyPiece ? p.page_bytes - off : kCopyPiece;
            const unsigned char *from = p.base + layer * p.layer_stride + live[j].x * p.page_stride + off;
            unsigned char *to = p.base + layer * p.layer_stride + live[j].y * p.page_stride + off;
            const int64_t region = (p.layers - 1) * p.layer_stride + (a.num_pages - 1) * p.page_stride + p.page_bytes;
            if (p.vec == 16) copy_piece<uint4, 8>(from, to, bytes, p, region);
            else if (p.vec == 4) copy_piece<uint32_t, 8>(from, to, bytes, p, region);
            else copy_piece<unsigned char, 4>(from, to, bytes, p, region);
        }
        turn -= pieces;  // the next window goes on with the warp whose turn it is
    }
}

}  // namespace vqk
