// vq_pattn.cuh -- attention of new tokens over a paged cache of product-VQ
// codes: the work split that all its kernels share, the general kernel, and
// the merge of partial results.
//
// For token i of request r (L_r tokens in the cache, its n_r new ones among
// them) at position p = L_r - n_r + i and query head h of KV head c:
//   s[t]  = kappa q . K^[t],  t in [max(0, p - window + 1), p],  kappa = scale log2 e
//   out   = sum_t 2^(s[t] - m) V^[t] / sum_t 2^(s[t] - m),       m = max_t s[t]
//   lse   = ln 2 (m + log2 sum_t 2^(s[t] - m))
// K^[t], V^[t] are the codebook rows that token t's codes select (a code
// >= n_centroids selects a zero row).  A token whose page entry is outside
// [0, num_pages) is not seen.  A row that sees nothing gets zeros and -inf.
//
// The work split.  An item is a run of up to tile_tokens new tokens of one
// request against one group of up to gc query heads of one KV head; its work
// is counted in units of kUnit cached tokens, at least one (so that rows that
// see nothing are written too).  Lengths live on the device, so the host
// knows only a bound on the items; each block lays the items out for itself:
// item j belongs to the last request r with start(r) = cu[r] / tile_tokens + r
// <= j, which needs no sum over the requests before it and leaves at most one
// hole per request.  The rows after the last request (a padded batch) form one
// more request that sees nothing.  The units of all items of all head groups
// are one line of U units, head groups outermost so that a block changes its
// codebooks seldom, and block b of N takes units [b U / N, (b + 1) U / N): every
// block has the same work to within one unit, however uneven the requests
// are.  An item that lies in one block is finished there; the blocks of a
// split item write (m, sum, sum of weighted rows) to the workspace, two slots
// a block (2b: the item it continues, 2b + 1: the item it begins and does not
// finish), and the block that begins it leaves a note for the merge.  The
// order of every sum is fixed by the lengths.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "vq_check.cuh"
#include "vq_kernels.cuh"

namespace vqk {

constexpr int kUnit = 128;       // cached tokens of one unit of work
constexpr int kStageCu = 512;    // requests + 2 up to which a block keeps cu and lens in shared memory (64 in the chunk kernel)

// The note of a split item (rows = 0: none).
struct PagedNote {
    int64_t tok0;    // first token (row of q)
    int32_t head0;   // first query head
    int32_t gc;      // heads of the item: row i is token tok0 + i / gc, head head0 + i % gc
    int32_t rows;
    int32_t first;   // blocks that hold its parts: slots 2 first + 1, 2 (first + 1), .., 2 last
    int32_t last;
    int32_t pad;
};

struct PagedArgs {
    const void *q;
    const uint8_t *k_codes, *v_codes;
    const void *kcb, *vcb;
    void *out;
    float *lse;            // or null
    const int32_t *cu, *lens, *table;
    const int64_t *slots;  // [tokens] or null: a request whose first new token has none is refused
    int64_t tokens;        // rows of q
    int64_t q_stride;      // elements between tokens of q
    int64_t page_stride;   // bytes between pages of codes
    int64_t num_pages;
    int64_t items;         // bound on the items of one head group
    int32_t requests, max_blocks, page_shift;
    int32_t hq, hkv, group;
    int32_t gc, gch;       // heads per item, head groups per KV head
    int32_t dim, sub, ns, nc;
    int32_t window;        // 0: none
    int32_t tile_tokens;
    int32_t item_cost;     // units that an item's set-up and write are worth
    int32_t no_split;      // every item costs 1 and stays in one block (no merge follows)
    int32_t cls, cls_tokens;  // 0: every request; 1: those of up to cls_tokens new tokens; 2: the others
    float kappa;
    float *part;           // [2 N][tile rows][dim] weighted sums
    float *ml;             // [2 N][tile rows][2] maximum, sum of weights
    PagedNote *notes;      // [N]
    int32_t tile_rows;
    // a cache of 4-bit scalar codes (sub = 2, kcb and vcb unused): codes come in pairs, low
    // half first, and stand for scale x centroid, the centroids in the rows' type
    const void *k_scales, *v_scales;  // page p at p * scale_stride, [heads][page_size], in the rows' type
    const float *k_cent, *v_cent;     // [nc]
    int64_t scale_stride;             // elements between pages of scales
};

struct PagedItem {
    int64_t tok0;   // first row of q
    int32_t ntok;
    int32_t pos0;   // position of the first token
    int32_t k_lo;   // first cached token seen by any of its rows, rounded down to a unit
    int32_t k_hi;   // one past the last
    int32_t units;  // 0: a hole
};

// Lengths as the kernel sees them: cu clamped into [0, tokens], request
// number `requests` being the rows after the last.  Rows are below 2^31, and so
// are items.  A refused request holds nothing, so that its rows see nothing.
struct PagedLens {
    const int32_t *cu, *lens;
    const int32_t *starts;  // start(0 .. requests), or null: computed
    int32_t requests, tile;
    int64_t tokens;
    // (where starts are staged, so are lengths: those of refused requests are 0 there)
    __host__ __device__ __forceinline__ int32_t length(int r, const int64_t *slots) const
    {
        if (slots && !starts) {
            const int64_t at = first(r);
            if (at < tokens && slots[at] < 0) return 0;
        }
        return lens[r] > 0 ? lens[r] : 0;
    }
    __host__ __device__ __forceinline__ int64_t first(int r) const
    {
        if (r > requests) return tokens;
        const int64_t c = cu[r];
        return c < 0 ? 0 : c > tokens ? tokens : c;
    }
    __host__ __device__ __forceinline__ int64_t compute_start(int r) const
    {
        return (int64_t)((uint32_t)first(r) / (uint32_t)tile) + r;
    }
    __host__ __device__ __forceinline__ int64_t start(int r) const { return starts ? starts[r] : compute_start(r); }
    // the last r in [0, requests] with start(r) <= j
    __host__ __device__ __forceinline__ int find(int64_t j) const
    {
        int lo = 0, hi = requests;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (start(mid) <= j) lo = mid;
            else hi = mid - 1;
        }
        return lo;
    }
};

// b * all / n for 0 <= b <= n, in 32 bits where they do.
__host__ __device__ __forceinline__ int64_t part_of(int64_t b, int64_t all, int64_t n)
{
    if (all * n <= 0xffffffffll) return (uint32_t)(b * all) / (uint32_t)n;
    return b * all / n;
}

// Item j, which belongs to request r; units = 0 for a hole (then *skip is the
// next item worth a look).
__host__ __device__ __forceinline__ PagedItem paged_item(const PagedArgs &a, const PagedLens &l, int64_t j, int r,
                                                int64_t *skip)
{
    PagedItem it{};
    *skip = j + 1;
    const int64_t c0 = l.first(r), c1 = l.first(r + 1);
    const int64_t n = c1 > c0 ? c1 - c0 : 0;
    const int64_t i0 = (j - l.start(r)) * l.tile;
    const bool mine = a.cls == 0 || (a.cls == 1) == (n <= a.cls_tokens);
    if (!mine || i0 >= n || i0 < 0) {
        const int64_t next = r < a.requests ? l.start(r + 1) : a.items;
        if (next > j + 1) *skip = next;
        return it;
    }
    const int64_t len = r < a.requests ? l.length(r, a.slots) : 0;
    const int64_t cap = (int64_t)a.max_blocks << a.page_shift;
    const int64_t i1 = i0 + l.tile < n ? i0 + l.tile : n;
    const int64_t pos0 = len - n + i0;
    int64_t hi = len - n + i1;
    if (hi > cap) hi = cap;
    if (r >= a.requests || hi < 0) hi = 0;
    int64_t lo = a.window > 0 ? pos0 - a.window + 1 : 0;
    if (lo < 0) lo = 0;
    lo &= ~(int64_t)(kUnit - 1);
    it.tok0 = c0 + i0;
    it.ntok = (int32_t)(i1 - i0);
    it.pos0 = (int32_t)pos0;
    it.k_lo = (int32_t)lo;
    it.k_hi = (int32_t)hi;
    it.units = hi > lo ? (int32_t)((hi - lo + kUnit - 1) / kUnit) : 1;
    return it;
}

// What an item costs (0: a hole).
__host__ __device__ __forceinline__ int32_t paged_cost(const PagedArgs &a, int32_t units)
{
    return units == 0 ? 0 : a.no_split ? 1 : units + a.item_cost;
}

// The items that one of `threads` threads lays out.
struct PagedRun {
    int64_t j0, j1;
    __host__ __device__ __forceinline__ PagedRun(const PagedArgs &a, int tid, int threads)
    {
        const int64_t per = (a.items + threads - 1) / threads;
        j0 = tid * per;
        j1 = j0 + per < a.items ? j0 + per : a.items;
    }
    // their cost; *r0: the first one's request
    __host__ __device__ __forceinline__ int64_t cost(const PagedArgs &a, const PagedLens &l, int *r0) const
    {
        int64_t sum = 0;
        if (j0 < j1) {
            *r0 = l.find(j0);
            int r = *r0;
            for (int64_t j = j0; j < j1;) {
                while (r < a.requests && l.start(r + 1) <= j) ++r;
                int64_t skip;
                sum += paged_cost(a, paged_item(a, l, j, r, &skip).units);
                j = skip;
            }
        }
        return sum;
    }
    // the item at `left` of that cost, and where in its cost
    __host__ __device__ __forceinline__ bool locate(const PagedArgs &a, const PagedLens &l, int r, int64_t left,
                                                    int64_t *item, int32_t *request, int32_t *at) const
    {
        for (int64_t j = j0; j < j1;) {
            while (r < a.requests && l.start(r + 1) <= j) ++r;
            int64_t skip;
            const int32_t u = paged_cost(a, paged_item(a, l, j, r, &skip).units);
            if (left < u) {
                *item = j;
                *request = r;
                *at = (int32_t)left;
                return true;
            }
            left -= u;
            j = skip;
        }
        return false;
    }
};

// Where a block stands on the line of costs.
template <int STAGE>
struct PagedStage {
    int32_t cu[STAGE], lens[STAGE], start[STAGE];
};
template <int STAGE = kStageCu, int SCRATCH = 33>
struct PagedWalk {
    PagedStage<STAGE> stage;
    int64_t scratch[SCRATCH];  // of the plan alone
    int64_t total;  // the costs of one head group
    int64_t u0, u1; // this block's part of the line
    int32_t blocks; // blocks with work
    int32_t hx;     // head group
    int64_t j;      // item
    int32_t r;
    int32_t at;     // where in its cost
};

// The lengths as a block reads them: from its stage if they fit there.
template <int STAGE, int SCRATCH>
__device__ __forceinline__ PagedLens paged_lens(const PagedArgs &a, const PagedWalk<STAGE, SCRATCH> &w)
{
    PagedLens l{a.cu, a.lens, nullptr, a.requests, a.tile_tokens, a.tokens};
    if (a.requests + 2 <= STAGE) {
        l.cu = w.stage.cu;
        l.lens = w.stage.lens;
        l.starts = w.stage.start;
    }
    return l;
}

// Lay the items out and find this block's part (all THREADS threads; w in
// shared memory).  Returns whether the block has any.
template <int THREADS, int STAGE, int SCRATCH>
__device__ __forceinline__ bool paged_plan(const PagedArgs &a, PagedWalk<STAGE, SCRATCH> &w, PagedLens &l)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.requests + 2 <= STAGE) {
        const PagedLens from{a.cu, a.lens, nullptr, a.requests, a.tile_tokens, a.tokens};
        for (int i = tid; i <= a.requests; i += THREADS) {
            w.stage.cu[i] = a.cu[i];
            w.stage.start[i] = (int32_t)from.compute_start(i);
            if (i < a.requests) w.stage.lens[i] = from.length(i, a.slots);
        }
        __syncthreads();
    }
    l = paged_lens(a, w);
    const PagedRun run(a, tid, THREADS);
    int r0 = 0;
    const int64_t mine = run.cost(a, l, &r0);
    int64_t s = mine;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int64_t p = __shfl_up_sync(0xffffffffu, s, off);
        if (lane >= off) s += p;
    }
    if (lane == 31) w.scratch[warp] = s;
    __syncthreads();
    int64_t before = s - mine, total = 0;
    for (int k = 0; k < THREADS / 32; ++k) {
        if (k < warp) before += w.scratch[k];
        total += w.scratch[k];
    }
    const int64_t all = total * ((int64_t)a.hkv * a.gch);
    const int64_t n = all < (int64_t)gridDim.x ? all : (int64_t)gridDim.x;
    const int64_t b = blockIdx.x;
    if (tid == 0) {
        w.total = total;
        w.blocks = (int32_t)n;
        w.u0 = b < n ? part_of(b, all, n) : 0;
        w.u1 = b < n ? part_of(b + 1, all, n) : 0;
        w.hx = 0;
        w.j = w.r = w.at = 0;
    }
    if (b >= n) return false;  // block-uniform
    const int64_t u0 = part_of(b, all, n);
    const int64_t hx = total <= 0xffffffffll && u0 <= 0xffffffffll ? (uint32_t)u0 / (uint32_t)total : u0 / total;
    const int64_t rem = u0 - hx * total;
    __syncthreads();
    if (mine > 0 && before <= rem && rem < before + mine) {
        int64_t j;
        int32_t r, at;
        if (run.locate(a, l, r0, rem - before, &j, &r, &at)) {
            w.hx = (int32_t)hx;
            w.j = j;
            w.r = r;
            w.at = at;
        }
    }
    __syncthreads();
    return true;
}

// One block's part of one item.
struct PagedSegment {
    PagedItem it;
    int32_t hx;          // head group
    int32_t begin, end;  // units of the item
    bool whole;          // all of them
    int64_t slot;        // of the workspace, if not
};

// Walks this block's segments in order; every thread holds its own copy and
// computes the same.
struct PagedCursor {
    int64_t u, u1, j;
    int32_t r, at, hx, block;
    template <typename W>
    __host__ __device__ __forceinline__ void init(const W &w, int32_t b)
    {
        block = b;
        u = w.u0;
        u1 = w.u1;
        j = w.j;
        r = w.r;
        at = w.at;
        hx = w.hx;
    }
    // The next segment; false at the end.  `note` is filled if the block
    // begins an item that it does not finish.
    template <typename W>
    __host__ __device__ __forceinline__ bool next(const PagedArgs &a, const W &w, const PagedLens &l, PagedSegment &s,
                                         PagedNote &note)
    {
        for (;;) {
            if (u >= u1) return false;
            for (;;) {
                if (j >= a.items) {  // the next head group
                    j = 0;
                    r = 0;
                    if (++hx >= a.hkv * a.gch) {
                        // only if cu descends, so that the walk finds less than the
                        // plan: nothing more to do
                        u = u1;
                        return false;
                    }
                }
                while (r < a.requests && l.start(r + 1) <= j) ++r;
                int64_t skip;
                s.it = paged_item(a, l, j, r, &skip);
                if (s.it.units > 0) break;
                j = skip;
            }
            // from `at` on in the item's cost: set-up first, then its units
            const int64_t cost = paged_cost(a, s.it.units);
            if (a.no_split) {
                s.begin = 0;
                s.end = s.it.units;
                s.whole = true;
                s.hx = hx;
                s.slot = 0;
                ++u;
                ++j;
                return true;
            }
            const int64_t to = cost - at <= u1 - u ? cost : at + (u1 - u);
            s.begin = at > a.item_cost ? at - a.item_cost : 0;
            s.end = to > a.item_cost ? (int32_t)(to - a.item_cost) : 0;
            const int64_t u_item = u - at;  // where the item starts on the line
            u += to - at;
            at = 0;
            ++j;
            if (s.end == 0) continue;  // only set-up: the next block begins the item
            s.hx = hx;
            s.whole = s.begin == 0 && s.end == s.it.units;
            s.slot = 2 * (int64_t)block + (s.begin == 0 ? 1 : 0);
            if (s.begin == 0 && !s.whole) {
                const int64_t all = w.total * ((int64_t)a.hkv * a.gch);
                const int64_t last = u_item + cost;  // one past its last unit
                const int32_t g0 = hx % a.gch * a.gc;
                note.tok0 = s.it.tok0;
                note.head0 = hx / a.gch * a.group + g0;
                note.gc = a.group - g0 < a.gc ? a.group - g0 : a.gc;
                note.rows = s.it.ntok * note.gc;
                note.first = block;
                // the block of position x: the c with floor(c U / N) <= x < floor((c + 1) U / N);
                // past the last block only if cu descends, so that the walk finds more than
                // the plan: the workspace ends there
                const int64_t c = (last * w.blocks - 1) / all;
                note.last = (int32_t)(c < w.blocks ? c : w.blocks - 1);
            }
            return true;
        }
    }
};

template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }

constexpr float kLn2 = 0.69314718055994531f;

// A row's state is its maximum m and its sum of weights l: l = 0 if it has seen nothing,
// m = -inf and l = 1 if every score it has seen is -inf.  Beside a part with other
// scores such a part weighs nothing; a row of nothing else is 0 / 0, NaN as in the
// definition.  What its weighted sum is multiplied by, and its lse:
__device__ __forceinline__ float paged_inv(float m, float l)
{
    return l == 0.f ? 0.f : m == __int_as_float(0xff800000) ? __int_as_float(0x7fffffff) : 1.f / l;
}
__device__ __forceinline__ float paged_lse(float m, float l)
{
    if (l == 0.f) return __int_as_float(0xff800000);
    return m == __int_as_float(0xff800000) ? __int_as_float(0x7fffffff) : kLn2 * (m + log2f(l));
}

// Block table entry of cached token t, whatever it holds.
__device__ __forceinline__ int32_t paged_entry(const PagedArgs &a, int32_t r, int32_t t)
{
    const int32_t *e = a.table + (int64_t)r * a.max_blocks + (t >> a.page_shift);
    if (!VQ_SPAN(e, 1, a.table, (int64_t)a.requests * a.max_blocks)) return -1;
    return __ldg(e);
}

// Page of cached token t; -1 if the entry is no page.
__device__ __forceinline__ int64_t paged_page(const PagedArgs &a, int32_t r, int32_t t)
{
    const int32_t pg = paged_entry(a, r, t);
    return pg >= 0 && pg < a.num_pages ? pg : -1;
}

// ------------------------------------------------------------------ the general kernel
//
// Any type, head size up to kSimpleDim, sub-vector size and page size.  A
// block of kUnit threads takes one new token and up to kSimpleRows query heads
// of its KV head; a unit is one cached token per thread for the scores and one
// column (or more) per thread for the weighted sum, all in fp32.  What bounds
// it is the codebook rows, read through the L1 for every cached token, twice;
// it carries the types and shapes that the tensor kernels do not.

constexpr int kSimpleRows = 8;
constexpr int kSimpleDim = 512;

template <typename T>
__global__ void __launch_bounds__(kUnit) paged_attn_simple(const __grid_constant__ PagedArgs a)
{
    __shared__ PagedWalk<> w;
    __shared__ float sp[kSimpleRows][kUnit];
    __shared__ float red[kSimpleRows][kUnit / 32];
    __shared__ int64_t spage[kUnit];
    extern __shared__ float sq[];  // [kSimpleRows][dim]
    constexpr int kCols = kSimpleDim / kUnit;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const T *__restrict__ q = static_cast<const T *>(a.q);
    T *__restrict__ out = static_cast<T *>(a.out);
    const int64_t cb_elems = (int64_t)a.hkv * a.nc * a.sub;

    PagedLens l;
    PagedNote note{};
    if (paged_plan<kUnit>(a, w, l)) {
        PagedCursor cur;
        cur.init(w, (int32_t)blockIdx.x);
        PagedSegment s;
        while (cur.next(a, w, l, s, note)) {
            const int r = cur.r;
            const int h = s.hx / a.gch, g0 = s.hx % a.gch * a.gc;
            const int rows = a.group - g0 < a.gc ? a.group - g0 : a.gc;  // one token: a row per head
            const int head0 = h * a.group + g0;
            const int64_t tok = s.it.tok0;
            const int64_t code_head = (int64_t)h << a.page_shift;
            const T *__restrict__ kcb = static_cast<const T *>(a.kcb) + (int64_t)h * a.nc * a.sub;
            const T *__restrict__ vcb = static_cast<const T *>(a.vcb) + (int64_t)h * a.nc * a.sub;
            __syncthreads();
            for (int i = tid; i < kSimpleRows * a.dim; i += kUnit) {
                const int g = i / a.dim, d = i - g * a.dim;
                const T *src = q + tok * a.q_stride + (int64_t)(head0 + g) * a.dim + d;
                float v = 0.f;
                if (g < rows && VQ_SPAN(src, 1, q, (a.tokens - 1) * a.q_stride + (int64_t)a.hq * a.dim))
                    v = a.kappa * widen(*src);
                sq[i] = v;
            }
            float m[kSimpleRows], sum[kSimpleRows], acc[kSimpleRows][kCols];
#pragma unroll
            for (int g = 0; g < kSimpleRows; ++g) {
                m[g] = __int_as_float(0xff800000);
                sum[g] = 0.f;
#pragma unroll
                for (int c = 0; c < kCols; ++c) acc[g][c] = 0.f;
            }
            bool saw = false;
            for (int unit = s.begin; unit < s.end; ++unit) {
                const int32_t t = s.it.k_lo + unit * kUnit + tid;
                bool seen = t < s.it.k_hi && t <= s.it.pos0 && (a.window == 0 || (int64_t)t > (int64_t)s.it.pos0 - a.window);
                int64_t code_row = -1;
                if (seen) {
                    const int64_t pg = paged_page(a, r, t);
                    if (pg < 0) seen = false;
                    else code_row = pg * a.page_stride + (code_head + (t & ((1 << a.page_shift) - 1))) * a.ns;
                }
                saw |= seen;
                __syncthreads();  // sq is written; the last unit's sp and spage are read
                spage[tid] = code_row;
                float dot[kSimpleRows];
#pragma unroll
                for (int g = 0; g < kSimpleRows; ++g) dot[g] = 0.f;
                if (seen && span_ok(a.k_codes + code_row, a.ns, a.k_codes, (a.num_pages - 1) * a.page_stride + (((int64_t)a.hkv * a.ns) << a.page_shift), 1)) {
                    for (int sidx = 0; sidx < a.ns; ++sidx) {
                        const int code = __ldg(a.k_codes + code_row + sidx);
                        if (code >= a.nc) continue;
                        const T *row = kcb + (int64_t)code * a.sub;
                        if (!VQ_SPAN(row, a.sub, static_cast<const T *>(a.kcb), cb_elems)) continue;
                        for (int i = 0; i < a.sub; ++i) {
                            const float kv = widen(__ldg(row + i));
#pragma unroll
                            for (int g = 0; g < kSimpleRows; ++g)
                                dot[g] = fmaf(sq[g * a.dim + sidx * a.sub + i], kv, dot[g]);
                        }
                    }
                }
#pragma unroll
                for (int g = 0; g < kSimpleRows; ++g) {
                    if (!seen) dot[g] = __int_as_float(0xff800000);
                    float top = dot[g];
#pragma unroll
                    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
                    if (lane == 0) red[g][warp] = top;
                }
                __syncthreads();
                float scale[kSimpleRows];
#pragma unroll
                for (int g = 0; g < kSimpleRows; ++g) {
                    float top = m[g];
#pragma unroll
                    for (int k = 0; k < kUnit / 32; ++k) top = fmaxf(top, red[g][k]);
                    // nothing seen yet: keep the (empty) sums
                    scale[g] = m[g] == top ? 1.f : exp2f(m[g] - top);
                    m[g] = top;
                    // -inf weighs 0, whatever the maximum so far
                    const float p = dot[g] == __int_as_float(0xff800000) ? 0.f : exp2f(dot[g] - top);
                    sp[g][tid] = p;
                    sum[g] = sum[g] * scale[g] + p;
                }
                __syncthreads();
#pragma unroll
                for (int c = 0; c < kCols; ++c) {
                    const int d = tid + c * kUnit;
                    if (d >= a.dim) break;
                    const int sidx = d / a.sub, i = d - sidx * a.sub;
#pragma unroll
                    for (int g = 0; g < kSimpleRows; ++g) acc[g][c] *= scale[g];
                    for (int k = 0; k < kUnit; ++k) {
                        const int64_t cr = spage[k];
                        if (cr < 0) continue;  // not seen: whatever its page holds
                        if (!span_ok(a.v_codes + cr + sidx, 1, a.v_codes, (a.num_pages - 1) * a.page_stride + (((int64_t)a.hkv * a.ns) << a.page_shift), 1)) continue;
                        const int code = __ldg(a.v_codes + cr + sidx);
                        if (code >= a.nc) continue;
                        const T *e = vcb + (int64_t)code * a.sub + i;
                        if (!VQ_SPAN(e, 1, static_cast<const T *>(a.vcb), cb_elems)) continue;
                        const float v = widen(__ldg(e));
#pragma unroll
                        for (int g = 0; g < kSimpleRows; ++g) acc[g][c] = fmaf(sp[g][k], v, acc[g][c]);
                    }
                }
            }
            // the rows' sums of weights over the threads
#pragma unroll
            for (int g = 0; g < kSimpleRows; ++g) {
#pragma unroll
                for (int off = 16; off > 0; off >>= 1) sum[g] += __shfl_xor_sync(0xffffffffu, sum[g], off);
            }
            __syncthreads();
            if (lane == 0) {
#pragma unroll
                for (int g = 0; g < kSimpleRows; ++g) red[g][warp] = sum[g];
            }
            const bool any = __syncthreads_or(saw);
#pragma unroll
            for (int g = 0; g < kSimpleRows; ++g) {
                if (g >= rows) break;
                float total = 0.f;
#pragma unroll
                for (int k = 0; k < kUnit / 32; ++k) total += red[g][k];
                if (total == 0.f && any) total = 1.f;  // m = -inf: scores of -inf alone
                const int64_t orow = tok * a.hq + head0 + g;
                if (s.whole) {
                    const float inv = paged_inv(m[g], total);
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        const int d = tid + c * kUnit;
                        if (d < a.dim && VQ_SPAN(out + orow * a.dim + d, 1, out, a.tokens * a.hq * a.dim))
                            out[orow * a.dim + d] = narrow<T>(acc[g][c] * inv);
                    }
                    if (tid == 0 && a.lse && VQ_SPAN(a.lse + orow, 1, a.lse, a.tokens * a.hq))
                        a.lse[orow] = paged_lse(m[g], total);
                } else {
                    const int64_t prow = s.slot * a.tile_rows + g, prows = 2 * (int64_t)gridDim.x * a.tile_rows;
#pragma unroll
                    for (int c = 0; c < kCols; ++c) {
                        const int d = tid + c * kUnit;
                        if (d < a.dim && VQ_SPAN(a.part + prow * a.dim + d, 1, a.part, prows * a.dim))
                            a.part[prow * a.dim + d] = acc[g][c];
                    }
                    if (tid == 0 && VQ_SPAN(a.ml + prow * 2, 2, a.ml, prows * 2)) {
                        a.ml[prow * 2] = m[g];
                        a.ml[prow * 2 + 1] = total;
                    }
                }
            }
        }
    }
    if (tid == 0 && VQ_SPAN(a.notes + blockIdx.x, 1, a.notes, gridDim.x)) a.notes[blockIdx.x] = note;
}

// ------------------------------------------------------------------ the merge
//
// Block (b, y) merges rows [y kMergeRows, ..) of the item that block b of the
// attention began and did not finish: a warp per row, lanes over the parts for
// the maximum and the weights, then over the columns, several parts' loads in
// flight (one part after the other took 4 us for 7 parts of one token, all of it
// latency).  Reads every part once.

constexpr int kMergeThreads = 256;
constexpr int kMergeRows = kMergeThreads / 32;

// VEC: dim is a multiple of 4 (16-byte loads); LOADS: loads of a lane and part,
// dim <= 32 x LOADS x the columns of one.
template <typename T, bool VEC, int LOADS>
__global__ void __launch_bounds__(kMergeThreads)
    paged_attn_merge(const float *__restrict__ part, const float *__restrict__ ml,
                     const PagedNote *__restrict__ notes, int32_t tile_rows, int32_t dim, int32_t hq,
                     int64_t tokens, T *__restrict__ out, float *__restrict__ lse)
{
    constexpr int kW = VEC ? 4 : 1;                   // columns of a load
    constexpr int kMax = LOADS;
    constexpr int kBatch = 4;                         // parts in flight
    // launched while the attention's last blocks still run
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PagedNote n = notes[blockIdx.x];
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.y * kMergeRows + (threadIdx.x >> 5);
    if (row >= n.rows) return;  // warp-uniform
    const int parts = n.last - n.first + 1;
    auto slot_row = [&](int k) {
        return (k == 0 ? 2 * (int64_t)n.first + 1 : 2 * (int64_t)(n.first + k)) * tile_rows + row;
    };
    const int64_t prows = 2 * (int64_t)gridDim.x * tile_rows;
    auto state = [&](int k, float *m, float *l) {  // of part k; l = 0: it saw nothing, or there is none
        *m = __int_as_float(0xff800000);
        *l = 0.f;
        const float2 *p = reinterpret_cast<const float2 *>(ml) + slot_row(k);
        if (k < parts && VQ_SPAN(p, 1, reinterpret_cast<const float2 *>(ml), prows)) {
            *m = p->x;
            *l = p->y;
        }
    };
    float top = __int_as_float(0xff800000);
    for (int k = lane; k < parts; k += 32) {
        float m, l;
        state(k, &m, &l);
        if (l != 0.f) top = fmaxf(top, m);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    float total = 0.f, acc[kMax][kW];
#pragma unroll
    for (int c = 0; c < kMax; ++c)
#pragma unroll
        for (int i = 0; i < kW; ++i) acc[c][i] = 0.f;
    for (int k0 = 0; k0 < parts; k0 += 32) {
        float m, l;
        state(k0 + lane, &m, &l);
        const float w = l == 0.f ? 0.f : exp2f(m - top);  // a NaN sum is not 0: it goes on
        float t = w * l;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
        total += t;
        const int upto = parts - k0 < 32 ? parts - k0 : 32;
        for (int k = 0; k < upto; k += kBatch) {
            float f[kBatch], v[kBatch][kMax][kW];
#pragma unroll
            for (int x = 0; x < kBatch; ++x) {
                // (lanes past the parts hold 0)
                f[x] = __shfl_sync(0xffffffffu, w, (k + x) & 31);
                const bool live = k + x < upto && __shfl_sync(0xffffffffu, l, (k + x) & 31) != 0.f;
                const float *src = part + slot_row(k0 + k + x) * dim;
#pragma unroll
                for (int c = 0; c < kMax; ++c) {
                    const int col = (c * 32 + lane) * kW;
#pragma unroll
                    for (int i = 0; i < kW; ++i) v[x][c][i] = 0.f;
                    // a part that saw nothing has written zeros, one past the end nothing
                    if (live && col < dim && VQ_VSPAN(src + col, kW, part, prows * dim, 4 * kW)) {
                        if constexpr (VEC) {
                            const float4 q = __ldcg(reinterpret_cast<const float4 *>(src + col));
                            v[x][c][0] = q.x;
                            v[x][c][1] = q.y;
                            v[x][c][2] = q.z;
                            v[x][c][3] = q.w;
                        } else {
                            v[x][c][0] = __ldcg(src + col);
                        }
                    }
                }
            }
#pragma unroll
            for (int x = 0; x < kBatch; ++x)
#pragma unroll
                for (int c = 0; c < kMax; ++c)
#pragma unroll
                    for (int i = 0; i < kW; ++i) acc[c][i] = fmaf(f[x], v[x][c][i], acc[c][i]);
        }
    }
    const int64_t orow = (n.tok0 + row / n.gc) * hq + n.head0 + row % n.gc;
    const float inv = paged_inv(top, total);
#pragma unroll
    for (int c = 0; c < kMax; ++c) {
        const int col = (c * 32 + lane) * kW;
        if (col < dim && VQ_SPAN(out + orow * dim + col, kW, out, tokens * hq * dim)) {
#pragma unroll
            for (int i = 0; i < kW; ++i) out[orow * dim + col + i] = narrow<T>(acc[c][i] * inv);
        }
    }
    if (lane == 0 && lse && VQ_SPAN(lse + orow, 1, lse, tokens * hq)) lse[orow] = paged_lse(top, total);
}

}  // namespace vqk
