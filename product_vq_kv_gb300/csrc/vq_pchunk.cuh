// vq_pchunk.cuh -- paged attention of chunks of new tokens (prefill beside a
// cache, long verification runs): tiles of 128 rows (tokens x query heads of one
// KV head) on the 5th-generation tensor cores, 16-bit types, head sizes 64, 128
// and 256, sub-vectors of 4 or 8.
//
// Per block of kKeys cached tokens, with the accumulators in tensor memory:
//   S (128 x kKeys) = Q K^^T     tcgen05.mma, both operands in shared memory
//   P = 2^(kappa S - m)          one thread per row: its lane of S in registers
//   O (128 x dim)  += P V^       tcgen05.mma, P from tensor memory (over S)
// K^ and V^ are rebuilt from their codes into shared memory by warps that do
// nothing else, from the conflict-free codebook images of the few-row kernel,
// a stage ring ahead of the products.  A rebuilt row is stored as 16-byte
// pieces, piece c of token t at c * 16 kKeys + 16 t: the core matrices (8 rows x
// 16 bytes) of the unswizzled operand layout, with columns as the contraction
// index for the keys and tokens for the values, from one way of writing; eight
// lanes write 128 consecutive bytes, so the writes have no conflict either.
//
// What bounds it at dim 128: the products of a block and two tiles are 4 x 512
// cycles of the tensor pipe; the shared memory moves 2 x 64 KiB for the rebuild,
// 2 x 64 KiB for Q K^^T and 2 x 32 KiB for P V^, 2560 cycles at 128 bytes a
// cycle.  Two tiles share each rebuilt block, or the rebuild alone would take as
// long as the products.  The exponentials (2 x 16384, 32 a cycle) and the rest
// of the softmax run beside both: while the rows of one tile are at their
// softmax the tensor pipe works for the other.  At dim 256 one tile's O fills
// half the tensor memory, so there is one tile, S is double-buffered and Q lies in
// tensor memory too: 1024 cycles of products a block of 64 keys, 1536 of shared
// memory.
//
// The maximum a row's weights refer to follows its scores only when one
// exceeds it by 2^8; then the row's O is rescaled in tensor memory, after the
// product before has finished.  Weights are rounded to the input type for the
// product with V^; their sum takes them unrounded.  (In two pieces, as the few-row
// kernel takes them, the products would grow by half, from 2048 to 3072 of about 3500
// cycles a block at dim 128, and the softmax between them by two packings and a
// subtraction a pair of weights; the error against 64 bits is 0.0017 in bf16 and 0.00022
// in fp16 with one piece, 0.0016 and 0.00021 with fp32 weights.)
//
// Roles (16 warps): 0-3 and 4-7 the softmax and output of tile 0 and 1, 8-11
// rebuild (with one tile 4-7 too), 12 issues the products, 13 walks the segments, 14-15
// only fill the warpgroup (the register
// split below is by warpgroups: 2 x 160 + 96 + 96 registers of each four threads,
// the 4 x 128 that the block is launched with).  Every wait is bounded: one that gives up
// sets the block's abort word and kStatusWaitGaveUp, the others see it and all
// leave; the issuer first waits (bounded) for its products in flight, the tensor
// memory is freed, and the rows that the block has not written become NaN.
#pragma once

#include "vq_pfew.cuh"
#include "vq_status.cuh"
#include "vq_umma.cuh"

namespace vqk {

constexpr int kChunkThreads = 16 * 32;

template <int D>
struct ChunkShape {
    static constexpr int kTiles = D == 256 ? 1 : 2;
    static constexpr int kKeys = D == 256 ? 64 : 128;
    // tensor memory columns: two S buffers from 0, O of tile 0 from 256, O of tile 1
    // D further; with one tile S and O leave 128, which hold its Q (the products
    // Q K^^T then read half as much shared memory, and there are more stages)
    static constexpr int kS = kKeys;  // between the two S buffers
    static constexpr int kO = 256;
    static constexpr bool kQTmem = D == 256;
    static constexpr int kQCol = 128;
    static constexpr int kStages = D == 64 ? 6 : D == 128 ? 3 : 5;
    static constexpr int kStageBytes = kKeys * D * 2;
    static constexpr int kQBytes = kQTmem ? 0 : 128 * D * 2;  // a tile
    static constexpr size_t kSmem = (size_t)kTiles * kQBytes + kStages * kStageBytes + 65536;
};

// Instruction descriptor: kind::f16, fp32 accumulator, 16-bit operands of one
// type (0: fp16, 1: bf16), M = 128, N = n, A K-major, B K-major or MN-major.
__host__ __device__ constexpr uint32_t umma_idesc_16(uint32_t bf16, uint32_t n, bool b_mn)
{
    return (1u << 4) | (bf16 << 7) | (bf16 << 10) | (b_mn ? 1u << 16 : 0u) | ((n >> 3) << 17) | ((128u >> 4) << 24);
}

// The products are issued by one elected lane of a warp whose lanes all run the
// same code: operands that are the same in all of them can stay in uniform
// registers, which is where the instruction takes them from (issued under
// `if (lane == 0)` each cost about 85 cycles, most of it moves).
__device__ __forceinline__ void umma_16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
                 "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// A from tensor memory.
__device__ __forceinline__ void umma_16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate)
{
    asm volatile("{\n\t.reg .pred p, e;\n\tsetp.ne.b32 p, %4, 0;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
                 "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
                 : "memory");
}

// umma_commit by the lane that elect.sync picks (the same one each time).
__device__ __forceinline__ void umma_commit_elected(uint64_t *bar)
{
    asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
                 "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
                 : "memory");
}

__device__ __forceinline__ void tmem_store16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
                 "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
        "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
        "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Polls of a wait: about a second (2^22 took 15 s), where a block of keys takes
// microseconds.  The waits for the next segment, and for room to announce one, last as
// long as a segment: on the longest cache of 2^30 tokens 2^23 units of 2 us, 17 s, so
// their limit is a minute (they also end as soon as any other wait gives up).
constexpr int kChunkPolls = 1 << 18;
constexpr int kSegmentPolls = 1 << 24;

// Bounded wait for phase `parity`: false if it gave up or another role did.
template <int POLLS>
__device__ __forceinline__ bool chunk_wait(uint64_t *bar, uint32_t parity, volatile uint32_t *abort_word)
{
    for (int it = 0; it < POLLS; ++it) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "selp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(smem_addr(bar)), "r"(parity)
                     : "memory");
        if (done) return true;
        if ((it & 15) == 15 && *abort_word) return false;
    }
    *abort_word = 1;
    raise_status(kStatusWaitGaveUp);
    return false;
}

// Bounded wait for a phase of each of two barriers, polled together: one wait after
// the other leaves the tensor pipe idle for the second's round trip (about 270
// cycles where the products wait for both a stage and the weights).
template <int POLLS>
__device__ __forceinline__ bool chunk_wait2(uint64_t *bar0, uint32_t parity0, uint64_t *bar1, uint32_t parity1,
                                            volatile uint32_t *abort_word)
{
    for (int it = 0; it < POLLS; ++it) {
        uint32_t done;
        asm volatile("{\n\t.reg .pred p, q;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
                     "mbarrier.try_wait.parity.shared::cta.b64 q, [%3], %4;\n\t"
                     "and.pred p, p, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
                     : "=r"(done)
                     : "r"(smem_addr(bar0)), "r"(parity0), "r"(smem_addr(bar1)), "r"(parity1)
                     : "memory");
        if (done) return true;
        if ((it & 15) == 15 && *abort_word) return false;
    }
    *abort_word = 1;
    raise_status(kStatusWaitGaveUp);
    return false;
}

// One segment as the roles take it from shared memory.
struct ChunkSeg {
    int64_t tok0, slot;
    int32_t ntok, pos0, k_hi;
    int32_t key0, nb;  // first key, key blocks
    int32_t h, head0, gc;
    int32_t r;
    int32_t whole;     // written to the output, else to the workspace
    int32_t live;      // 0: no more segments
};

// POLLS: the limit of every wait but the last, kChunkPolls except in a test.
template <typename T, int D, int SUB, int POLLS = kChunkPolls>
__global__ void __launch_bounds__(kChunkThreads, 1) paged_attn_chunk(const __grid_constant__ PagedArgs a)
{
    using S = ChunkShape<D>;
    constexpr int NS = D / SUB;
    constexpr int kTiles = S::kTiles, kKeys = S::kKeys, kChunkStages = S::kStages;
    constexpr int kPieces = D / 8;               // 16-byte pieces of a row
    // With one tile warps 4-7 are free to rebuild too: four warps the keys, four the
    // values, each at its own pace (280 -> 241 us at 2048 tokens on 8192 cached).
    // With two tiles the four warps fill stage after stage: two for each kind take
    // twice as long for a stage, and three stages do not hide that (273 -> 287 us).
    constexpr bool kHalves = kTiles == 1;
    constexpr int kKinds = kHalves ? 1 : 2;      // kinds (keys, values) a warp rebuilds
    constexpr int kHalf = 128;                   // threads that fill one stage
    constexpr int kSplit = kHalf / kKeys;        // of them per token
    constexpr int kMyCodes = NS / kSplit;        // code bytes of a thread's token
    constexpr int kMyVec = kMyCodes < 16 ? kMyCodes : 16;
    constexpr int kCodeWords = kMyCodes < 4 ? 1 : kMyCodes / 4;
    constexpr uint32_t kBf16 = std::is_same<T, __nv_bfloat16>::value ? 1u : 0u;
    constexpr float kShift = weight_shift<T>();
    extern __shared__ __align__(128) unsigned char chunk_mem[];
    __shared__ PagedWalk<64> w;
    __shared__ uint64_t full[kChunkStages], empty[kChunkStages], q_full[2], s_full[2], p_full[2], o_done[2], image[2], drain, seg_full[2], seg_empty[2];
    __shared__ ChunkSeg segs[2];
    __shared__ uint32_t valid[8][4];  // per key block (mod 8): which tokens are in a page
    __shared__ uint32_t tmem_slot;
    __shared__ volatile uint32_t abort_word;
    unsigned char *q_mem = chunk_mem;
    unsigned char *ring = chunk_mem + (size_t)kTiles * S::kQBytes;
    unsigned char *k_image = ring + kChunkStages * S::kStageBytes, *v_image = k_image + 32768;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const float kNone = __int_as_float(0xff800000);
    const int tpq = 128 / a.gc;  // tokens of a tile

    if (tid == 0) {
        for (int i = 0; i < kChunkStages; ++i) {
            mbar_init(&full[i], kHalf);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&q_full[i], 128);
            mbar_init(&s_full[i], 1);
            mbar_init(&p_full[i], 128);
            mbar_init(&o_done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&seg_full[i], 1);
            mbar_init(&seg_empty[i], 13);  // a lane of each softmax, rebuild and product warp
        }
        mbar_init(&image[0], kHalf);
        mbar_init(&image[1], kHalf);
        mbar_init(&drain, 1);
        abort_word = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(&tmem_slot)) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_slot;

    PagedLens l;
    const bool work = paged_plan<kChunkThreads>(a, w, l);  // has barriers for the whole block
    if (warp < 8) asm volatile("setmaxnreg.inc.sync.aligned.u32 160;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
    // the next segment of a role's warp: seg_n counts those it has taken; false at
    // the end (or if a wait gave up)
    auto next_seg = [&](uint32_t &seg_n, ChunkSeg &s) -> bool {
        const uint32_t i = seg_n & 1;
        if (!__all_sync(0xffffffffu, chunk_wait<(POLLS == kChunkPolls ? kSegmentPolls : POLLS)>(&seg_full[i], (seg_n >> 1) & 1, &abort_word))) return false;
        s = segs[i];
        __syncwarp();
        if (lane == 0) (void)mbar_arrive(&seg_empty[i]);
        ++seg_n;
        return s.live != 0;
    };
    uint32_t seg_n = 0;
    ChunkSeg s;

    if (work && warp < 4 * kTiles) {
        // ------------------------------------------------ softmax and output
        const int tile = warp >> 2, row = tid & 127;
        const T *__restrict__ q = static_cast<const T *>(a.q);
        T *__restrict__ out = static_cast<T *>(a.out);
        const bool q_vec = (uintptr_t)a.q % 16 == 0 && a.q_stride % 8 == 0;
        const bool out_vec = (uintptr_t)a.out % 16 == 0;
        const int64_t q_elems = (a.tokens - 1) * a.q_stride + (int64_t)a.hq * D;
        const uint32_t lane_base = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const uint32_t o_addr = lane_base + S::kO + (kTiles == 2 ? tile * D : 0);
        uint32_t seen_s[2] = {0, 0};  // phases of s_full that this thread has waited for
        // phases of o_done so far: with one tile the products P V^, with two the
        // segments (there the commit of a block's scores covers the product before)
        uint32_t seen_o = 0;
        uint32_t block = 0;           // key blocks of the segments so far
        bool go = true;
        uint32_t done_n = 0;  // segments written
        while (go && next_seg(seg_n, s)) {
            const int gc = s.gc;
            if (tile * tpq >= s.ntok) {  // no rows here
                block += s.nb;
                ++done_n;
                continue;
            }
            const int tok_in = tile * tpq + row / gc;
            const bool mine = row < tpq * gc && tok_in < s.ntok;
            const int64_t tok = s.tok0 + (mine ? tok_in : 0);
            const int head = s.head0 + (mine ? row % gc : 0);
            // Q: in tensor memory 16-bit pairs by column, in shared memory core
            // matrices: piece c of row r at c * 2048 + 16 r
            {
                const T *src = q + tok * a.q_stride + (int64_t)head * D;
                const bool ok = mine && VQ_SPAN(src, D, q, q_elems);
                auto piece = [&](int c) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (ok) {
                        if (q_vec) {
                            v = __ldg(reinterpret_cast<const uint4 *>(src) + c);
                        } else {
                            const uint16_t *e = reinterpret_cast<const uint16_t *>(src) + 8 * c;
                            v.x = (uint32_t)__ldg(e) | ((uint32_t)__ldg(e + 1) << 16);
                            v.y = (uint32_t)__ldg(e + 2) | ((uint32_t)__ldg(e + 3) << 16);
                            v.z = (uint32_t)__ldg(e + 4) | ((uint32_t)__ldg(e + 5) << 16);
                            v.w = (uint32_t)__ldg(e + 6) | ((uint32_t)__ldg(e + 7) << 16);
                        }
                    }
                    return v;
                };
                if constexpr (S::kQTmem) {
#pragma unroll 1
                    for (int c = 0; c < kPieces; c += 8) {
                        uint32_t v[32];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const uint4 x = piece(c + i);
                            v[4 * i] = x.x;
                            v[4 * i + 1] = x.y;
                            v[4 * i + 2] = x.z;
                            v[4 * i + 3] = x.w;
                        }
                        tmem_store32(lane_base + S::kQCol + c * 4, v);
                    }
                    tmem_wait_st();
                    tc_fence_before();
                } else {
                    unsigned char *dst = q_mem + tile * S::kQBytes + row * 16;
#pragma unroll 8
                    for (int c = 0; c < kPieces; ++c) {
                        const uint4 v = piece(c);
                        if (dyn_smem_ok(dst + c * 2048, 16, 16)) *reinterpret_cast<uint4 *>(dst + c * 2048) = v;
                    }
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                }
                (void)mbar_arrive(&q_full[tile]);
            }
            // what this row sees: tokens in (low, lim]
            const int32_t pos = s.pos0 + (mine ? tok_in : tile * tpq);
            const int32_t lim = pos < s.k_hi ? pos : s.k_hi - 1;
            const int64_t low64 = (int64_t)pos - a.window;
            const int32_t low = a.window == 0 || low64 < -1 ? -1 : (int32_t)low64;
            // what every row of the tile sees
            const int32_t pos_first = s.pos0 + tile * tpq;
            const int ntile = s.ntok - tile * tpq < tpq ? s.ntok - tile * tpq : tpq;
            const int32_t all_hi = pos_first < s.k_hi ? pos_first : s.k_hi - 1;
            const int64_t all_lo = a.window == 0 ? -1 : (int64_t)pos_first + ntile - 1 - a.window;

            float m = kNone;
            uint32_t saw = 0;  // not 0: this row has seen a token
            float2 sum2 = make_float2(0.f, 0.f);  // over the even and the odd tokens
            for (int j = 0; j < s.nb; ++j, ++block) {
                const int buf = kTiles == 2 ? tile : j & 1;
                if (!__all_sync(0xffffffffu, chunk_wait<POLLS>(&s_full[buf], seen_s[buf] & 1, &abort_word))) {
                    go = false;
                    break;
                }
                ++seen_s[buf];
                tc_fence_after();
                const uint32_t s_addr = lane_base + buf * S::kS;
                const int32_t k0 = s.key0 + j * kKeys;
                bool whole = k0 + kKeys - 1 <= all_hi && k0 > all_lo;
#pragma unroll
                for (int i = 0; i < kKeys / 32; ++i) whole &= valid[block & 7][i] == 0xffffffffu;
                // bit i: this row sees token 32 c + i of the block
                auto seen_bits = [&](int c) -> uint32_t {
                    const int32_t hi = lim - (k0 + 32 * c), lo = low - (k0 + 32 * c);
                    const uint32_t upto = hi < 0 ? 0u : hi >= 31 ? 0xffffffffu : (2u << hi) - 1u;
                    const uint32_t past = lo < 0 ? 0u : lo >= 31 ? 0xffffffffu : (2u << lo) - 1u;
                    return upto & ~past & valid[block & 7][c];
                };
                // scores to weights, two at a time; adds them up
                auto weights = [&](const uint32_t *v, uint32_t *p, int n, float ref, float2 &add) {
#pragma unroll
                    for (int i = 0; i < n; i += 2) {
                        float2 x = fma2_rn(make_float2(__uint_as_float(v[i]), __uint_as_float(v[i + 1])),
                                           make_float2(a.kappa, a.kappa), make_float2(-ref, -ref));
                        x.x = exp2_fast(x.x);
                        x.y = exp2_fast(x.y);
                        add = add2_rn(add, x);
                        p[i / 2] = pack2<T>(x.x, x.y);
                    }
                };
                bool done = false;
                if (whole && j > 0) {  // the same for all rows of the tile
                    // one pass with the maximum so far, kept if no score of the warp's
                    // rows exceeds it by more than the slack; the scores still stand then
                    uint32_t p[kKeys / 2];
                    float tops[4] = {kNone, kNone, kNone, kNone};
                    float2 add = make_float2(0.f, 0.f);
#pragma unroll
                    for (int c = 0; c < kKeys / 32; ++c) {
                        uint32_t v[32];
                        tmem_load32_async(s_addr + c * 32, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 32; i += 8)
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                tops[k] = max3(tops[k], __uint_as_float(v[i + 2 * k]), __uint_as_float(v[i + 2 * k + 1]));
                        weights(v, p + c * 16, 32, m, add);
                    }
                    const float top = max3(fmaxf(tops[0], tops[1]), tops[2], tops[3]) * a.kappa;
                    if (!__any_sync(0xffffffffu, top > m + (kFewSlack + kShift) || m == kNone)) {
                        done = true;
                        sum2 = add2_rn(sum2, add);
#pragma unroll
                        for (int c = 0; c < kKeys / 32; ++c) tmem_store16(s_addr + c * 16, *reinterpret_cast<uint32_t(*)[16]>(p + c * 16));
                    }
                }
                if (!done) {
                    // first the maximum, then the weights
                    float top = kNone;
#pragma unroll 1
                    for (int c = 0; c < kKeys / 32; ++c) {
                        uint32_t v[32];
                        tmem_load32_async(s_addr + c * 32, v);
                        const uint32_t bits = seen_bits(c);
                        saw |= bits;
                        tmem_wait_ld(v);
#pragma unroll
                        for (int i = 0; i < 32; ++i) top = fmaxf(top, (bits >> i) & 1u ? __uint_as_float(v[i]) : kNone);
                    }
                    top *= a.kappa;  // kappa > 0
                    // a row rises for its own scores alone, so that what it computes does
                    // not depend on the rows beside it; the others are scaled by 1
                    const bool rise = top > m + (kFewSlack + kShift);
                    if (__any_sync(0xffffffffu, rise)) {
                        const float to = rise ? top - kShift : m;
                        const float f = rise ? exp2_fast(m - to) : 1.f;
                        m = to;
                        sum2 = make_float2(sum2.x * f, sum2.y * f);
                        if (j > 0) {
                            // the product before this block has to be done
                            if (kTiles == 1 && !__all_sync(0xffffffffu, chunk_wait<POLLS>(&o_done[tile], (seen_o - 1) & 1, &abort_word))) {
                                go = false;
                                break;
                            }
                            tc_fence_after();
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t v[32];
                                tmem_load32_async(o_addr + c * 32, v);
                                tmem_wait_ld(v);
#pragma unroll
                                for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * f);
                                tmem_store32(o_addr + c * 32, v);
                            }
                        }
                    }
                    const float ref = m == kNone ? 0.f : m;  // nothing seen yet: every weight is 0
                    float2 add = make_float2(0.f, 0.f);
                    // (a load of 32 columns is read before the 16 columns of its weights
                    // are written below it)
#pragma unroll 1
                    for (int c = 0; c < kKeys / 32; ++c) {
                        uint32_t v[32], p[16];
                        tmem_load32_async(s_addr + c * 32, v);
                        const uint32_t bits = seen_bits(c);
                        tmem_wait_ld(v);
                        // a score that is not seen is left out as -inf: weight 0, whatever it was
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = (bits >> i) & 1u ? v[i] : 0xff800000u;
                        weights(v, p, 32, ref, add);
                        tmem_store16(s_addr + c * 16, p);
                    }
                    sum2 = add2_rn(sum2, add);
                }
                tmem_wait_st();
                if (kTiles == 1 && j > 0) {
                    // a wait tells only the last two phases of a barrier apart, and the
                    // scores of this block were issued before the product before: wait for
                    // each product in turn
                    if (!__all_sync(0xffffffffu, chunk_wait<POLLS>(&o_done[tile], (seen_o - 1) & 1, &abort_word))) {
                        go = false;
                        break;
                    }
                }
                tc_fence_before();
                (void)mbar_arrive(&p_full[buf]);
                if (kTiles == 1) ++seen_o;
            }
            if (!go) break;
            if (kTiles == 2) ++seen_o;
            if (!__all_sync(0xffffffffu, chunk_wait<POLLS>(&o_done[tile], (seen_o - 1) & 1, &abort_word))) break;
            tc_fence_after();
            float sum = sum2.x + sum2.y;
            // (scores of -inf alone: m is -inf still, and every block came through the
            // path that looks at the masks)
            if (sum == 0.f && saw) sum = 1.f;
            const float inv = paged_inv(m, sum);
            const int64_t orow = tok * a.hq + head;
            const int64_t prow = s.slot * a.tile_rows + tile * tpq * gc + row, prows = 2 * (int64_t)gridDim.x * a.tile_rows;
            T *dst = out + orow * D;
            float *pdst = a.part + prow * D;
            const bool put = mine && (s.whole ? VQ_SPAN(dst, D, out, a.tokens * a.hq * D) : VQ_VSPAN(pdst, D, a.part, prows * D, 16));
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
                uint32_t v[32];
                tmem_load32_async(o_addr + c * 32, v);
                tmem_wait_ld(v);
                if (!put) continue;
                if (s.whole) {
                    if (out_vec) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t x[4];
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                x[k] = pack2<T>(__uint_as_float(v[8 * i + 2 * k]) * inv, __uint_as_float(v[8 * i + 2 * k + 1]) * inv);
                            reinterpret_cast<uint4 *>(dst)[c * 4 + i] = make_uint4(x[0], x[1], x[2], x[3]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) dst[c * 32 + i] = narrow<T>(__uint_as_float(v[i]) * inv);
                    }
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        reinterpret_cast<uint4 *>(pdst)[c * 8 + i] = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
                }
            }
            tc_fence_before();
            if (mine && s.whole && a.lse && VQ_SPAN(a.lse + orow, 1, a.lse, a.tokens * a.hq)) a.lse[orow] = paged_lse(m, sum);
            if (mine && !s.whole && VQ_SPAN(a.ml + prow * 2, 2, a.ml, prows * 2)) {
                a.ml[prow * 2] = m;
                a.ml[prow * 2 + 1] = sum;
            }
            ++done_n;
        }
        if (abort_word) {
            // a wait gave up: this thread's rows of the segments not written become NaN, in
            // the output or by way of the merge
            const float nan = __int_as_float(0x7fffffff);
            PagedCursor cur;
            cur.init(w, (int32_t)blockIdx.x);
            PagedSegment seg;
            PagedNote note{};
            const PagedLens lens = paged_lens(a, w);
            for (uint32_t n = 0; cur.next(a, w, lens, seg, note); ++n) {
                const int g0 = seg.hx % a.gch * a.gc, gc = a.group - g0 < a.gc ? a.group - g0 : a.gc;
                const int tok_in = tile * tpq + row / gc;
                if (n < done_n || row >= tpq * gc || tok_in >= seg.it.ntok) continue;
                const int64_t orow = (seg.it.tok0 + tok_in) * a.hq + seg.hx / a.gch * a.group + g0 + row % gc;
                const int64_t prow = seg.slot * a.tile_rows + tile * tpq * gc + row, prows = 2 * (int64_t)gridDim.x * a.tile_rows;
                if (!seg.whole) {
                    if (VQ_SPAN(a.ml + prow * 2, 2, a.ml, prows * 2)) {
                        a.ml[prow * 2] = 0.f;
                        a.ml[prow * 2 + 1] = nan;
                    }
                    continue;
                }
                if (VQ_SPAN(out + orow * D, D, out, a.tokens * a.hq * D)) {
#pragma unroll 1
                    for (int d = 0; d < D; ++d) out[orow * D + d] = narrow<T>(nan);
                }
                if (a.lse && VQ_SPAN(a.lse + orow, 1, a.lse, a.tokens * a.hq)) a.lse[orow] = nan;
            }
        }
    } else if (work && warp < 12) {
        // ------------------------------------------------ rebuild
        const int me = tid - 128 * kTiles;
        const int vals = kHalves && me >= kHalf ? 1 : 0;  // warp-uniform: which half this is
        const int in_half = me - vals * kHalf;
        const int tk = in_half % kKeys, part = in_half / kKeys;  // token of the block, which part of its row
        const uint32_t copy = (uint32_t)(lane % (64 / SUB)) * (2 * SUB);
        const int64_t cb_elems = (int64_t)a.hkv * a.nc * SUB;
        const int64_t code_bytes = (a.num_pages - 1) * a.page_stride + (((int64_t)a.hkv * NS) << a.page_shift);
        uint32_t base_n = 0;  // stages of the segments so far
        uint32_t block = 0;   // key blocks of them
        int built = -1;
        bool go = true;
        // the warps that share an image meet (bounded, as every wait here)
        uint32_t met = 0;
        auto meet = [&]() -> bool {
            (void)mbar_arrive(&image[vals]);
            return __all_sync(0xffffffffu, chunk_wait<POLLS>(&image[vals], met++ & 1, &abort_word));
        };
        while (go && next_seg(seg_n, s)) {
            const int h = s.h;
            if (h != built) {
                // the images of this head: only these warps read them
                if (!(go = meet())) break;
#pragma unroll 1
                for (int kd = 0; kd < kKinds; ++kd) {
                    const bool v = kHalves ? vals : kd;
                    const T *all = static_cast<const T *>(v ? a.vcb : a.kcb);
#pragma unroll 1
                    for (int c = in_half; c < 256; c += kHalf) {
                        uint32_t wd[SUB / 2];
                        book_row<T, SUB>(all + (int64_t)h * a.nc * SUB, c, a.nc, all, cb_elems, wd);
                        image_line<SUB>(v ? v_image : k_image, c, wd);
                    }
                }
                if (!(go = meet())) break;
                built = h;
            }
            const int32_t key0 = s.key0;
            const int nb = s.nb;
            const int64_t none_lo = a.window == 0 ? -1 : (int64_t)s.pos0 - a.window;  // no row sees at or below
            // this thread's token of block j: its page entry, or -1; checked when it is
            // used (a check here would wait for the load)
            auto page_of = [&](int j) -> int32_t {
                const int64_t t = (int64_t)key0 + (int64_t)j * kKeys + tk;
                if (j >= nb || t >= s.k_hi || t <= none_lo) return -1;
                return paged_entry(a, s.r, (int32_t)t);
            };
            const int64_t head_off = ((int64_t)h << a.page_shift) * NS + part * kMyCodes;
            auto load = [&](int j, int32_t &pg, uint32_t (&codes)[kKinds][kCodeWords]) {
                if (pg < 0 || pg >= a.num_pages) {
                    pg = -1;
                    return;
                }
                const int32_t off = (key0 + j * kKeys + tk) & ((1 << a.page_shift) - 1);
                const int64_t at = head_off + (int64_t)pg * a.page_stride + off * NS;
#pragma unroll
                for (int kd = 0; kd < kKinds; ++kd) {
                    const uint8_t *all = (kHalves ? vals : kd) ? a.v_codes : a.k_codes;
                    if (!span_ok(all + at, kMyCodes, all, code_bytes, kMyVec)) continue;
#pragma unroll
                    for (int i = 0; i < kMyCodes / kMyVec; ++i) {
                        uint32_t v[(kMyVec + 3) / 4];
                        load_codes<kMyVec>(all + at + i * kMyVec, v);
#pragma unroll
                        for (int k = 0; k < (kMyVec + 3) / 4; ++k) codes[kd][i * (kMyVec / 4) + k] = v[k];
                    }
                }
            };
            // a block's place in the ring: with two tiles the stages go K0 V0 K1 V1 ..,
            // with one K0 K1 V0 K2 V1 .. (there the scores of a block are issued before
            // the product of the one before)
            auto stage_of = [&](int j, int v) -> uint32_t {
                if (kTiles == 2) return base_n + 2 * j + v;
                if (v) return base_n + (j + 1 < nb ? 2 * j + 2 : 2 * j + 1);
                return base_n + (j > 0 ? 2 * j - 1 : 0);
            };
            // rebuild this thread's part of its token of block j
            auto fill = [&](int j, int v, bool live, const uint32_t (&codes)[kCodeWords]) -> bool {
                const unsigned char *base = (v ? v_image : k_image) + copy;
                const uint32_t n = stage_of(j, v), st = n % kChunkStages, round = n / kChunkStages;
                // (the stages are released in ring order, so that the phase before the one
                // waited for is over)
                if (round > 0 && !__all_sync(0xffffffffu, chunk_wait<POLLS>(&empty[st], (round - 1) & 1, &abort_word))) return false;
                if (v == 0) {
                    // the words that lay here, eight blocks back, have been read: the stage
                    // just released held keys or values of a block at most four back, and
                    // was released after the weights of the one before that
                    const uint32_t have = __ballot_sync(0xffffffffu, live);
                    if (lane == 0 && part == 0) valid[block & 7][tk / 32] = have;
                }
                unsigned char *dst = ring + st * S::kStageBytes + (part * (kPieces / kSplit)) * (16 * kKeys) + tk * 16;
                // eight pieces at a time, so that their loads overlap
                constexpr int kMyPieces = kPieces / kSplit, kBatch = kMyPieces < 8 ? kMyPieces : 8;
#pragma unroll
                for (int c0 = 0; c0 < kMyPieces; c0 += kBatch) {
                    uint32_t w[kBatch][4];
#pragma unroll
                    for (int c = 0; c < kBatch; ++c) {
                        if constexpr (SUB == 8) {
                            image_row<8>(base, code_at(codes, c0 + c), w[c]);
                        } else {
                            uint32_t lo[2], hi[2];
                            image_row<4>(base, code_at(codes, 2 * (c0 + c)), lo);
                            image_row<4>(base, code_at(codes, 2 * (c0 + c) + 1), hi);
                            w[c][0] = lo[0];
                            w[c][1] = lo[1];
                            w[c][2] = hi[0];
                            w[c][3] = hi[1];
                        }
                    }
                    if (!live) {  // no token: finite whatever its codes would be
#pragma unroll
                        for (int c = 0; c < kBatch; ++c) w[c][0] = w[c][1] = w[c][2] = w[c][3] = 0;
                    }
#pragma unroll
                    for (int c = 0; c < kBatch; ++c) {
                        unsigned char *to = dst + (c0 + c) * (16 * kKeys);
                        if (dyn_smem_ok(to, 16, 16)) *reinterpret_cast<uint4 *>(to) = make_uint4(w[c][0], w[c][1], w[c][2], w[c][3]);
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                (void)mbar_arrive(&full[st]);
                return true;
            };
            // codes one block ahead, page entries two
            uint32_t codes[2][kKinds][kCodeWords] = {};
            int32_t pg[3];
            pg[0] = page_of(0);
            pg[1] = page_of(1);
            load(0, pg[0], codes[0]);
            for (int j = 0; j < nb; ++j, ++block) {
                load(j + 1, pg[1], codes[1]);
                pg[2] = page_of(j + 2);
#pragma unroll
                for (int kd = 0; kd < kKinds; ++kd)
                    if (go) go = fill(j, kHalves ? vals : kd, pg[0] >= 0, codes[0][kd]);
                if (!go) break;
                pg[0] = pg[1];
                pg[1] = pg[2];
#pragma unroll
                for (int kd = 0; kd < kKinds; ++kd)
#pragma unroll
                    for (int i = 0; i < kCodeWords; ++i) codes[0][kd][i] = codes[1][kd][i];
            }
            base_n += 2 * nb;
        }
    } else if (work && warp == 12) {
        // ------------------------------------------------ the products
        const uint32_t idesc_s = umma_idesc_16(kBf16, kKeys, false), idesc_o = umma_idesc_16(kBf16, D, true);
        const uint32_t q_addr = smem_addr(q_mem), ring_addr = smem_addr(ring);
        uint32_t taken = 0;  // stages taken so far
        uint32_t n_q[2] = {0, 0}, n_p[2] = {0, 0};
        bool go = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
            return __all_sync(0xffffffffu, chunk_wait<POLLS>(bar, parity, &abort_word));
        };
        // wait for the next stage in ring order; its index
        auto take = [&](uint32_t *st) -> bool {
            *st = taken % kChunkStages;
            const uint32_t round = taken / kChunkStages;
            ++taken;
            return wait(&full[*st], round & 1);
        };
        // the next stage and a tile's weights (with one tile: 243 -> 234 us at 2048
        // tokens on 8192 cached; with two the tiles then fall into step, their softmax
        // side by side instead of one beside the other's products: 265 -> 281)
        auto take_with = [&](uint32_t *st, int buf) -> bool {
            *st = taken % kChunkStages;
            const uint32_t round = taken / kChunkStages;
            ++taken;
            return __all_sync(0xffffffffu, chunk_wait2<POLLS>(&full[*st], round & 1, &p_full[buf], n_p[buf]++ & 1, &abort_word));
        };
        // operand descriptors differ in the address field alone (16-byte units,
        // no carry out of it below 256 KiB): one addition each
        const uint64_t q_desc = umma_smem_desc(q_addr, 2048, 128);
        const uint64_t k_desc = umma_smem_desc(ring_addr, 16 * kKeys, 128);
        const uint64_t v_desc = umma_smem_desc(ring_addr, 128, 16 * kKeys);
        auto scores = [&](int tile, int buf, uint32_t st) {
            const uint64_t qd = q_desc + (uint32_t)(tile * (S::kQBytes / 16)), kd = k_desc + st * (uint32_t)(S::kStageBytes / 16);
            const uint32_t d = tmem + buf * S::kS;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                if constexpr (S::kQTmem) umma_16_ts(d, tmem + S::kQCol + k * 8, kd + k * (2 * kKeys), idesc_s, k > 0);
                else umma_16_ss(d, qd + k * 256, kd + k * (2 * kKeys), idesc_s, k > 0);
            }
            umma_commit_elected(&s_full[buf]);
        };
        auto values = [&](int tile, int buf, uint32_t st, bool add) {
            const uint64_t vd = v_desc + st * (uint32_t)(S::kStageBytes / 16);
            const uint32_t d = tmem + S::kO + (kTiles == 2 ? tile * D : 0), p = tmem + buf * S::kS;
#pragma unroll
            for (int k = 0; k < kKeys / 16; ++k) umma_16_ts(d, p + k * 8, vd + k * 16, idesc_o, add || k > 0);
        };
        while (go && next_seg(seg_n, s)) {
            const int nb = s.nb;
            const int tiles = kTiles == 2 && s.ntok > tpq ? 2 : 1;
            for (int t = 0; go && t < tiles; ++t) go = wait(&q_full[t], n_q[t]++ & 1);
            uint32_t ks, vs;
            if (!go || !take(&ks)) break;
            tc_fence_after();
            for (int t = 0; t < tiles; ++t) scores(t, kTiles == 2 ? t : 0, ks);
            umma_commit_elected(&empty[ks]);
            for (int j = 0; j < nb; ++j) {
                const bool more = j + 1 < nb;
                if (kTiles == 1) {
                    if (more) {
                        // into the other S buffer: its weights were taken by the product before
                        if (!(go = take(&ks))) break;
                        tc_fence_after();
                        scores(0, (j + 1) & 1, ks);
                        umma_commit_elected(&empty[ks]);
                    }
                    if (!(go = take_with(&vs, j & 1))) break;
                    tc_fence_after();
                    values(0, j & 1, vs, j > 0);
                    umma_commit_elected(&o_done[0]);
                    umma_commit_elected(&empty[vs]);
                    continue;
                }
                if (!(go = take(&vs))) break;
                for (int t = 0; t < tiles; ++t) {
                    if (!(go = wait(&p_full[t], n_p[t]++ & 1))) break;
                    tc_fence_after();
                    values(t, t, vs, j > 0);
                    if (!more) umma_commit_elected(&o_done[t]);  // else the next scores' commit covers it
                    if (t == tiles - 1) umma_commit_elected(&empty[vs]);
                    if (more) {
                        // the next keys are waited for while the first product runs (the
                        // next values, waited for here too, would hold the scores up)
                        if (t == 0 && !(go = take(&ks))) break;
                        tc_fence_after();
                        // products run in the order of issue: the weights, which lie over
                        // S, are read before the next scores are written there
                        scores(t, t, ks);
                        if (t == tiles - 1) umma_commit_elected(&empty[ks]);
                    }
                }
                if (!go) break;
            }
        }
        // products in flight write tensor memory and read shared memory: let them end
        umma_commit_elected(&drain);
        (void)mbar_wait(&drain, 0);
    } else if (work && warp == 13) {
        // ------------------------------------------------ the segments
        PagedCursor cur;
        cur.init(w, (int32_t)blockIdx.x);
        PagedSegment seg;
        PagedNote note{};
        bool more = true;
        for (uint32_t n = 0; more; ++n) {
            const uint32_t i = n & 1;
            more = cur.next(a, w, l, seg, note);
            if (n >= 2 && !__all_sync(0xffffffffu, chunk_wait<(POLLS == kChunkPolls ? kSegmentPolls : POLLS)>(&seg_empty[i], ((n >> 1) - 1) & 1, &abort_word))) break;
            if (lane == 0) {
                ChunkSeg &to = segs[i];
                to.live = more;
                if (more) {
                    const int g0 = seg.hx % a.gch * a.gc;
                    to.h = seg.hx / a.gch;
                    to.gc = a.group - g0 < a.gc ? a.group - g0 : a.gc;
                    to.head0 = to.h * a.group + g0;
                    to.tok0 = seg.it.tok0;
                    to.slot = seg.slot;
                    to.ntok = seg.it.ntok;
                    to.pos0 = seg.it.pos0;
                    to.k_hi = seg.it.k_hi;
                    to.r = cur.r;
                    to.whole = seg.whole;
                    const int32_t k0 = seg.it.k_lo + seg.begin * kUnit;
                    const int64_t k1 = (int64_t)seg.it.k_lo + (int64_t)seg.end * kUnit;
                    const int32_t end = k1 < seg.it.k_hi ? (int32_t)k1 : seg.it.k_hi;
                    to.key0 = k0;
                    to.nb = end > k0 ? (end - k0 + kKeys - 1) / kKeys : 1;
                }
                (void)mbar_arrive(&seg_full[i]);
            }
            __syncwarp();
        }
        while (more) more = cur.next(a, w, l, seg, note);  // a wait gave up: the note is due all the same
        if (lane == 0 && VQ_SPAN(a.notes + blockIdx.x, 1, a.notes, gridDim.x)) a.notes[blockIdx.x] = note;
    } else if (!work && warp == 13 && lane == 0) {
        if (VQ_SPAN(a.notes + blockIdx.x, 1, a.notes, gridDim.x)) a.notes[blockIdx.x] = PagedNote{};
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 12) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

}  // namespace vqk
