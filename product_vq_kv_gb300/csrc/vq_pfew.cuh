// vq_pfew.cuh -- paged attention of a few rows (decode, verification of
// drafts): up to 8 rows (tokens x query heads of one KV head) against the whole
// cache, 16-bit types, head sizes 64, 128 and 256, sub-vectors of 4 or 8.
//
// What bounds it.  From HBM a cached token costs 2 ns bytes a KV head (32 at
// head size 128, sub-vectors of 8); rebuilding its key and value rows costs 2 x
// 2 dim = 512 bytes out of the codebooks.  An SM reads 128 bytes of shared
// memory a cycle, so with the codebooks there the rebuild is the bound: 4 cycles
// a token and KV head, against 1.4 cycles of its share of HBM.  Everything is
// laid out so that a rebuilt value is read once, without a bank conflict, and
// goes nowhere but into the registers of the matrix instruction that uses it:
//   * mma.m16n8k16 with the cached tokens (keys) or the head's columns (values)
//     as the 16 rows and the query rows as the 8 columns, so that few rows cost
//     few instructions:  S^T = K^ Q^T,  O^T = V^^T P^T.  (tcgen05 takes its
//     operands from shared or tensor memory, which would cost a write and a second
//     read of every rebuilt value.)
//   * Which column of the head an instruction's k index means is free as long as
//     both operands agree.  Lane (g, t) = (lane / 4, lane % 4) takes columns
//     [t dim/4, (t+1) dim/4) of keys g and g + 8: whole codebook rows, one 16- or
//     8-byte load each, and its codes are consecutive bytes of the cache.  For the
//     values it takes columns [g dim/8, (g+1) dim/8) of tokens 2t, 2t+1, 2t+8,
//     2t+9 and pairs the tokens with byte permutes.
//   * Each codebook lies in shared memory as 256 lines of 128 bytes, a line
//     holding 8 (16) copies of one 16 (8) byte row.  The lanes that a 128-byte
//     wavefront serves read different copies: no conflicts, whatever the codes.
//   * P^T reaches the second product through movmatrix, an 8x8 transpose inside
//     the warp.  Nothing of the inner loop but the codebooks touches shared
//     memory, and no barrier stands in it: the warps take groups of 16 tokens
//     in turn and keep their own softmax states.
//   * Codes come straight from global memory into registers two groups ahead, the
//     page numbers three.
//   * The running maximum follows the scores only when one exceeds it by 2^8
//     (a vote); until then nothing is rescaled (weight_shift says what range the
//     weights then have).
// A weight goes into the second product in two pieces of the input type, the second
// what rounding the first leaves: 22 bits of fp16, 16 of bf16, where one piece would add
// half a step of the type to every row that one token decides (its weight is any number
// up to 2^8 and not 1, as the maximum lags).  Twice the products and the packing cost
// 6 to 8 % (8 requests of 32768 at dim 128: 70 -> 74 us; 32 uneven ones 134 -> 145), and
// the error against 64 bits is that of fp32 weights, 0.00021 where it was 0.00025 for one
// token on 777.  The sum of weights takes them as they are, in fp32.
#pragma once

#include <type_traits>

#include "vq_pattn.cuh"

namespace vqk {

constexpr float kFewSlack = 8.f;  // powers of two by which a row's maximum may lag

// Powers of two that the weights of 16-bit products are shifted up by: the
// reference of a row is its maximum (as far as it has followed) less this much.
// fp16 has nothing below 2^-24: unshifted, 131072 tokens at 2^-26 beside one token
// at 1 would count in the sum, 2^-9 of it, and not in the product.  At 7 the largest
// weight is 2^(7 + 8), inside fp16, and the least one that is kept 2^-32 of the
// maximum's.  bf16 has fp32's range and needs none.
template <typename T>
__host__ __device__ constexpr float weight_shift()
{
    return std::is_same<T, __half>::value ? 7.f : 0.f;
}

constexpr int kFewRows = 8;     // columns of a matrix instruction
// A row's maximum before it has seen a token: finite, so that the weight of a
// hidden score, -inf, is 0 against it too (-inf less -inf would be NaN).
constexpr float kFewLow = -3.402823466e38f;

// Warps of a block and blocks of an SM: two blocks where a lane's accumulators
// and queries (dim/16 x 6 registers) fit 128 registers.  At dim 256 one block of 8
// warps at 255 registers (8 requests of 32768: 78 us): 12 at 168 spill (105 against 74
// us, with weights in one piece).  Items of 16 rows, two columns of instructions on each
// rebuilt value, took 70 us for drafts where two items of 8 took 52: twice the registers
// leave fewer warps.
template <int D>
struct FewShape {
    static constexpr int kWarps = 8;
    static constexpr int kBlocks = D > 128 ? 1 : 2;
    // shared memory: two codebook images of 32 KiB, then the merge's slots
    static constexpr size_t kSmem = 2 * 32768 + (size_t)(kWarps / 2) * kFewRows * D * sizeof(float);
};

template <typename T>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    if constexpr (std::is_same<T, __half>::value)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Two fp32 values rounded to the 16-bit type, the first in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    uint32_t r;
    if constexpr (std::is_same<T, __half>::value)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// The two values of a pack2, in fp32.
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t v)
{
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    else return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

// 2^x, 0 for -inf; error 2 ulp (2^-22).
__device__ __forceinline__ float exp2_fast(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// BYTES consecutive code bytes in words, low byte first.
template <int BYTES>
__device__ __forceinline__ void load_codes(const uint8_t *p, uint32_t (&w)[(BYTES + 3) / 4])
{
    if constexpr (BYTES == 1) w[0] = __ldg(p);
    if constexpr (BYTES == 2) w[0] = __ldg(reinterpret_cast<const uint16_t *>(p));
    if constexpr (BYTES == 4) w[0] = __ldg(reinterpret_cast<const uint32_t *>(p));
    if constexpr (BYTES == 8) {
        const uint2 v = __ldg(reinterpret_cast<const uint2 *>(p));
        w[0] = v.x;
        w[1] = v.y;
    }
    if constexpr (BYTES == 16) {
        const uint4 v = __ldg(reinterpret_cast<const uint4 *>(p));
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    }
}

// Byte i of w[] as an unsigned number; i is a constant after unrolling.
template <int W>
__device__ __forceinline__ uint32_t code_at(const uint32_t (&w)[W], int i)
{
    return __byte_perm(w[i >> 2], 0, 0x4440 | (i & 3));
}

// One codebook row of SUB 16-bit values from its image: SUB / 2 words.  `base`
// = the image (in shared memory) plus this lane's copy offset.  (A plain load and
// not an asm statement, which would stand in the order of the matrix
// instructions: the compiler then starts the loads ahead of them.)
template <int SUB>
__device__ __forceinline__ void image_row(const unsigned char *base, uint32_t code, uint32_t (&w)[SUB / 2])
{
    const unsigned char *at = base + code * 128u;
    if constexpr (SUB == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(at);
        w[0] = v.x;
        w[1] = v.y;
        w[2] = v.z;
        w[3] = v.w;
    } else {
        const uint2 v = *reinterpret_cast<const uint2 *>(at);
        w[0] = v.x;
        w[1] = v.y;
    }
}

// Row c of a codebook (zero past its end) as SUB / 2 words.
template <typename T, int SUB>
__device__ __forceinline__ void book_row(const T *__restrict__ cb, int c, int nc, const T *all, int64_t all_elems,
                                         uint32_t (&w)[SUB / 2])
{
#pragma unroll
    for (int i = 0; i < SUB / 2; ++i) w[i] = 0;
    if (c < nc && VQ_SPAN(cb + (int64_t)c * SUB, SUB, all, all_elems)) {
        const uint16_t *src = reinterpret_cast<const uint16_t *>(cb + (int64_t)c * SUB);
#pragma unroll
        for (int i = 0; i < SUB / 2; ++i) w[i] = (uint32_t)__ldg(src + 2 * i) | ((uint32_t)__ldg(src + 2 * i + 1) << 16);
    }
}

// Line c of a codebook's image: its row 64 / SUB times.  The copies are
// written in an order that starts at c, so that the lanes of a wavefront meet in
// no bank.  The caller synchronises.
template <int SUB>
__device__ __forceinline__ void image_line(unsigned char *image, int c, const uint32_t (&w)[SUB / 2])
{
    constexpr int kCopies = 64 / SUB;
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
        unsigned char *dst = image + c * 128 + ((c + k) % kCopies) * (2 * SUB);
        if (!dyn_smem_ok(dst, 2 * SUB, 2 * SUB)) continue;
        if constexpr (SUB == 8) *reinterpret_cast<uint4 *>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
        else *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
    }
}

template <typename T, int D, int SUB>
__global__ void __launch_bounds__(FewShape<D>::kWarps * 32, FewShape<D>::kBlocks)
    paged_attn_few(const __grid_constant__ PagedArgs a)
{
    constexpr int kFewWarps = FewShape<D>::kWarps, kFewThreads = kFewWarps * 32;
    constexpr int NS = D / SUB;
    constexpr int KB = NS / 4, VB = NS / 8;        // code bytes a lane takes of a key, of a value
    constexpr int KW = (KB + 3) / 4, VW = (VB + 3) / 4;
    constexpr int kMma = D / 16;                   // instructions per 16 tokens and 8 rows, each product
    constexpr float kShift = weight_shift<T>();
    static_assert(SUB == 4 || SUB == 8, "sub-vectors of 4 or 8");
    extern __shared__ __align__(128) unsigned char few_mem[];
    __shared__ PagedWalk<> w;
    __shared__ float wm[kFewWarps][kFewRows], wl[kFewWarps][kFewRows];
    unsigned char *k_image = few_mem, *v_image = few_mem + 32768;
    float *slots = reinterpret_cast<float *>(few_mem + 65536);

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const float kNone = __int_as_float(0xff800000);
    const uint32_t copy = (uint32_t)(lane % (64 / SUB)) * (2 * SUB);
    const unsigned char *k_base = k_image + copy, *v_base = v_image + copy;
    const T *__restrict__ q = static_cast<const T *>(a.q);
    T *__restrict__ out = static_cast<T *>(a.out);
    const bool q_vec = (uintptr_t)a.q % 8 == 0 && a.q_stride % 4 == 0;
    const bool out_vec = (uintptr_t)a.out % 16 == 0;
    const int64_t cb_elems = (int64_t)a.hkv * a.nc * SUB;
    const int64_t q_elems = (a.tokens - 1) * a.q_stride + (int64_t)a.hq * D;
    const int64_t code_bytes = (a.num_pages - 1) * a.page_stride + (((int64_t)a.hkv * NS) << a.page_shift);

    // the merge's blocks may take the room that idle blocks leave (they wait there)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    PagedLens l;
    PagedNote note{};
    if (paged_plan<kFewThreads>(a, w, l)) {
        PagedCursor cur;
        cur.init(w, (int32_t)blockIdx.x);
        PagedSegment s;
        int built = -1;  // the KV head whose codebooks are in shared memory
        while (cur.next(a, w, l, s, note)) {
            const int h = s.hx / a.gch, g0 = s.hx % a.gch * a.gc;
            const int gc = a.group - g0 < a.gc ? a.group - g0 : a.gc;
            const int rows = s.it.ntok * gc;
            const int head0 = h * a.group + g0;
            __syncthreads();  // the last segment's slots and images are read
            if (h != built) {  // block-uniform
                // a row of either codebook for each of 256 threads
                static_assert(kFewThreads >= 256, "a codebook row per thread");
                if (tid < 256) {
                    uint32_t k_row[SUB / 2], v_row[SUB / 2];
                    book_row<T, SUB>(static_cast<const T *>(a.kcb) + (int64_t)h * a.nc * SUB, tid, a.nc, static_cast<const T *>(a.kcb), cb_elems, k_row);
                    book_row<T, SUB>(static_cast<const T *>(a.vcb) + (int64_t)h * a.nc * SUB, tid, a.nc, static_cast<const T *>(a.vcb), cb_elems, v_row);
                    image_line<SUB>(k_image, tid, k_row);
                    image_line<SUB>(v_image, tid, v_row);
                }
                built = h;
            }

            // query fragments: row g, columns t dim/4 + 4 i .. + 3
            uint32_t qf[kMma][2];
            const int row = g;
            const T *src = q + (s.it.tok0 + row / gc) * a.q_stride + (int64_t)(head0 + row % gc) * D + t * (D / 4);
            const bool ok = row < rows && VQ_SPAN(src, D / 4, q, q_elems);
#pragma unroll
            for (int i = 0; i < kMma; ++i) {
                uint2 v = make_uint2(0, 0);
                if (ok) {
                    if (q_vec) {
                        v = __ldg(reinterpret_cast<const uint2 *>(src + 4 * i));
                    } else {
                        const uint16_t *e = reinterpret_cast<const uint16_t *>(src + 4 * i);
                        v.x = (uint32_t)__ldg(e) | ((uint32_t)__ldg(e + 1) << 16);
                        v.y = (uint32_t)__ldg(e + 2) | ((uint32_t)__ldg(e + 3) << 16);
                    }
                }
                qf[i][0] = v.x;
                qf[i][1] = v.y;
            }
            // this lane's rows 2 t + c: the last token each sees
            int32_t lim[2];
            float m[2], sum[2];
            float o[kMma][4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 2 * t + c;
                const int32_t p = s.it.pos0 + (row < rows ? row / gc : 0);
                lim[c] = p < s.it.k_hi ? p : s.it.k_hi - 1;
                m[c] = kFewLow;
                sum[c] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < kMma; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
            // positions are lim + window apart from the first token not seen;
            // a row whose limit k_hi cut keeps its own window
            int32_t low[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 2 * t + c;
                const int64_t p = (int64_t)s.it.pos0 + (row < rows ? row / gc : 0) - a.window;
                low[c] = a.window == 0 || p < -1 ? -1 : (int32_t)p;  // tokens above it are seen
            }
            const int32_t all_hi = s.it.pos0 < s.it.k_hi ? s.it.pos0 : s.it.k_hi - 1;  // every row sees up to here
            const int64_t last_pos = (int64_t)s.it.pos0 + s.it.ntok - 1;
            const int64_t all_lo = a.window == 0 ? -1 : last_pos - a.window;       // and above here
            const int64_t none_lo = a.window == 0 ? -1 : (int64_t)s.it.pos0 - a.window;  // no row sees at or below

            // groups of 16 tokens, warp after warp
            const int g_begin = s.begin * (kUnit / 16) + warp, g_end = s.end * (kUnit / 16);
            auto first_of = [&](int group) { return s.it.k_lo + group * 16; };
            auto page_of = [&](int group) -> int32_t {
                if (group >= g_end) return -1;
                const int32_t k0 = first_of(group);
                if (k0 >= s.it.k_hi || k0 + 15 <= none_lo) return -1;
                return paged_entry(a, cur.r, k0);  // checked when it is used: a check here would wait for the load
            };
            auto load = [&](int group, int32_t &pg, uint32_t (&kc)[2][KW], uint32_t (&vc)[4][VW]) {
                if (pg < 0 || pg >= a.num_pages) {  // warp-uniform
                    pg = -1;
                    return;
                }
                const int32_t off = first_of(group) & ((1 << a.page_shift) - 1);
                const int64_t base = (int64_t)pg * a.page_stride + (((int64_t)h << a.page_shift) + off) * NS;
                if (!span_ok(a.k_codes + base, 16 * NS, a.k_codes, code_bytes, NS < 16 ? NS : 16) ||
                    !span_ok(a.v_codes + base, 16 * NS, a.v_codes, code_bytes, NS < 16 ? NS : 16))
                    return;
                const uint8_t *kp = a.k_codes + base + g * NS + t * KB;
                load_codes<KB>(kp, kc[0]);
                load_codes<KB>(kp + 8 * NS, kc[1]);
                const uint8_t *vp = a.v_codes + base + 2 * t * NS + g * VB;
                load_codes<VB>(vp, vc[0]);
                load_codes<VB>(vp + NS, vc[1]);
                load_codes<VB>(vp + 8 * NS, vc[2]);
                load_codes<VB>(vp + 9 * NS, vc[3]);
            };

            // Three sets of registers in turn (X of the unit, X + 2 being loaded): moving
            // a loaded register from set to set would wait for the load.
            uint32_t kc[3][2][KW] = {}, vc[3][4][VW] = {};
            int32_t pg[3];
#pragma unroll
            for (int x = 0; x < 3; ++x) pg[x] = page_of(g_begin + x * kFewWarps);
#pragma unroll
            for (int x = 0; x < 2; ++x) load(g_begin + x * kFewWarps, pg[x], kc[x], vc[x]);
            __syncthreads();  // the images are written

            auto step = [&](auto set, int group) {
                constexpr int X = decltype(set)::value, Y = (X + 2) % 3;
                load(group + 2 * kFewWarps, pg[Y], kc[Y], vc[Y]);
                const bool live = pg[X] >= 0;
                pg[X] = page_of(group + 3 * kFewWarps);
                if (live) {  // warp-uniform
                    // S^T = K^ Q^T
                    float st[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) st[c] = 0.f;
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        uint32_t lo[SUB / 2], hi[SUB / 2];
                        image_row<SUB>(k_base, code_at(kc[X][0], b), lo);
                        image_row<SUB>(k_base, code_at(kc[X][1], b), hi);
#pragma unroll
                        for (int i = 0; i < SUB / 4; ++i)
                            mma16816<T>(st, lo[2 * i], hi[2 * i], lo[2 * i + 1], hi[2 * i + 1],
                                        qf[b * (SUB / 4) + i][0], qf[b * (SUB / 4) + i][1]);
                    }
                    const int32_t k0 = first_of(group);
                    const bool whole = k0 + 15 <= all_hi && k0 > all_lo;
                    bool rise = false;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        st[c] *= a.kappa;
                        if (!whole) {
                            const int32_t key = k0 + g + (c >> 1) * 8;
                            if (key > lim[c & 1] || key <= low[c & 1]) st[c] = kNone;
                        }
                        rise |= st[c] > m[c & 1] + (kFewSlack + kShift);
                    }
                    if (__any_sync(0xffffffffu, rise)) {
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float top = fmaxf(st[c], st[c + 2]);
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                            // a row rises for its own scores alone, so that what it
                            // computes does not depend on the rows beside it
                            const bool up = top > m[c] + (kFewSlack + kShift);
                            const float ref = up ? top - kShift : m[c];
                            const float f = up ? exp2_fast(m[c] - ref) : 1.f;
                            m[c] = ref;
                            sum[c] *= f;
#pragma unroll
                            for (int i = 0; i < kMma; ++i) {
                                o[i][c] *= f;
                                o[i][c + 2] *= f;
                            }
                        }
                    }
                    float p[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        p[c] = exp2_fast(st[c] - m[c & 1]);
                    }
                    sum[0] += p[0] + p[2];
                    sum[1] += p[1] + p[3];
                    // the weights in two pieces of the input type, what the first leaves in
                    // the second: together 22 bits of fp16, 16 of bf16
                    uint32_t pf[2][2];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        const uint32_t high = pack2<T>(p[2 * c], p[2 * c + 1]);
                        const float2 kept = unpack2<T>(high);
                        pf[0][c] = transpose8x8(high);
                        pf[1][c] = transpose8x8(pack2<T>(p[2 * c] - kept.x, p[2 * c + 1] - kept.y));
                    }
                    // O^T += V^^T P^T
#pragma unroll
                    for (int b = 0; b < VB; ++b) {
                        uint32_t e[4][SUB / 2];
#pragma unroll
                        for (int k = 0; k < 4; ++k) image_row<SUB>(v_base, code_at(vc[X][k], b), e[k]);
#pragma unroll
                        for (int i = 0; i < SUB / 2; ++i) {
                            const uint32_t a0 = __byte_perm(e[0][i], e[1][i], 0x5410);
                            const uint32_t a1 = __byte_perm(e[0][i], e[1][i], 0x7632);
                            const uint32_t a2 = __byte_perm(e[2][i], e[3][i], 0x5410);
                            const uint32_t a3 = __byte_perm(e[2][i], e[3][i], 0x7632);
                            mma16816<T>(o[b * (SUB / 2) + i], a0, a1, a2, a3, pf[0][0], pf[0][1]);
                            mma16816<T>(o[b * (SUB / 2) + i], a0, a1, a2, a3, pf[1][0], pf[1][1]);
                        }
                    }
                }
            };
            for (int group = g_begin; group < g_end; group += 3 * kFewWarps) {
                step(std::integral_constant<int, 0>{}, group);
                if (group + kFewWarps < g_end) step(std::integral_constant<int, 1>{}, group + kFewWarps);
                if (group + 2 * kFewWarps < g_end) step(std::integral_constant<int, 2>{}, group + 2 * kFewWarps);
            }

            // the warps' states: maxima and sums first
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 4);
                sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 8);
                sum[c] += __shfl_xor_sync(0xffffffffu, sum[c], 16);
            }
            // A sum of 0: the warp has seen no token of the row, or scores of -inf alone.
            // Its groups are looked through once more for a token that the row sees
            // (here and not in the loop, which has no register to spare; most such rows
            // overlap no group, and nothing is loaded).
            if (__any_sync(0xffffffffu, sum[0] == 0.f || sum[1] == 0.f)) {
                bool saw[2] = {false, false};
                for (int group = g_begin; group < g_end; group += kFewWarps) {
                    const int32_t k0 = first_of(group);
                    bool at[2];
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        at[c] = sum[c] == 0.f && k0 <= lim[c] && k0 + 15 > low[c] && low[c] < lim[c];
                    if (!__any_sync(0xffffffffu, at[0] || at[1])) continue;
                    const int32_t entry = page_of(group);
                    if (entry < 0 || entry >= a.num_pages) continue;
                    saw[0] |= at[0];
                    saw[1] |= at[1];
                }
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    if (saw[c]) {
                        m[c] = kNone;
                        sum[c] = 1.f;
                    }
            }
            if (g == 0) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    wm[warp][2 * t + c] = m[c];
                    wl[warp][2 * t + c] = sum[c];
                }
            }
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = 2 * t + c;
                float top = kNone;
#pragma unroll
                for (int k = 0; k < kFewWarps; ++k)
                    if (wl[k][row] != 0.f) top = fmaxf(top, wm[k][row]);
                float total = 0.f;
#pragma unroll
                for (int k = 0; k < kFewWarps; ++k)
                    if (wl[k][row] != 0.f) total = fmaf(exp2_fast(wm[k][row] - top), wl[k][row], total);
                if (top == kNone && total != 0.f) total = 1.f;
                const float f = sum[c] == 0.f || m[c] == kNone ? 0.f : exp2_fast(m[c] - top);
                m[c] = top;
                sum[c] = total;
#pragma unroll
                for (int i = 0; i < kMma; ++i) {
                    o[i][c] *= f;
                    o[i][c + 2] *= f;
                }
            }
            // then the weighted sums: the upper half of the warps to the lower, until one is left
#pragma unroll
            for (int live = kFewWarps; live > 1; live = (live + 1) / 2) {
                const int half = (live + 1) / 2;  // warps half .. live - 1 give to warps 0 ..
                float4 *slot = reinterpret_cast<float4 *>(slots) + (int64_t)(warp < half ? warp : warp - half) * kMma * 32 + lane;
                if (warp >= half && warp < live) {
#pragma unroll
                    for (int i = 0; i < kMma; ++i)
                        if (dyn_smem_ok(slot + i * 32, 16, 16))
                            slot[i * 32] = make_float4(o[i][0], o[i][1], o[i][2], o[i][3]);
                }
                __syncthreads();
                if (warp < live - half) {
#pragma unroll
                    for (int i = 0; i < kMma; ++i)
                        if (dyn_smem_ok(slot + i * 32, 16, 16)) {
                            const float4 v = slot[i * 32];
                            o[i][0] += v.x;
                            o[i][1] += v.y;
                            o[i][2] += v.z;
                            o[i][3] += v.w;
                        }
                }
                __syncthreads();
            }
            if (warp == 0) {
                // lane (g, t) holds columns [g dim/8, (g+1) dim/8) of rows 2 t + c
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int row = 2 * t + c;
                    if (row >= rows) continue;
                    if (s.whole) {
                        const int64_t orow = (s.it.tok0 + row / gc) * a.hq + head0 + row % gc;
                        const float inv = paged_inv(m[c], sum[c]);
                        T *dst = out + orow * D + g * (D / 8);
                        if (VQ_SPAN(dst, D / 8, out, a.tokens * a.hq * D)) {
                            if (out_vec) {
#pragma unroll
                                for (int i = 0; i < kMma; i += 4) {
                                    uint32_t v[4];
#pragma unroll
                                    for (int x = 0; x < 4; ++x)
                                        v[x] = pack2<T>(o[i + x][c] * inv, o[i + x][c + 2] * inv);
                                    reinterpret_cast<uint4 *>(dst)[i / 4] = make_uint4(v[0], v[1], v[2], v[3]);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < kMma; ++i) {
                                    dst[2 * i] = narrow<T>(o[i][c] * inv);
                                    dst[2 * i + 1] = narrow<T>(o[i][c + 2] * inv);
                                }
                            }
                        }
                        if (g == 0 && a.lse && VQ_SPAN(a.lse + orow, 1, a.lse, a.tokens * a.hq))
                            a.lse[orow] = paged_lse(m[c], sum[c]);
                    } else {
                        const int64_t prow = s.slot * a.tile_rows + row, prows = 2 * (int64_t)gridDim.x * a.tile_rows;
                        float *dst = a.part + prow * D + g * (D / 8);
                        if (VQ_VSPAN(dst, D / 8, a.part, prows * D, 16)) {
#pragma unroll
                            for (int i = 0; i < kMma; i += 2)
                                reinterpret_cast<float4 *>(dst)[i / 2] =
                                    make_float4(o[i][c], o[i][c + 2], o[i + 1][c], o[i + 1][c + 2]);
                        }
                        if (g == 0 && VQ_SPAN(a.ml + prow * 2, 2, a.ml, prows * 2)) {
                            a.ml[prow * 2] = m[c];
                            a.ml[prow * 2 + 1] = sum[c];
                        }
                    }
                }
            }
        }
    }
    if (tid == 0 && VQ_SPAN(a.notes + blockIdx.x, 1, a.notes, gridDim.x)) a.notes[blockIdx.x] = note;
}

}  // namespace vqk
