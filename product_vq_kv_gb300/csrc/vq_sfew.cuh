// vq_sfew.cuh -- paged attention of a few rows (decode, verification of drafts) over 4-bit
// scalar codes: up to 8 rows (tokens x query heads of one KV head) against the whole
// cache, 16-bit types, head sizes 64, 128 and 256.
//
// The frame is that of the few-row kernel of product-VQ codes (vq_pfew.cuh): S^T = K^ Q^T
// and O^T = V^^T P^T by mma.m16n8k16 with the query rows as its 8 columns, a warp a group of
// 16 tokens, rebuilt values in the registers of the instruction that uses them, weights in
// two pieces.  What differs is the rebuild.
//
// What bounds it.  From HBM a cached token costs dim + 4 bytes a KV head, 132 at dim 128:
// 5.8 cycles of an SM's share at 6.78 TB/s and 1.9 GHz.  Rebuilding its 2 dim values from
// pairs of codes is 128 lookups, 4 warp instructions and 4 cycles of shared memory if each
// lookup of a warp takes one; beside them stand the address of each lookup, 24 matrix
// instructions per 16 tokens and the softmax, about 5 cycles of issue.  So all three are
// close, and the kernel is laid out to issue little.  (As measured no unit is full: 16 x 32768 tokens at
// dim 128 in fp16 take 142 us, 3.9 TB/s, at 61 % of the issue slots, 22 % of the tensor pipe and a third
// of the shared-memory port.  Of 359 warp instructions per 16 tokens 128 are the lookups and their
// addresses; three warps a scheduler wait first for fixed latencies.)
//   * A table of 256 lines, one per byte, holds the pair (c[low half], c[high half]) as one
//     32-bit word 32 times, a copy for each lane in its own bank: no lookup conflicts.  A line
//     is 256 bytes, the keys' copies then the values', and the table lies at a fixed address of
//     shared memory, so that one byte permute of the code word and a lane's constant (byte << 8 |
//     4 lane) is the whole address but for the load's offset.
//   * Keys: a byte's two codes are neighbouring columns of a key, one operand register.
//     The scale multiplies the score, in fp32.
//   * Values: an operand register takes one column of two tokens.  The nibbles of two
//     tokens' words are exchanged (a shift and a select a word), so that a byte holds the two
//     tokens' codes of one column.  The values' scales multiply the weights, in fp32 and
//     before their rounding to two pieces, so that no rebuilt value is rounded.
//   * A warp takes 32 tokens at a time, so that addresses, page lookups, waits and the vote
//     are paid once and the two groups' chains of dependent instructions overlap.
//   * Up to 4 rows (one token of up to 4 query heads a KV head) leave half of an instruction's
//     columns free: there the rows stand twice, and the second pieces of the weights take the
//     columns that would be idle, one instruction instead of two (32 uneven decodes at dim 128: 159 -> 157 us; heads of 64 120
//     -> 116).
//   * Codes and scales come by cp.async into two slots a warp, 16-byte pieces exchanged so
//     that the keys' and the values' reads meet no bank twice; a slot is filled again as
//     soon as its codes are in registers, two runs ahead of their use.
#pragma once

#include "vq_pfew.cuh"
#include "vq_sattn.cuh"
#include "vq_umma.cuh"

namespace vqk {

template <int D>
struct SFewShape {
    // One block an SM, with as many warps as leave the accumulators and queries (dim/16 x 6
    // registers) and a run's codes in registers.
    static constexpr int kWarps = D == 64 ? 16 : D == 128 ? 12 : 8;
    static constexpr int kHalves = 2;             // groups of 16 tokens that a warp takes at a time: a run
    static constexpr int kRun = 16 * kHalves;
    static constexpr int kSlots = 2;              // of a warp, a run each
    static constexpr int kCodes = 16 * (D / 2);   // code bytes of a group, keys or values
    static constexpr int kValues = kHalves * kCodes, kScales = 2 * kValues;  // in a slot: keys, values, scales
    static constexpr int kSlot = kScales + kHalves * 64;
    static constexpr int kWarpRing = kSlots * kSlot;
    static constexpr size_t kMerge = (size_t)((kWarps + 1) / 2) * kFewRows * D * sizeof(float);  // over the upper ring
    // Addresses in shared memory: static memory, the ring of the first kLow warps from kRing,
    // the table from kTable, the other warps' ring from kUpper.
    static constexpr uint32_t kTable = 65536, kUpper = kTable + 65536;
    static constexpr uint32_t kRing = D == 64 ? 18432 : 15360;
    static constexpr int kLow = (kTable - kRing) / kWarpRing < kWarps ? (kTable - kRing) / kWarpRing : kWarps;
    static constexpr size_t kAbove = (size_t)(kWarps - kLow) * kWarpRing;
    static constexpr size_t kSmem = kUpper + (kAbove > kMerge ? kAbove : kMerge);  // (of which the array has the part from its start on)
};

// Where byte `at` of a group's codes lies in its slot: of each 128 bytes the 16-byte pieces
// change places.  A warp reads keys row by row and values two rows apart, and with this
// neither meets a bank twice in one pass.  Rows 8 apart change alike.
template <int D>
__device__ __forceinline__ uint32_t sfew_place(uint32_t at)
{
    const uint32_t line = at >> 7, turn = D == 256 ? line & 7 : D == 128 ? 2 * (line & 3) : 2 * (line & 1);
    return at ^ (turn << 4);
}

// A row's state beside its maximum m and its sum of p = 2^(score - m): what the weights
// p s_v of the second product are multiplied by.  It starts at its most and falls when a
// weight's magnitude passes kSFewTop; a rise of m lifts it by as much, so that the accumulators stay as
// they are.
constexpr float kSFewMost = 1.2676506e30f;   // 2^100
constexpr float kSFewTop = 32768.f;          // the largest weight: 2^15, inside fp16
constexpr float kSFewLess = 7.6293945e-6f;   // 2^-17: p, which stays fp32, may reach 2^32

// The scores of H groups of 16 tokens against this lane's two rows to weights, as
// few_weights does it, but the product takes p s_v, the scale of the token's value (vs: of
// tokens g and g + 8) folded in.  m follows the scores alone and the factor f the weights alone: a value's scale
// does not touch the sum, and tokens whose values are large do not push others, of larger
// weight, out of fp16.
// PAIR: this lane's columns hold the first or (`second`) the second piece of their weights.
template <typename T, bool PAIR, int H, int MMA>
__device__ __forceinline__ void sfew_weights(const float (&st)[H][4], const float (&vs)[H][2], bool second, float (&m)[2],
                                             float (&sum)[2], float (&f)[2], float (&o)[MMA][4], uint32_t (&pf)[H][PAIR ? 1 : 2][2])
{
    float p[H][4], w[H][4], high = 0.f;
#pragma unroll
    for (int h = 0; h < H; ++h)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            p[h][c] = exp2_fast(st[h][c] - m[c & 1]);
            w[h][c] = p[h][c] * vs[h][c >> 1] * f[c & 1];
            high = max3(high, p[h][c] * kSFewLess, fabsf(w[h][c]));
        }
    if (__any_sync(0xffffffffu, high > kSFewTop)) {
        // a row rises for its own scores and weights alone, so that what it computes does not
        // depend on the rows beside it
        auto over_lanes = [](float v) {
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 4));
            v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 8));
            return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 16));
        };
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float top = __int_as_float(0xff800000);
#pragma unroll
            for (int h = 0; h < H; ++h) top = fmaxf(top, fmaxf(st[h][c], st[h][c + 2]));
            top = over_lanes(top);
            float scale = 1.f;  // of the accumulators
            // for its scores, or for a weight whose product with the value's scale passes fp32's
            // largest (against the largest score none does)
            bool past = false;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = c; k < 4; k += 2) past |= !(p[h][k] * fabsf(vs[h][k >> 1]) <= 3.402823466e38f);
            past = (__ballot_sync(0xffffffffu, past) & (0x11111111u << (threadIdx.x & 3))) != 0;  // the row's lanes
            if (past || exp2_fast(top - m[c]) * kSFewLess > kSFewTop) {
                const float to = f[c] * exp2_fast(top - m[c]);
                f[c] = fminf(to, kSFewMost);
                scale = f[c] / to;  // (0 where `to` is infinite: what was is nothing beside it)
                sum[c] *= exp2_fast(m[c] - top);
                m[c] = top;
            }
            float most = 0.f;
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = c; k < 4; k += 2) {
                    p[h][k] = exp2_fast(st[h][k] - m[c]);
                    most = fmaxf(most, p[h][k] * fabsf(vs[h][k >> 1]));
                }
            most = over_lanes(most);
            if (most * f[c] > kSFewTop) {
                // the power of two that brings it to [2^6, 2^7): most >= 2^-85 here
                const uint32_t e = __float_as_uint(most) >> 23;
                const float to = __uint_as_float((uint32_t)(127 + 6 + 127 - (int)(e > 250u ? 250u : e)) << 23);
                scale *= to / f[c];
                f[c] = to;
            }
#pragma unroll
            for (int h = 0; h < H; ++h)
#pragma unroll
                for (int k = c; k < 4; k += 2) w[h][k] = p[h][k] * vs[h][k >> 1] * f[c];
#pragma unroll
            for (int i = 0; i < MMA; ++i) {
                o[i][c] *= scale;
                o[i][c + 2] *= scale;
            }
        }
    }
#pragma unroll
    for (int h = 0; h < H; ++h) {
        sum[0] += p[h][0] + p[h][2];
        sum[1] += p[h][1] + p[h][3];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const uint32_t first = pack2<T>(w[h][2 * c], w[h][2 * c + 1]);
            const float2 kept = unpack2<T>(first);
            const uint32_t rest = pack2<T>(w[h][2 * c] - kept.x, w[h][2 * c + 1] - kept.y);
            pf[h][0][c] = transpose8x8(PAIR && second ? rest : first);
            if constexpr (!PAIR) pf[h][1][c] = transpose8x8(rest);
        }
    }
}

template <int OFF, int FROM>
__device__ __forceinline__ void copy_async16(uint32_t to, const void *from)
{
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(to), "l"(from), "n"(OFF), "n"(FROM) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int PENDING>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(PENDING) : "memory");
    __syncwarp();
}

// W words of codes at address `at` + OFF (of two 16-byte pieces the second at `next` + OFF).
// Not moved across the waits and fetches around them, which are volatile too.
template <int W, int OFF>
__device__ __forceinline__ void load_shared(uint32_t at, uint32_t next, uint32_t (&v)[W])
{
    if constexpr (W == 1) asm volatile("ld.shared.b32 %0, [%1 + %2];" : "=r"(v[0]) : "r"(at), "n"(OFF) : "memory");
    if constexpr (W == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2 + %3];" : "=r"(v[0]), "=r"(v[1]) : "r"(at), "n"(OFF) : "memory");
    if constexpr (W >= 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(at), "n"(OFF)
                     : "memory");
    if constexpr (W == 8)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4 + %5];"
                     : "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(next), "n"(OFF)
                     : "memory");
}

template <typename T, int OFF>
__device__ __forceinline__ float load_shared16(uint32_t at)
{
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1 + %2];" : "=h"(v) : "r"(at), "n"(OFF) : "memory");
    if constexpr (std::is_same<T, __half>::value) return __half2float(__ushort_as_half(v));
    else return __uint_as_float((uint32_t)v << 16);
}

// f(0), .., f(N - 1) with the numbers as constants.
template <int N, typename F>
__device__ __forceinline__ void each(F f)
{
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// PAIR: items of up to 4 rows, which lie in columns 0 to 3 of the instructions and once more in
// 4 to 7; there the weights' second pieces enter the second product.
template <typename T, int D, bool PAIR>
__global__ void __launch_bounds__(SFewShape<D>::kWarps * 32, 1)
    paged_attn_sfew(const __grid_constant__ PagedArgs a)
{
    using S = SFewShape<D>;
    constexpr int kWarps = S::kWarps, kThreads = kWarps * 32;
    constexpr int NS = D / 2;
    constexpr int KB = NS / 4, VB = NS / 8;      // code bytes a lane takes of a key, of a value
    constexpr int KW = KB / 4, VW = VB / 4;
    constexpr int kMma = D / 16;                 // instructions per 16 tokens and 8 rows, each product
    extern __shared__ __align__(128) unsigned char sfew_mem[];
    __shared__ PagedWalk<> w;
    __shared__ float wm[kWarps][kFewRows], wl[kWarps][kFewRows];
    __shared__ int32_t batch[kWarps][2][S::kHalves][32];
    static_assert(1024 + sizeof w + sizeof wm + sizeof wl + sizeof batch + 256 <= S::kRing, "static memory (and the system's) below the ring");
    // (the array begins behind the static memory, which ends below kRing)
    unsigned char *lines = sfew_mem + (S::kTable - smem_addr(sfew_mem));
    float *slots = reinterpret_cast<float *>(lines + (S::kUpper - S::kTable));

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const float kNone = __int_as_float(0xff800000);
    const uint32_t copy[2] = {(uint32_t)lane * 4, (uint32_t)lane * 4 + 128};  // this lane's copies in a line
    const T *__restrict__ q = static_cast<const T *>(a.q);
    const unsigned char *ks = static_cast<const unsigned char *>(a.k_scales), *vs = static_cast<const unsigned char *>(a.v_scales);
    const bool q_vec = (uintptr_t)a.q % 8 == 0 && a.q_stride % 4 == 0;
    const bool out_vec = (uintptr_t)a.out % 16 == 0;
    const int64_t q_elems = (a.tokens - 1) * a.q_stride + (int64_t)a.hq * D;
    const int64_t code_bytes = (a.num_pages - 1) * a.page_stride + (((int64_t)a.hkv * NS) << a.page_shift);
    const int64_t scale_bytes = 2 * ((a.num_pages - 1) * a.scale_stride + ((int64_t)a.hkv << a.page_shift));
    const uint32_t ring = warp < S::kLow ? S::kRing + warp * S::kWarpRing : S::kUpper + (warp - S::kLow) * S::kWarpRing;
    // where this lane puts and finds codes in a slot
    const uint32_t put_at = sfew_place<D>(lane * 16);
    const uint32_t k_at = sfew_place<D>(g * NS + t * KB), v_at[2] = {sfew_place<D>(2 * t * NS + g * VB), sfew_place<D>((2 * t + 1) * NS + g * VB)};

    // the merge's blocks may take the room that idle blocks leave (they wait there)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    PagedLens l;
    PagedNote note{};
    if (paged_plan<kThreads>(a, w, l)) {
        PagedCursor cur;
        cur.init(w, (int32_t)blockIdx.x);
        PagedSegment s;
        scalar_lines<T>(a.k_cent, a.nc, 0, lines, tid, kThreads);
        scalar_lines<T>(a.v_cent, a.nc, 1, lines, tid, kThreads);
        while (cur.next(a, w, l, s, note)) {
            const int h = s.hx / a.gch, g0 = s.hx % a.gch * a.gc;
            const int gc = a.group - g0 < a.gc ? a.group - g0 : a.gc;
            const int rows = s.it.ntok * gc;
            const int head0 = h * a.group + g0;

            // query fragments: row g, columns t dim/4 + 4 i .. + 3
            uint32_t qf[kMma][2];
            const int row = PAIR ? g & 3 : g;
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
            // this lane's rows 2 t + c: the tokens in (low, lim] are seen
            int32_t lim[2], low[2];
            float m[2], sum[2], factor[2];
            float o[kMma][4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int row = PAIR ? (2 * t + c) & 3 : 2 * t + c;
                const int32_t p = s.it.pos0 + (row < rows ? row / gc : 0);
                lim[c] = p < s.it.k_hi ? p : s.it.k_hi - 1;
                // (a row whose limit k_hi cut keeps its own window)
                const int64_t from = (int64_t)p - a.window;
                low[c] = a.window == 0 || from < -1 ? -1 : (int32_t)from;
                m[c] = kFewLow;
                sum[c] = 0.f;
                factor[c] = kSFewMost;
            }
#pragma unroll
            for (int i = 0; i < kMma; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
            const int32_t all_hi = s.it.pos0 < s.it.k_hi ? s.it.pos0 : s.it.k_hi - 1;  // every row sees up to here
            const int64_t last_pos = (int64_t)s.it.pos0 + s.it.ntok - 1;
            const int64_t all_lo = a.window == 0 ? -1 : last_pos - a.window;       // and above here
            const int64_t none_lo = a.window == 0 ? -1 : (int64_t)s.it.pos0 - a.window;  // no row sees at or below

            // runs of 32 tokens, warp after warp
            const int g_begin = s.begin * (kUnit / S::kRun) + warp, g_end = s.end * (kUnit / S::kRun);
            auto first_of = [&](int run) { return s.it.k_lo + run * S::kRun; };
            auto entry_of = [&](int32_t k0) -> int32_t {  // the page of 16 tokens
                if (k0 >= s.it.k_hi || k0 + 15 <= none_lo) return -1;
                return paged_entry(a, cur.r, k0);  // checked when it is used: a check here would wait for the load
            };
            // The pages of 32 runs of this warp, a run a lane, kept in shared memory one batch ahead
            // of their use: a load for each run would be waited for where its register is handed
            // on.
            struct Pages { int32_t pg[S::kHalves]; };
            auto keep_batch = [&](int b) {  // runs 32 b .. of this warp
                const int run = g_begin + (32 * b + lane) * kWarps;
                __syncwarp();  // the batch that was there is read
#pragma unroll
                for (int x = 0; x < S::kHalves; ++x) batch[warp][b & 1][x][lane] = run < g_end ? entry_of(first_of(run) + 16 * x) : -1;
                __syncwarp();
            };
            keep_batch(0);
            keep_batch(1);
            auto pages_of = [&](int n) {  // of this warp's n-th run
                Pages p;
#pragma unroll
                for (int x = 0; x < S::kHalves; ++x) p.pg[x] = batch[warp][n >> 5 & 1][x][n & 31];
                return p;
            };
            auto is_page = [&](int32_t pg) { return pg >= 0 && pg < a.num_pages; };
            // this head's rows of page 0; of 4 lanes two fetch the keys' scales, two the values'
            const int64_t head = (int64_t)h << a.page_shift;
            const uint8_t *k_head = a.k_codes + head * NS + lane * 16, *v_head = a.v_codes + head * NS + lane * 16;
            const unsigned char *s_head = (lane % 4 < 2 ? ks : vs) + 2 * head + (lane & 1) * 16;
            // a run on its way into a slot: the keys and both scales, or the values
            struct Places { int64_t at[S::kHalves]; bool is[S::kHalves]; };
            auto places_of = [&](int run, const Pages &p) {
                Places to;
#pragma unroll
                for (int x = 0; x < S::kHalves; ++x) {
                    const int32_t row = (first_of(run) + 16 * x) & ((1 << a.page_shift) - 1);
                    to.is[x] = is_page(p.pg[x]);  // warp-uniform
                    to.at[x] = (int64_t)p.pg[x] * a.page_stride + row * NS;
                }
                return to;
            };
            auto fetch_keys = [&](int run, const Pages &p, const Places &from, uint32_t slot) {
                each<S::kHalves>([&](auto half) {
                    constexpr int X = decltype(half)::value;
                    if (!from.is[X]) return;
                    each<S::kCodes / 512>([&](auto piece) {
                        constexpr int I = decltype(piece)::value;
                        if (span_ok(k_head + from.at[X] + I * 512, 16, a.k_codes, code_bytes, 16))
                            copy_async16<X * S::kCodes + I * 512, I * 512>(slot + (D == 256 && I % 2 ? put_at ^ 64 : put_at), k_head + from.at[X]);
                    });
                    if (lane / 4 == X) {
                        const int32_t row = (first_of(run) + 16 * X) & ((1 << a.page_shift) - 1);
                        const unsigned char *scale = s_head + 2 * ((int64_t)p.pg[X] * a.scale_stride + row);
                        if (span_ok(scale, 16, lane % 4 < 2 ? ks : vs, scale_bytes, 16)) copy_async16<S::kScales, 0>(slot + lane * 16, scale);
                    }
                });
                copy_commit();  // (an empty group keeps the count)
            };
            auto fetch_values = [&](const Places &from, uint32_t slot) {
                each<S::kHalves>([&](auto half) {
                    constexpr int X = decltype(half)::value;
                    if (!from.is[X]) return;
                    each<S::kCodes / 512>([&](auto piece) {
                        constexpr int I = decltype(piece)::value;
                        if (span_ok(v_head + from.at[X] + I * 512, 16, a.v_codes, code_bytes, 16))
                            copy_async16<S::kValues + X * S::kCodes + I * 512, I * 512>(slot + (D == 256 && I % 2 ? put_at ^ 64 : put_at),
                                                                                        v_head + from.at[X]);
                    });
                });
                copy_commit();
            };
            Pages pages[S::kSlots];
#pragma unroll
            for (int x = 0; x < S::kSlots; ++x) pages[x] = pages_of(x);
            __syncthreads();  // the table is written, the last segment's merge has left the ring
#pragma unroll
            for (int x = 0; x < S::kSlots; ++x) {
                const Places from = places_of(g_begin + x * kWarps, pages[x]);
                fetch_keys(g_begin + x * kWarps, pages[x], from, ring + x * S::kSlot);
                fetch_values(from, ring + x * S::kSlot);
            }

            auto table = [&](uint32_t word, int i, int kind) { return scalar_lookup<S::kTable>(word, i, copy[kind]); };
            uint32_t slot = ring;
            int n = 0;  // of the warp's runs
            for (int run = g_begin; run < g_end; run += kWarps) {
                const Pages ahead = pages_of(n + S::kSlots);
                const Places from = places_of(run + S::kSlots * kWarps, ahead);
                bool live[S::kHalves], any = false, both = true;  // warp-uniform
#pragma unroll
                for (int x = 0; x < S::kHalves; ++x) {
                    live[x] = is_page(pages[0].pg[x]);
                    any |= live[x];
                    both &= live[x];
                }
#pragma unroll
                for (int x = 0; x + 1 < S::kSlots; ++x) pages[x] = pages[x + 1];
                pages[S::kSlots - 1] = ahead;
                copy_wait<2 * S::kSlots - 1>();  // this run's keys, and both its scales
                if (any) {
                    uint32_t kc[S::kHalves][2][KW];
                    float kscale[S::kHalves][2], vscale[S::kHalves][2];
                    each<2 * S::kHalves>([&](auto at) {
                        constexpr int X = decltype(at)::value / 2, K = decltype(at)::value % 2;
                        constexpr int kOff = X * S::kCodes + 8 * K * NS;  // (rows 8 apart lie alike)
                        load_shared<KW, kOff>(slot + k_at, slot + (k_at ^ 16), kc[X][K]);
                        kscale[X][K] = a.kappa * load_shared16<T, S::kScales + 64 * X + 16 * K>(slot + 2 * g);
                        vscale[X][K] = load_shared16<T, S::kScales + 64 * X + 32 + 16 * K>(slot + 2 * g);
                    });
                    __syncwarp();
                    fetch_keys(run + S::kSlots * kWarps, ahead, from, slot);
                    const int32_t k0 = first_of(run);
                    // S^T = K^ Q^T
                    float st[S::kHalves][4];
#pragma unroll
                    for (int x = 0; x < S::kHalves; ++x)
#pragma unroll
                        for (int c = 0; c < 4; ++c) st[x][c] = 0.f;
#pragma unroll
                    for (int b = 0; b < KB; b += 2)
#pragma unroll
                        for (int x = 0; x < S::kHalves; ++x) {
                            const uint32_t a0 = table(kc[x][0][b / 4], b % 4, 0), a1 = table(kc[x][1][b / 4], b % 4, 0);
                            const uint32_t a2 = table(kc[x][0][b / 4], b % 4 + 1, 0), a3 = table(kc[x][1][b / 4], b % 4 + 1, 0);
                            mma16816<T>(st[x], a0, a1, a2, a3, qf[b / 2][0], qf[b / 2][1]);
                        }
#pragma unroll
                    for (int x = 0; x < S::kHalves; ++x)
#pragma unroll
                        for (int c = 0; c < 4; ++c) st[x][c] *= kscale[x][c >> 1];
                    if (!(both && k0 + S::kRun - 1 <= all_hi && k0 > all_lo)) {
#pragma unroll
                        for (int x = 0; x < S::kHalves; ++x)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const int32_t key = k0 + 16 * x + g + 8 * k;
#pragma unroll
                                for (int c = 0; c < 2; ++c)
                                    if (!live[x] || key > lim[c] || key <= low[c]) st[x][2 * k + c] = kNone;
                                // tokens that no row sees weigh nothing, whatever their scales hold
                                if (!live[x] || key >= s.it.k_hi || key > last_pos || key <= none_lo) vscale[x][k] = 0.f;
                            }
                    }
                    uint32_t pf[S::kHalves][PAIR ? 1 : 2][2];
                    sfew_weights<T, PAIR>(st, vscale, t >= 2, m, sum, factor, o, pf);
                    copy_wait<2 * S::kSlots - 1>();  // its values
                    uint32_t vc[S::kHalves][4][VW];
                    each<4 * S::kHalves>([&](auto at) {
                        constexpr int X = decltype(at)::value / 4, K = decltype(at)::value % 4;
                        load_shared<VW, S::kValues + X * S::kCodes + 8 * (K / 2) * NS>(slot + v_at[K % 2], 0, vc[X][K]);
                    });
                    __syncwarp();
                    fetch_values(from, slot);
                    // O^T += V^^T P^T
#pragma unroll
                    for (int i = 0; i < VW; ++i)
#pragma unroll
                        for (int x = 0; x < S::kHalves; ++x) {
                            constexpr uint32_t kLow = 0x0f0f0f0fu;
                            uint32_t even[2], odd[2];  // of columns 2 b and 2 b + 1, two tokens a byte
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                const uint32_t v0 = vc[x][2 * k][i], v1 = vc[x][2 * k + 1][i];
                                even[k] = (v0 & kLow) | (v1 << 4 & ~kLow);
                                odd[k] = (v0 >> 4 & kLow) | (v1 & ~kLow);
                            }
#pragma unroll
                            for (int b = 0; b < 4; ++b) {
                                const uint32_t a0 = table(even[0], b, 1), a1 = table(odd[0], b, 1);
                                const uint32_t a2 = table(even[1], b, 1), a3 = table(odd[1], b, 1);
                                mma16816<T>(o[4 * i + b], a0, a1, a2, a3, pf[x][0][0], pf[x][0][1]);
                                if constexpr (!PAIR) mma16816<T>(o[4 * i + b], a0, a1, a2, a3, pf[x][1][0], pf[x][1][1]);
                            }
                        }
                } else {
                    fetch_keys(run + S::kSlots * kWarps, ahead, from, slot);
                    copy_wait<2 * S::kSlots - 1>();
                    fetch_values(from, slot);
                }
                static_assert(S::kSlots == 2, "two slots in turn");
                slot = slot == ring ? ring + S::kSlot : ring;
                if ((++n & 31) == 0) keep_batch((n >> 5) + 1);
            }
            copy_wait<0>();
            if constexpr (PAIR) {  // the two pieces' sums
#pragma unroll
                for (int i = 0; i < kMma; ++i)
#pragma unroll
                    for (int c = 0; c < 4; ++c) o[i][c] += __shfl_xor_sync(0xffffffffu, o[i][c], 2);
            }
            // to weights without the factors, and no larger than 1 (a maximum may have lagged): by
            // powers of two, so that sums of large values stay in fp32 where values do
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float all = sum[c];
                all += __shfl_xor_sync(0xffffffffu, all, 4);
                all += __shfl_xor_sync(0xffffffffu, all, 8);
                all += __shfl_xor_sync(0xffffffffu, all, 16);
                const int lag = all > 1.f && all <= 3.402823466e38f ? (int)(__float_as_uint(all) >> 23) - 127 : 0;
                const float less = __uint_as_float((uint32_t)(127 - lag) << 23), inv = 1.f / factor[c];
                m[c] += (float)lag;
                sum[c] *= less;
#pragma unroll
                for (int i = 0; i < kMma; ++i) {
                    o[i][c] = o[i][c] * less * inv;
                    o[i][c + 2] = o[i][c + 2] * less * inv;
                }
            }
            // (what it looks through for tokens that rows see: this warp's groups of 16)
            few_finish<T, D, kWarps>(a, s, rows, gc, head0, lim, low, m, sum, o, wm, wl, slots, out_vec, s.begin * (kUnit / 16) + warp,
                                     s.end * (kUnit / 16), [&](int group) { return s.it.k_lo + group * 16; },
                                     [&](int group) { return entry_of(s.it.k_lo + group * 16); });
        }
    }
    if (tid == 0 && VQ_SPAN(a.notes + blockIdx.x, 1, a.notes, gridDim.x)) a.notes[blockIdx.x] = note;
}

}  // namespace vqk
