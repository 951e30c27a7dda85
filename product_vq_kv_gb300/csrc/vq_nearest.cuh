// vq_nearest.cuh -- the nearest-centroid rule of the scalar codes,
//   idx = argmin_j fl(fl(v - c_j)^2), strict "<" over ascending j from (+inf, 0),
// by a scan and by cut points, and loads of rows as fp32: what the scalar encoders
// (vq_scalar.cuh) and the append of scalar codes (vq_sappend.cuh) share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

namespace vqs {

__device__ __forceinline__ float widen16(uint16_t bits, bool bf16)
{
    return bf16 ? __uint_as_float((uint32_t)bits << 16) : __half2float(__ushort_as_half(bits));
}
__device__ __forceinline__ float widen_elem(float v) { return v; }
__device__ __forceinline__ float widen_elem(__half v) { return __half2float(v); }
__device__ __forceinline__ float widen_elem(__nv_bfloat16 v) { return __bfloat162float(v); }

// The nearest-centroid rule for one fp32 value, codebook c[0..n_c) in shared
// memory (every lane reads the same entry: broadcast).
__device__ __forceinline__ uint32_t nearest(float val, const float *c, int n_c)
{
    float best_dist = __int_as_float(0x7f800000);
    uint32_t best = 0;
    for (int j = 0; j < n_c; ++j) {
        const float d = __fsub_rn(val, c[j]);
        const float dist = __fmul_rn(d, d);
        if (dist < best_dist) {
            best_dist = dist;
            best = (uint32_t)j;
        }
    }
    return best;
}

// E consecutive elements of one row as fp32 (vector loads where E and the
// element size allow; rows are E-element aligned).
template <typename T, int E>
__device__ __forceinline__ void load_run(const T *p, float (&v)[E])
{
    constexpr int kBytes = E * (int)sizeof(T);
    if constexpr (kBytes >= 16 && kBytes % 16 == 0) {
        constexpr int kPer = 16 / (int)sizeof(T);
#pragma unroll
        for (int k = 0; k < E / kPer; ++k) {
            const uint4 q = __ldcs(reinterpret_cast<const uint4 *>(p) + k);
            const T *t = reinterpret_cast<const T *>(&q);
#pragma unroll
            for (int i = 0; i < kPer; ++i) v[k * kPer + i] = widen_elem(t[i]);
        }
    } else if constexpr (kBytes == 8) {
        const uint2 q = __ldcs(reinterpret_cast<const uint2 *>(p));
        const T *t = reinterpret_cast<const T *>(&q);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = widen_elem(t[i]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = widen_elem(p[i]);
    }
}

// ---- exact nearest centroid of NC distinct centroids by cut points
//
// Let s_0 < ... < s_{NC-1} be the centroids sorted, orig(k) the original
// index of s_k, and d_j(v) = fl(fl(v - s_j)^2) the rule's distance.  On
// [s_k, s_{k+1}] d_k never decreases and d_{k+1} never increases as v grows,
// so "s_{k+1} beats s_k under the rule" (d_{k+1} < d_k, or d_{k+1} <= d_k when
// orig(k+1) < orig(k): ties go to the lower original index) is false at s_k,
// true at s_{k+1} and monotone in between.  Its first fp32 value t_k, found by
// a binary search over the bit patterns of that interval, is the cut point of
// the pair.  For lo <= v <= hi, k = #{j : t_j <= v} and the answer is
// orig(k): s_k beats or ties-and-wins against its two neighbours by the cut
// points, and every farther centroid is strictly farther than the
// neighbour between them, because the set-up only accepts codebooks whose
// neighbouring gaps differ by at most 2^15, whose gaps are at least 2^-40 and
// whose span [lo, hi] (the centroids widened by 2^15 outer gaps) stays below
// 2^62: a distance ratio of at least 1 + 2^-16 then survives the two
// roundings, with no underflow or overflow.  Values outside [lo, hi], NaN,
// and codebooks that fail those conditions take the rule's scan.
template <int NC>
struct CutCb {
    const float *t;   // [NC - 1] cut points, ascending, in shared memory
    float lo, hi;     // the values they decide
    uint64_t perm;    // orig(k) in bits 4k .. 4k + 3
    bool ok;          // the cut points apply (false: the scan for everything)
};

// Total order of the fp32 values as unsigned keys (finite values; -0 just
// below +0), and back.
__device__ __forceinline__ uint32_t f32_key(float f)
{
    const uint32_t u = __float_as_uint(f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float f32_from_key(uint32_t k)
{
    return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Block set-up (every thread of the block calls it; three block barriers).
// `sm` is shared memory for 4 NC floats; on return sm[NC .. 2 NC) holds the
// codebook as given, for the rule's scan.  Thread i < NC ranks centroid i;
// thread k < NC - 1 checks the gaps around pair (k, k + 1) and searches its
// cut point; every thread then reads the result.
template <int NC>
__device__ __forceinline__ void build_cut_cb(const float *__restrict__ centroids, float *sm,
                                             CutCb<NC> &cb)
{
    static_assert(NC >= 2 && NC <= 16, "4-bit original indices");
    float *srt = sm;                                      // [NC] ascending
    float *cgiven = sm + NC;                              // [NC] as given
    float *cut = sm + 2 * NC;                             // [NC - 1]
    int *orig = reinterpret_cast<int *>(sm + 3 * NC);     // [NC]
    const int t = threadIdx.x;
    bool ok = true;
    if (t < NC) {
        const float ci = __ldg(centroids + t);
        int rank = 0;
        bool distinct = true;
#pragma unroll
        for (int j = 0; j < NC; ++j) {
            const float cj = __ldg(centroids + j);
            rank += cj < ci ? 1 : 0;
            distinct = distinct && (j >= t || cj != ci);
        }
        ok = fabsf(ci) <= 3.402823466e38f && distinct;
        cgiven[t] = ci;
        if (ok) {  // distinct finite values have distinct ranks 0 .. NC - 1
            srt[rank] = ci;
            orig[rank] = t;
        }
    }
    ok = __syncthreads_and(ok) != 0;
    bool pair_ok = true;
    if (ok && t < NC - 1) {
        const float a = srt[t], b = srt[t + 1];
        const float g = __fsub_rn(b, a);
        pair_ok = g >= 9.094947e-13f;  // 2^-40
        if (t + 1 < NC - 1) {          // neighbouring gaps within 2^15 of each other
            const float g2 = __fsub_rn(srt[t + 2], b);
            pair_ok = pair_ok && g2 <= 32768.f * g && g <= 32768.f * g2;
        }
        // the first fp32 value of [a, b] at which b beats a under the rule
        // (ties go to the lower original index)
        const bool upper_lower = orig[t + 1] < orig[t];
        uint32_t klo = f32_key(a), khi = f32_key(b);
        while (khi - klo > 1u) {  // at most 32 halvings
            const uint32_t km = klo + (khi - klo) / 2u;
            const float v = f32_from_key(km);
            const float da = __fmul_rn(__fsub_rn(v, a), __fsub_rn(v, a));
            const float db = __fmul_rn(__fsub_rn(v, b), __fsub_rn(v, b));
            const bool beats = upper_lower ? db <= da : db < da;
            if (beats) khi = km; else klo = km;
        }
        cut[t] = f32_from_key(khi);
    }
    ok = __syncthreads_and(ok && pair_ok) != 0;
    cb.ok = false;
    cb.lo = 0.f;
    cb.hi = 0.f;
    cb.perm = 0;
    cb.t = cut;
    if (ok) {
        const float lo = __fsub_rn(srt[0], __fmul_rn(32768.f, __fsub_rn(srt[1], srt[0])));
        const float hi = __fadd_rn(srt[NC - 1], __fmul_rn(32768.f, __fsub_rn(srt[NC - 1], srt[NC - 2])));
        cb.ok = __fsub_rn(hi, lo) <= 4.611686e18f;  // 2^62
        cb.lo = lo;
        cb.hi = hi;
#pragma unroll
        for (int k = 0; k < NC; ++k) cb.perm |= (uint64_t)(uint32_t)orig[k] << (4 * k);
    }
}

// Whether the cut points decide v (false for NaN, for values outside
// [lo, hi] and for codebooks that failed the set-up's conditions).
template <int NC>
__device__ __forceinline__ bool cut_decides(float v, const CutCb<NC> &cb)
{
    return cb.ok && v >= cb.lo && v <= cb.hi;
}

// The rule's answer for v through the cut points, valid when cut_decides(v):
// the original index of the k-th smallest centroid, k the number of cut
// points at or below v, by a branch-free binary search over the cut points
// in shared memory (the lanes read among NC - 1 consecutive words: no bank
// conflicts).  Callers take the rule's scan separately for the rare values
// the cut points do not decide.
template <int NC>
__device__ __forceinline__ int cut_rank(float v, const CutCb<NC> &cb)
{
    int k = 0;
#pragma unroll
    for (int step = NC / 2; step > 0; step >>= 1) k += v >= cb.t[k + step - 1] ? step : 0;
    return k;
}
template <int NC>
__device__ __forceinline__ uint32_t cut_code(float v, const CutCb<NC> &cb)
{
    return (uint32_t)(cb.perm >> (4 * cut_rank<NC>(v, cb))) & 15u;
}

}  // namespace vqs
