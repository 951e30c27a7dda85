// vq_sattn.cuh -- attention of new tokens over the paged cache of 4-bit scalar codes:
// the general kernel.  The work split and the merge are those of vq_pattn.cuh, and so is
// the definition, with
//   K^[t][d] = s_k[t] c_k[code],  V^[t][d] = s_v[t] c_v[code],
// the centroids rounded to the rows' type and a code >= n_centroids standing for 0.
//
// Any type, even head size up to kSimpleDim and page size: a block of kUnit threads takes
// one new token and up to kSimpleRows query heads; a unit is one cached token per thread
// for the scores and one pair of columns (or more) per thread for the weighted sum, all in
// fp32.  It carries what the tensor kernels do not (fp32, other head sizes, small pages,
// pools off 16-byte alignment) and is bound by its loads: the codes go through the L1
// once for the scores and once for the sum.
#pragma once

#include "vq_pattn.cuh"

namespace vqk {

constexpr int kScalarCodes = 16;

// The centroids in the rows' type, as fp32; 0 for codes past them.  The caller synchronises.
template <typename T>
__device__ __forceinline__ void scalar_book(const float *__restrict__ cent, int nc, float *book)
{
    const int i = threadIdx.x;
    if (i < kScalarCodes) book[i] = i < nc && VQ_SPAN(cent + i, 1, cent, nc) ? widen(narrow<T>(__ldg(cent + i))) : 0.f;
}

template <typename T>
__global__ void __launch_bounds__(kUnit) paged_attn_scalar_simple(const __grid_constant__ PagedArgs a)
{
    __shared__ PagedWalk<> w;
    __shared__ float sp[kSimpleRows][kUnit];
    __shared__ float red[kSimpleRows][kUnit / 32];
    __shared__ int64_t spage[kUnit];
    __shared__ float sv[kUnit];
    __shared__ float k_book[kScalarCodes], v_book[kScalarCodes];
    extern __shared__ float sq[];  // [kSimpleRows][dim]
    constexpr int kPairs = kSimpleDim / 2 / kUnit;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const T *__restrict__ q = static_cast<const T *>(a.q);
    const T *__restrict__ ks = static_cast<const T *>(a.k_scales);
    const T *__restrict__ vs = static_cast<const T *>(a.v_scales);
    T *__restrict__ out = static_cast<T *>(a.out);
    const int64_t code_bytes = (a.num_pages - 1) * a.page_stride + (((int64_t)a.hkv * a.ns) << a.page_shift);
    const int64_t scale_elems = (a.num_pages - 1) * a.scale_stride + ((int64_t)a.hkv << a.page_shift);

    scalar_book<T>(a.k_cent, a.nc, k_book);
    scalar_book<T>(a.v_cent, a.nc, v_book);
    PagedLens l;
    PagedNote note{};
    if (paged_plan<kUnit>(a, w, l)) {  // (has barriers: the books are written)
        PagedCursor cur;
        cur.init(w, (int32_t)blockIdx.x);
        PagedSegment s;
        while (cur.next(a, w, l, s, note)) {
            const int r = cur.r;
            const int h = s.hx / a.gch, g0 = s.hx % a.gch * a.gc;
            const int rows = a.group - g0 < a.gc ? a.group - g0 : a.gc;  // one token: a row per head
            const int head0 = h * a.group + g0;
            const int64_t tok = s.it.tok0;
            const int64_t head_rows = (int64_t)h << a.page_shift;
            __syncthreads();
            for (int i = tid; i < kSimpleRows * a.dim; i += kUnit) {
                const int g = i / a.dim, d = i - g * a.dim;
                const T *src = q + tok * a.q_stride + (int64_t)(head0 + g) * a.dim + d;
                float v = 0.f;
                if (g < rows && VQ_SPAN(src, 1, q, (a.tokens - 1) * a.q_stride + (int64_t)a.hq * a.dim))
                    v = widen(*src);
                sq[i] = v;
            }
            float m[kSimpleRows], sum[kSimpleRows], acc[kSimpleRows][kPairs][2];
#pragma unroll
            for (int g = 0; g < kSimpleRows; ++g) {
                m[g] = __int_as_float(0xff800000);
                sum[g] = 0.f;
#pragma unroll
                for (int c = 0; c < kPairs; ++c) acc[g][c][0] = acc[g][c][1] = 0.f;
            }
            bool saw = false;
            for (int unit = s.begin; unit < s.end; ++unit) {
                const int32_t t = s.it.k_lo + unit * kUnit + tid;
                bool seen = t < s.it.k_hi && t <= s.it.pos0 && (a.window == 0 || (int64_t)t > (int64_t)s.it.pos0 - a.window);
                int64_t page = -1, in_page = 0;
                if (seen) {
                    page = paged_page(a, r, t);
                    in_page = head_rows + (t & ((1 << a.page_shift) - 1));
                    if (page < 0) seen = false;
                }
                saw |= seen;
                __syncthreads();  // sq is written; the last unit's sp, sv and spage are read
                const int64_t code_row = seen ? page * a.page_stride + in_page * a.ns : -1;
                const T *vscale = vs + page * a.scale_stride + in_page, *kscale = ks + page * a.scale_stride + in_page;
                spage[tid] = code_row;
                sv[tid] = seen && VQ_SPAN(vscale, 1, vs, scale_elems) ? widen(__ldg(vscale)) : 0.f;
                float dot[kSimpleRows];
#pragma unroll
                for (int g = 0; g < kSimpleRows; ++g) dot[g] = 0.f;
                if (seen && span_ok(a.k_codes + code_row, a.ns, a.k_codes, code_bytes, 1) && VQ_SPAN(kscale, 1, ks, scale_elems)) {
                    for (int i = 0; i < a.ns; ++i) {
                        const int byte = __ldg(a.k_codes + code_row + i);
                        const float lo = k_book[byte & 15], hi = k_book[byte >> 4];
#pragma unroll
                        for (int g = 0; g < kSimpleRows; ++g)
                            dot[g] = fmaf(sq[g * a.dim + 2 * i + 1], hi, fmaf(sq[g * a.dim + 2 * i], lo, dot[g]));
                    }
                    const float f = a.kappa * widen(__ldg(kscale));
#pragma unroll
                    for (int g = 0; g < kSimpleRows; ++g) dot[g] *= f;
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
                for (int c = 0; c < kPairs; ++c) {
                    const int i = tid + c * kUnit;
                    if (i >= a.ns) break;
#pragma unroll
                    for (int g = 0; g < kSimpleRows; ++g) {
                        acc[g][c][0] *= scale[g];
                        acc[g][c][1] *= scale[g];
                    }
                    for (int k = 0; k < kUnit; ++k) {
                        const int64_t cr = spage[k];
                        if (cr < 0) continue;  // not seen: whatever its page holds
                        if (!span_ok(a.v_codes + cr + i, 1, a.v_codes, code_bytes, 1)) continue;
                        const int byte = __ldg(a.v_codes + cr + i);
                        const float lo = sv[k] * v_book[byte & 15], hi = sv[k] * v_book[byte >> 4];
#pragma unroll
                        for (int g = 0; g < kSimpleRows; ++g) {
                            acc[g][c][0] = fmaf(sp[g][k], lo, acc[g][c][0]);
                            acc[g][c][1] = fmaf(sp[g][k], hi, acc[g][c][1]);
                        }
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
                const float inv = s.whole ? paged_inv(m[g], total) : 1.f;
                const int64_t prow = s.slot * a.tile_rows + g, prows = 2 * (int64_t)gridDim.x * a.tile_rows;
#pragma unroll
                for (int c = 0; c < kPairs; ++c) {
                    const int i = tid + c * kUnit;
                    if (i >= a.ns) break;
                    T *dst = out + orow * a.dim + 2 * i;
                    float *pdst = a.part + prow * a.dim + 2 * i;
                    if (s.whole) {
                        if (VQ_SPAN(dst, 2, out, a.tokens * a.hq * a.dim)) {
                            dst[0] = narrow<T>(acc[g][c][0] * inv);
                            dst[1] = narrow<T>(acc[g][c][1] * inv);
                        }
                    } else if (VQ_SPAN(pdst, 2, a.part, prows * a.dim)) {
                        pdst[0] = acc[g][c][0];
                        pdst[1] = acc[g][c][1];
                    }
                }
                if (tid == 0 && s.whole && a.lse && VQ_SPAN(a.lse + orow, 1, a.lse, a.tokens * a.hq))
                    a.lse[orow] = paged_lse(m[g], total);
                if (tid == 0 && !s.whole && VQ_SPAN(a.ml + prow * 2, 2, a.ml, prows * 2)) {
                    a.ml[prow * 2] = m[g];
                    a.ml[prow * 2 + 1] = total;
                }
            }
        }
    }
    if (tid == 0 && VQ_SPAN(a.notes + blockIdx.x, 1, a.notes, gridDim.x)) a.notes[blockIdx.x] = note;
}

}  // namespace vqk
