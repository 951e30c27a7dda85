// vq_sappend.cuh -- new tokens appended to the paged cache of 4-bit scalar codes: each
// row of dim elements (a token's key or value of one head) is scaled to a root mean
// square of one and every element takes the index of its nearest centroid.
//
//   y = R x (keys, where signs are given: the rotation of vq_hadamard_rotate) or x, fp32
//   S = sum y^2: neighbours are added, then neighbouring sums, and so on (the row
//       padded with zeros to a power of two)
//   s = fl_T(sqrt(fl(S / dim))), T the rows' type; 0 if that is not finite; at most the
//       largest T whose product with every centroid (rounded to T) is finite in T, so
//       that whatever attends to the row may round s c_j to T
//   z = fl(y fl(1 / s)), 0 where s = 0;  code = argmin_j fl(fl(z - c_j)^2), the lowest
//       of equals (the rule of vq_scalar_quantize)
// Every step is one rounded fp32 operation in this order, so a code has one right
// answer.  Codes 2 i and 2 i + 1 share a byte, the even one in its low half.
//
// A lane holds kRowRun = 16 consecutive elements, two 16-byte loads of a 16-bit type, so
// that of the rotation's and the sum's log2 dim steps four stay in registers; a warp takes
// 32 / lanes rows side by side.  The cut points of the centroids (vq_nearest.cuh) decide a
// code: two comparisons find a quarter of them, whose three one 16-byte load brings.
//
// What bounds it: issue, 73 % of the slots for 8191 tokens of 8 heads of 128 in bf16 with rotated
// keys, 33 us a call (36 with a cold cache) where the bytes take 6.4; 49 thread instructions an
// element (rotation, comparisons, packing).  It was 43 us before rows were loaded ahead, a quarter of
// the cut points found first and 32-bit division used.  64 tokens: 13 us a call, one launch's latency.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include <type_traits>

#include "vq_check.cuh"
#include "vq_nearest.cuh"

namespace vqk {

constexpr int kRowRun = 16;
constexpr int kSAppendThreads = 256;

struct ScalarAppendArgs {
    const void *x[2];          // keys, values
    const float *centroids[2];
    uint8_t *codes[2];
    void *scales[2];
    int64_t stride[2];         // elements between tokens
    const float *signs;        // [dim] of the keys' rotation, or null
    const int64_t *slots;
    int64_t tokens, num_pages, page_stride, scale_stride;
    int32_t heads, dim, nc, page_shift;
    float norm;                // 1 / sqrt(dim)
    float over_dim;            // 1 / dim
    bool exact;                // dim is a power of two: a product with 1 / dim is the quotient
    bool vec[2];               // rows can be read in 16-byte pieces
    bool vec_codes;            // codes can be written in 8-byte pieces
};

template <typename T>
__device__ __forceinline__ T scale_of(float v);
template <>
__device__ __forceinline__ __half scale_of<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 scale_of<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ float scale_of<float>(float v) { return v; }

// The largest scale: the largest T not above (largest T) / max |c_j|, a quotient of at most
// the largest T.
template <typename T>
__device__ __forceinline__ T scale_cap(const float *__restrict__ centroids, int nc)
{
    constexpr float kMost = std::is_same<T, __half>::value ? 65504.f : std::is_same<T, float>::value ? 3.402823466e38f : 3.3895314e38f;
    float most = 1.f;
    for (int j = 0; j < nc; ++j)
        if (VQ_SPAN(centroids + j, 1, centroids, nc)) most = fmaxf(most, fabsf(vqs::widen_elem(scale_of<T>(__ldg(centroids + j)))));
    const float cap = __fdiv_rz(kMost, most);
    if constexpr (std::is_same<T, __half>::value) return __float2half_rz(cap);
    else if constexpr (std::is_same<T, float>::value) return cap;
    else return __float2bfloat16_rz(cap);
}

// LANES lanes to a row (LANES x 16 >= dim); CUTS: 16 centroids, through their cut points.
// blockIdx.y: keys or values.
template <typename T, int LANES, bool CUTS>
__global__ void __launch_bounds__(kSAppendThreads, 3) scalar_append(const __grid_constant__ ScalarAppendArgs a)
{
    constexpr int kRows = 32 / LANES;  // of a warp
    constexpr int kE = kRowRun;
    __shared__ float sm[4 * 16];
    __shared__ __align__(16) float quarters[16];
    const int kv = blockIdx.y;
    const int lane = threadIdx.x & 31, sub = lane / LANES, l = lane % LANES;
    const T *__restrict__ x = static_cast<const T *>(a.x[kv]);
    const int64_t x_elems = (a.tokens - 1) * a.stride[kv] + (int64_t)a.heads * a.dim;
    const bool rotate = kv == 0 && a.signs;
    const int64_t rows = a.tokens * a.heads, stride = (int64_t)gridDim.x * (kSAppendThreads / 32) * kRows;
    const int e0 = l * kE;
    float sg[kE];
#pragma unroll
    for (int j = 0; j < kE; ++j)
        sg[j] = rotate && e0 + j < a.dim && VQ_SPAN(a.signs + e0 + j, 1, a.signs, a.dim) ? __ldg(a.signs + e0 + j) : 0.f;
    // a warp's rows of the next pass are loaded before this pass's are worked on
    constexpr int kLoads = kE * (int)sizeof(T) / 16;
    const int64_t first = ((int64_t)blockIdx.x * (kSAppendThreads / 32) + (threadIdx.x >> 5)) * kRows;
    auto place = [&](int64_t row, int64_t *t, int *h) {
        if (rows <= 0x7fffffff) {  // (32 bits divide in a third of the steps)
            const uint32_t q = (uint32_t)row / (uint32_t)a.heads;
            *t = q;
            *h = (int)((uint32_t)row - q * (uint32_t)a.heads);
        } else {
            *t = row / a.heads;
            *h = (int)(row - *t * a.heads);
        }
    };
    uint4 raw[kLoads] = {};
    int64_t t_next = 0, slot_next = -1;
    int h_next = 0;
    auto load = [&](int64_t base) {
        const int64_t row = base + sub;
        slot_next = -1;
        if (row >= rows) return;
        place(row, &t_next, &h_next);
        if (VQ_SPAN(a.slots + t_next, 1, a.slots, a.tokens)) slot_next = __ldg(a.slots + t_next);
        const T *src = x + t_next * a.stride[kv] + (int64_t)h_next * a.dim + e0;
        if (a.vec[kv] && VQ_VSPAN(src, kE, x, x_elems, 16)) {  // (then LANES x 16 = dim)
#pragma unroll
            for (int k = 0; k < kLoads; ++k) raw[k] = __ldcs(reinterpret_cast<const uint4 *>(src) + k);
        }
    };
    if (first < rows) load(first);
    // the set-up, while the first rows come
    [[maybe_unused]] vqs::CutCb<16> cut{};
    if constexpr (CUTS) {
        vqs::build_cut_cb<16>(a.centroids[kv], sm, cut);
        if (threadIdx.x < 15) quarters[threadIdx.x] = cut.t[threadIdx.x];
        __syncthreads();
    } else {
        if ((int)threadIdx.x < a.nc) sm[16 + threadIdx.x] = __ldg(a.centroids[kv] + threadIdx.x);
        __syncthreads();
    }
    // cut points 3, 7 and 11; whether the centroids ascend
    [[maybe_unused]] const float mid[3] = {quarters[3], quarters[7], quarters[11]};
    [[maybe_unused]] const bool in_order = cut.perm == 0xfedcba9876543210ull;
    const T cap = scale_cap<T>(a.centroids[kv], a.nc);
    for (int64_t base = first; base < rows; base += stride) {
        const int64_t t = t_next, slot = slot_next;
        const int h = h_next;
        float v[kE];
        if (a.vec[kv]) {
#pragma unroll
            for (int j = 0; j < kE; ++j) v[j] = vqs::widen_elem(reinterpret_cast<const T *>(raw)[j]);
        } else {
            const T *src = x + t * a.stride[kv] + (int64_t)h * a.dim + e0;
#pragma unroll
            for (int j = 0; j < kE; ++j)
                v[j] = base + sub < rows && e0 + j < a.dim && VQ_SPAN(src + j, 1, x, x_elems) ? vqs::widen_elem(src[j]) : 0.f;
        }
        if (base + stride < rows) load(base + stride);
        const bool live = base + sub < rows && slot >= 0 && (slot >> a.page_shift) < a.num_pages;
        if (rotate) {  // (dim is a power of two; the padding of a row below 16 stays zero)
#pragma unroll
            for (int j = 0; j < kE; ++j) v[j] = __fmul_rn(v[j], sg[j]);
#pragma unroll
            for (int s = 1; s < kE; s <<= 1) {
                if (s >= a.dim) break;
#pragma unroll
                for (int j = 0; j < kE; ++j) {
                    if ((j & s) == 0) {
                        const float p = v[j], q = v[j + s];
                        v[j] = __fadd_rn(p, q);
                        v[j + s] = __fsub_rn(p, q);
                    }
                }
            }
#pragma unroll
            for (int ls = 1; ls < LANES; ls <<= 1) {
                // the upper of a pair is partner less own: fma(-1, own, partner), rounded once
                const float f = (l & ls) != 0 ? -1.0f : 1.0f;
#pragma unroll
                for (int j = 0; j < kE; ++j) v[j] = __fmaf_rn(f, v[j], __shfl_xor_sync(0xffffffffu, v[j], ls));
            }
#pragma unroll
            for (int j = 0; j < kE; ++j) v[j] = __fmul_rn(v[j], a.norm);
        }
        float q[kE];
#pragma unroll
        for (int j = 0; j < kE; ++j) q[j] = __fmul_rn(v[j], v[j]);
#pragma unroll
        for (int n = kE / 2; n > 0; n >>= 1)
#pragma unroll
            for (int j = 0; j < n; ++j) q[j] = __fadd_rn(q[2 * j], q[2 * j + 1]);
        float total = q[0];
#pragma unroll
        for (int ls = 1; ls < LANES; ls <<= 1) total = __fadd_rn(total, __shfl_xor_sync(0xffffffffu, total, ls));
        T scale = scale_of<T>(__fsqrt_rn(a.exact ? __fmul_rn(total, a.over_dim) : __fdiv_rn(total, (float)a.dim)));
        float s = vqs::widen_elem(scale);
        if (!(s <= 3.402823466e38f)) {  // NaN or infinite
            s = 0.f;
            scale = scale_of<T>(0.f);
        } else if (s > vqs::widen_elem(cap)) {
            scale = cap;
            s = vqs::widen_elem(cap);
        }
        const float inv = __frcp_rn(s);  // (infinite for the least scales: the scan decides their codes)
#pragma unroll
        for (int j = 0; j < kE; ++j) v[j] = __fmul_rn(v[j], inv);
        if (s == 0.f) {
#pragma unroll
            for (int j = 0; j < kE; ++j) v[j] = 0.f;
        }
        uint32_t code[kE];
        if constexpr (CUTS) {
            float least = v[0], most = v[0];
#pragma unroll
            for (int j = 0; j < kE; ++j) {
                const bool upper = v[j] >= mid[1], quarter = v[j] >= (upper ? mid[2] : mid[0]);
                code[j] = (upper ? 8u : 0u) + (quarter ? 4u : 0u);
                const float4 t = *reinterpret_cast<const float4 *>(quarters + code[j]);
                code[j] += (v[j] >= t.x ? 1u : 0u) + (v[j] >= t.y ? 1u : 0u) + (v[j] >= t.z ? 1u : 0u);
                least = fminf(least, v[j]);
                most = fmaxf(most, v[j]);
            }
            if (!in_order) {
#pragma unroll
                for (int j = 0; j < kE; ++j) code[j] = (uint32_t)(cut.perm >> (4 * code[j])) & 15u;
            }
            // values that the cut points do not decide (rare): the rule's scan
            if (!(cut.ok && least >= cut.lo && most <= cut.hi && inv <= 3.402823466e38f)) {
#pragma unroll
                for (int j = 0; j < kE; ++j)
                    if (!vqs::cut_decides<16>(v[j], cut)) code[j] = vqs::nearest(v[j], sm + 16, 16);
            }
        } else {
#pragma unroll
            for (int j = 0; j < kE; ++j) code[j] = vqs::nearest(v[j], sm + 16, a.nc);
        }
        if (!live) continue;
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int j = kE - 1; j >= 0; --j) w[j / 8] = w[j / 8] * 16 + code[j];
        const int64_t page = slot >> a.page_shift, off = slot & (((int64_t)1 << a.page_shift) - 1);
        const int64_t in_page = ((int64_t)h << a.page_shift) + off;
        const int ns = a.dim / 2;
        uint8_t *dst = a.codes[kv] + page * a.page_stride + in_page * ns + e0 / 2;
        const int64_t bytes = (a.num_pages - 1) * a.page_stride + (((int64_t)a.heads * ns) << a.page_shift);
        if (a.vec_codes && e0 + kE <= a.dim) {
            if (VQ_VSPAN(dst, 8, a.codes[kv], bytes, 8)) *reinterpret_cast<uint2 *>(dst) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int i = 0; i < kE / 2; ++i)
                if (e0 / 2 + i < ns && VQ_SPAN(dst + i, 1, a.codes[kv], bytes)) dst[i] = (uint8_t)(w[i / 4] >> (8 * (i % 4)));
        }
        if (l == 0) {
            T *to = static_cast<T *>(a.scales[kv]) + page * a.scale_stride + in_page;
            if (VQ_SPAN(to, 1, static_cast<T *>(a.scales[kv]), (a.num_pages - 1) * a.scale_stride + ((int64_t)a.heads << a.page_shift)))
                *to = scale;
        }
    }
}

}  // namespace vqk
