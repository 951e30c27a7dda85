// vq_append.cuh -- new tokens appended to the paged code cache: every
// sub-vector of their keys and values is encoded by the exact rule of
// vq_encode (fp32, each subtract, square and add rounded, lowest index of
// equals) and its code written to the token's slot.
//
// The keys and values of token t lie [heads][head_dim] at t * stride (a slice
// of a packed projection), its codes go to
//   codes[slot / P][head][slot % P][s],  P = page_size,
// and a slot outside [0, num_pages P) is skipped.
#pragma once

#include <stdint.h>

#include "vq_check.cuh"
#include "vq_kernels.cuh"

namespace vqk {

struct AppendArgs {
    const void *x[2];          // keys, values
    const void *codebooks[2];  // [heads][n_centroids][sub_dim]
    uint8_t *codes[2];
    int64_t stride[2];         // elements between tokens
    const float *smooth;       // [heads][head_dim] factors of the keys, or null
    const int64_t *slots;
    int64_t tokens, num_pages, page_stride;
    int32_t heads, ns, sub, nc, page_shift;
};

// Where the codes of (token, head) go; null if the token has no slot.
__device__ __forceinline__ uint8_t *append_dst(const AppendArgs &a, int kv, int64_t t, int32_t h)
{
    if (!VQ_SPAN(a.slots + t, 1, a.slots, a.tokens)) return nullptr;
    const int64_t slot = __ldg(a.slots + t);
    if (slot < 0 || (slot >> a.page_shift) >= a.num_pages) return nullptr;
    const int64_t off = slot & (((int64_t)1 << a.page_shift) - 1);
    return a.codes[kv] + (slot >> a.page_shift) * a.page_stride + (((int64_t)h << a.page_shift) + off) * a.ns;
}

__device__ __forceinline__ int64_t append_codes_bytes(const AppendArgs &a)
{
    return (a.num_pages - 1) * a.page_stride + (((int64_t)a.heads * a.ns) << a.page_shift);
}

constexpr int kAppendMaxSub = 32;

// Any shape: a thread per sub-vector, the codebook read through the L1.
// blockIdx.y: keys or values.
template <typename T>
__global__ void __launch_bounds__(128) append_general(const __grid_constant__ AppendArgs a, int kv0, float one)
{
    const int kv = kv0 + blockIdx.y;
    const int64_t e = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t per_token = (int64_t)a.heads * a.ns;
    if (e >= a.tokens * per_token) return;
    const int64_t t = e / per_token;
    const int32_t h = (int32_t)((e - t * per_token) / a.ns), s = (int32_t)(e % a.ns);
    uint8_t *dst = append_dst(a, kv, t, h);
    if (!dst) return;
    const T *x = static_cast<const T *>(a.x[kv]) + t * a.stride[kv] + ((int64_t)h * a.ns + s) * a.sub;
    if (!VQ_SPAN(x, a.sub, static_cast<const T *>(a.x[kv]), (a.tokens - 1) * a.stride[kv] + per_token * a.sub)) return;
    const float *f = kv == 0 && a.smooth ? a.smooth + ((int64_t)h * a.ns + s) * a.sub : nullptr;
    float v[kAppendMaxSub];
    for (int i = 0; i < a.sub; ++i) {
        v[i] = widen(__ldg(x + i));
        if (f) v[i] = __fdiv_rn(v[i], __ldg(f + i));
    }
    const T *cb = static_cast<const T *>(a.codebooks[kv]) + (int64_t)h * a.nc * a.sub;
    if (!VQ_SPAN(cb, (int64_t)a.nc * a.sub, static_cast<const T *>(a.codebooks[kv]), (int64_t)a.heads * a.nc * a.sub)) return;
    float best = __int_as_float(0x7f800000);
    int idx = 0;
    for (int c = 0; c < a.nc; ++c) {
        const T *row = cb + (int64_t)c * a.sub;
        float d = add_rn(v[0], -widen(__ldg(row)));
        float acc = mul_rn(d, d);
        for (int i = 1; i < a.sub; ++i) {
            d = add_rn(v[i], -widen(__ldg(row + i)));
            acc = fma_rn(one, mul_rn(d, d), acc);
        }
        if (acc < best) {
            best = acc;
            idx = c;
        }
    }
    if (VQ_SPAN(dst + s, 1, a.codes[kv], append_codes_bytes(a))) dst[s] = (uint8_t)idx;
}

}  // namespace vqk
