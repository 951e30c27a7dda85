// vq_append.cuh -- new tokens appended to the paged code cache: every
// sub-vector of their keys and values is encoded by the exact rule of
// vq_encode (fp32, each subtract, square and add rounded, lowest index of
// equals) and its code written to the token's slot.
//
// The keys and values of token t lie [heads][head_dim] at t * stride (a slice
// of a packed projection), its codes go to
//   codes[slot / P][head][slot % P][s],  P = page_size,
// and a slot outside [0, num_pages P) is skipped.
//
// What bounds it is the encode's own work, not its 8 to 20 bytes a sub-vector: so
// the kernel is the tensor-core encode (vq_tc.cuh: screening on tcgen05, the
// exact formula where the bound cannot decide) with rows that are addressed
// through the token stride and indices that go through the slot map, one launch
// for the keys and values of all heads.  A group of the launch is one head of
// one of the two; its rows are its sub-vectors, token by token.
#pragma once

#include <stdint.h>

#include "vq_check.cuh"
#include "vq_kernels.cuh"
#include "vq_tc.cuh"

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

// The sub-vectors of one head, as encode_tc_block takes its rows: row m is
// sub-vector m % ns of token m / ns.  Rows of one launch stay below 2^31, so the
// division is a 32-bit one.
template <typename T, int SUB, bool SMOOTH>
struct AppendRows {
    const AppendArgs &a;
    const T *__restrict__ x;       // the head's first sub-vector
    const float *__restrict__ sg;  // the head's smooth factors
    int kv;
    int32_t h;
    uint32_t n;                    // rows
    __device__ __forceinline__ const T *at(uint32_t m, uint32_t *s) const
    {
        const uint32_t t = m / (uint32_t)a.ns;
        *s = m - t * (uint32_t)a.ns;
        return x + (int64_t)t * a.stride[kv] + *s * SUB;
    }
    __device__ __forceinline__ int64_t elems() const
    {
        return (a.tokens - 1) * a.stride[kv] + (int64_t)a.heads * a.ns * SUB;
    }
    __device__ __forceinline__ void smooth(uint32_t s, float (&v)[SUB]) const
    {
        if constexpr (SMOOTH) {
#pragma unroll
            for (int i = 0; i < SUB; ++i) v[i] = __fdiv_rn(v[i], __ldg(sg + s * SUB + i));
        }
    }
    __device__ __forceinline__ void load(int64_t m, float (&v)[SUB]) const
    {
        constexpr uint32_t kRowAlign = SUB * sizeof(T) < 16 ? SUB * sizeof(T) : 16;
        uint32_t s;
        const T *p = at((uint32_t)m, &s);
        if (m < n && VQ_VSPAN(p, SUB, static_cast<const T *>(a.x[kv]), elems(), kRowAlign)) {
            load_row<T, SUB>(p, v);
            smooth(s, v);
        } else {
#pragma unroll
            for (int i = 0; i < SUB; ++i) v[i] = 0.f;
        }
    }
    __device__ __forceinline__ bool load_same(int64_t m, float (&v)[SUB]) const
    {
        uint32_t s;
        const T *p = at((uint32_t)m, &s);
        if (!VQ_SPAN(p, SUB, static_cast<const T *>(a.x[kv]), elems())) return false;
#pragma unroll
        for (int i = 0; i < SUB; ++i) v[i] = widen(p[i]);
        smooth(s, v);
        return true;
    }
    __device__ __forceinline__ void put(int64_t m, uint32_t id) const
    {
        const uint32_t t = (uint32_t)m / (uint32_t)a.ns, s = (uint32_t)m - t * (uint32_t)a.ns;
        uint8_t *dst = append_dst(a, kv, t, h);
        if (dst && VQ_SPAN(dst + s, 1, a.codes[kv], append_codes_bytes(a))) dst[s] = (uint8_t)id;
    }
};

// blockIdx.x: kinds * heads groups of blocks_per_group blocks; kinds (keys
// and values, or one of them) from kv0 on.
template <typename T, int SUB, int NCOL, int GC, int MINB, bool SMOOTH, int TPS>
__global__ void __launch_bounds__(128 * TPS, MINB)
    append_tc(const __grid_constant__ AppendArgs a, int kv0, int32_t blocks_per_group, int32_t tiles_per_block,
              float one)
{
    const int32_t g = blockIdx.x / blocks_per_group, blk = blockIdx.x - g * blocks_per_group;
    const int kv = kv0 + g / a.heads;
    const int32_t h = g % a.heads;
    if (!index_ok(kv, 2)) return;  // block-uniform
    const T *codebooks = static_cast<const T *>(a.codebooks[kv]);
    const uint32_t n = (uint32_t)(a.tokens * a.ns);
    const AppendRows<T, SUB, SMOOTH> rows{a, static_cast<const T *>(a.x[kv]) + (int64_t)h * a.ns * SUB,
                                          SMOOTH ? a.smooth + (int64_t)h * a.ns * SUB : nullptr, kv, h, n};
    encode_tc_block<T, SUB, NCOL, GC, SMOOTH, kWaitPolls, TPS>(rows, codebooks + (int64_t)h * a.nc * SUB, codebooks, a.heads, n, a.nc,
                                                               (int64_t)blk * tiles_per_block * 128, tiles_per_block, one);
}

}  // namespace vqk
