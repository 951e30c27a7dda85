// vq_tc_host.h -- launch planning of the tensor-core encode (vq_tc.cuh), shared
// by the dense and the paged encode (internal; not part of the C ABI).
#pragma once

#include <stdint.h>

#include <type_traits>

#include "vq_host.h"
#include "vq_tc.cuh"

namespace vqh {

// The least centroids the screening kernels take.
constexpr int kFilterMinCentroids = 64;
// The most centroids the tensor-core kernel takes.
constexpr int kTcMaxCentroids = 256;

// Blocks per group and 128-row tiles per block.  A block works through its
// tiles `tps` at a time; its time is taken as its steps plus half a step of
// set-up (codebook staging), the launch's time as waves of `slots` resident
// blocks times that.  The best of 1..64 tiles per block and the one-wave
// shape is used.
inline void tc_shape(int64_t n_groups, int64_t n_per_group, int slots, int tps, int64_t *blocks_per_group,
              int32_t *tiles_per_block)
{
    const int64_t tiles = (n_per_group + 127) / 128;
    int64_t per_group = slots / n_groups;
    if (per_group < 1) per_group = 1;
    const int64_t one_wave = (tiles + per_group - 1) / per_group;
    int64_t best_t = 1;
    double best_cost = 1e300;
    auto consider = [&](int64_t t) {
        if (t < 1 || t > tiles) return;
        const int64_t blocks = n_groups * ((tiles + t - 1) / t);
        const int64_t waves = (blocks + slots - 1) / slots;
        const double cost = (double)waves * ((double)((t + tps - 1) / tps) + 0.5);
        if (cost < best_cost) {
            best_cost = cost;
            best_t = t;
        }
    };
    consider(one_wave);
    for (int64_t t = 1; t <= 64; ++t) consider(t);
    if (best_t > (1 << 30)) best_t = 1 << 30;
    *tiles_per_block = (int32_t)best_t;
    *blocks_per_group = (tiles + best_t - 1) / best_t;
}

// A holds two tf32 pieces of each row when the rows are not 16-bit values
// (smoothed or fp32), B two pieces of -2c for fp32 codebooks.
template <int SUB, bool SMOOTH = false>
size_t tc_smem(int32_t n_centroids, vq_dtype dtype)
{
    if (dtype == VQ_F32) {
        using C = vqk::TcConfig<SUB, true>;
        return vqk::TcLayout<SUB, C::kCols, C::kGroup, 2, 2, C::kTps>::bytes(n_centroids);
    }
    using C = vqk::TcConfig<SUB, SMOOTH>;
    return vqk::TcLayout<SUB, C::kCols, C::kGroup, SMOOTH ? 2 : 1, 1, C::kTps>::bytes(n_centroids);
}

// Rows go to the tensor cores as two tf32 pieces when they are smoothed or fp32.
template <typename T, bool SMOOTH>
constexpr bool tc_split() { return SMOOTH || std::is_same<T, float>::value; }

// Resident tensor-core CTAs on the device: the register budget of the launch
// bounds admits kMinBlocks per SM, the tensor memory 512 / kCols, and the
// shared memory of an SM (228 KiB, 1 KiB reserved per block) what `smem`
// allows.
// Tiles per step of the tensor-core kernel; `split` as in tc_split.
inline int tc_tps(int sub_dim, bool split)
{
    if (sub_dim == 4) return split ? vqk::TcConfig<4, true>::kTps : vqk::TcConfig<4, false>::kTps;
    return split ? vqk::TcConfig<8, true>::kTps : vqk::TcConfig<8, false>::kTps;
}

inline int tc_slots(int sub_dim, bool split, size_t smem)
{
    const int sms = vqh_device_sms();
    int per_sm = sub_dim == 4 ? (split ? vqk::TcConfig<4, true>::kMinBlocks : vqk::TcConfig<4, false>::kMinBlocks)
                              : (split ? vqk::TcConfig<8, true>::kMinBlocks : vqk::TcConfig<8, false>::kMinBlocks);
    const int by_smem = (int)((size_t)228 * 1024 / (smem + 1024));
    if (by_smem < per_sm) per_sm = by_smem;
    if (per_sm < 1) per_sm = 1;
    return (sms > 0 ? sms : 152) * per_sm;
}

}  // namespace vqh
