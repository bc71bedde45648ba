// Sums over the rows that one or several waves hold, as the norms' kernels use them.
#pragma once

#include "ssd_block.h"

namespace ssd {

// Sum over the 64 lanes, the same in every lane: 4 steps within rows of 16 lanes on the vector
// units' own lane permutations, then the 4 rows' sums by way of scalar registers.  (Shuffles
// through LDS wait for it at each of 6 steps.)
template <int CTRL>
__device__ __forceinline__ float permuted(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
    return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ float wave_sum(float v) {
    v += permuted<0xb1>(v);       // lanes 1 apart
    v += permuted<0x4e>(v);       // 2 apart
    v += permuted<0x141>(v);      // the other 4 of 8, mirrored
    v += permuted<0x140>(v);      // the other 8 of 16, mirrored
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

// Sums over the WPR waves that share a row (WPR > 1: every wave of the workgroup).
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *red) {
    v = wave_sum(v);
    if constexpr (WPR > 1) {
        const int wave = threadIdx.x / 64;
        __syncthreads();                       // the previous sum has been read
        if (threadIdx.x % 64 == 0) red[wave] = v;
        __syncthreads();
        v = 0.f;
#pragma unroll
        for (int k = 0; k < WPR; ++k) v += red[k];
    }
    return v;
}

}  // namespace ssd
