// lanes_device.hpp - values joined over groups of neighbouring lanes (gfx950).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace exl3 {

// The value of another lane of the group: step 1, 2, 4 or 8 pairs each lane of 2, 4, 8 or 16 with one
// whose half of them it is not in.  (A mirrored half or whole row of 16 lanes, from 4 on.)
template <int STEP> __device__ inline uint32_t other_lane(uint32_t v) {
    constexpr int CTRL = STEP == 1 ? 0xB1 : STEP == 2 ? 0x4E : STEP == 4 ? 0x141 : 0x140;  // quad_perm 1 0 3 2, 2 3 0 1, row_half_mirror, row_mirror
    return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
template <int STEP> __device__ inline float other_lane(float v) { return __builtin_bit_cast(float, other_lane<STEP>(__builtin_bit_cast(uint32_t, v))); }
template <int STEP> __device__ inline double other_lane(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, (uint64_t)other_lane<STEP>((uint32_t)b) | ((uint64_t)other_lane<STEP>((uint32_t)(b >> 32)) << 32));
}
// The values of the two halves of 32 or 64 lanes, in each of them: a swap of v with itself leaves the lower
// rows' values in one result and the upper ones' in the other.
template <int STEP> __device__ inline void halves(uint32_t v, uint32_t* lower, uint32_t* upper) {
    if constexpr (STEP == 16) {
        const auto both = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        *lower = both[0];
        *upper = both[1];
    } else {
        const auto both = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        *lower = both[0];
        *upper = both[1];
    }
}
template <int STEP> __device__ inline void halves(float v, float* lower, float* upper) {
    uint32_t a, b;
    halves<STEP>(__builtin_bit_cast(uint32_t, v), &a, &b);
    *lower = __builtin_bit_cast(float, a);
    *upper = __builtin_bit_cast(float, b);
}
template <int STEP> __device__ inline void halves(double v, double* lower, double* upper) {
    const uint64_t w = __builtin_bit_cast(uint64_t, v);
    uint32_t a[2], b[2];
    halves<STEP>((uint32_t)w, &a[0], &b[0]);
    halves<STEP>((uint32_t)(w >> 32), &a[1], &b[1]);
    *lower = __builtin_bit_cast(double, (uint64_t)a[0] | ((uint64_t)a[1] << 32));
    *upper = __builtin_bit_cast(double, (uint64_t)b[0] | ((uint64_t)b[1] << 32));
}

// v joined over each group of LANES lanes (a power of two), in every lane of it.  All lanes of a
// group are active, or none.
template <int LANES, typename V, typename F> __device__ inline V over_lanes(V v, F join) {
    if constexpr (LANES > 1) v = join(v, other_lane<1>(v));
    if constexpr (LANES > 2) v = join(v, other_lane<2>(v));
    if constexpr (LANES > 4) v = join(v, other_lane<4>(v));
    if constexpr (LANES > 8) v = join(v, other_lane<8>(v));
    V lower, upper;
    if constexpr (LANES > 16) {
        halves<16>(v, &lower, &upper);
        v = join(lower, upper);
    }
    if constexpr (LANES > 32) {
        halves<32>(v, &lower, &upper);
        v = join(lower, upper);
    }
    return v;
}

}  // namespace exl3
