// mxfp4_device.hpp - device building blocks of the MXFP4 kernels (gfx950).
//
// The matrix core's v_mfma_scale_f32_16x16x128_f8f6f4 takes, per lane, 32 codes
// (16 bytes) of one row and the scale byte of those 32: lane l holds row l % 16
// and the (l / 16)th of the four blocks of 128 inputs, the code of the lower
// input in the lower half of its byte; accumulator i of lane l is row
// 4 * (l / 16) + i of the first operand against row l % 16 of the second.
//
// The order of the inputs is free as long as both operands agree.  A span is
// 512 inputs (16 blocks); lane quarter q holds blocks 4q .. 4q + 3 of it and
// feeds block 4q + j to the jth of four MFMAs.  A lane then reads 64 consecutive
// bytes of codes and one dword of scales per span, and MFMA j selects byte j of
// that dword (op_sel), so no instruction moves a scale.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mxfp4_plan.hpp"

namespace exl3 {
namespace mx {

typedef int i32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Type tags of the 16- and 32-bit tensors.
struct F16 { typedef uint16_t raw; static constexpr int bytes = 2; };
struct BF16 { typedef uint16_t raw; static constexpr int bytes = 2; };
struct F32 { typedef uint32_t raw; static constexpr int bytes = 4; };

__device__ inline float to_f32(F16, uint16_t v) { return (float)__builtin_bit_cast(_Float16, v); }
__device__ inline float to_f32(BF16, uint16_t v) { return __builtin_bit_cast(float, (uint32_t)v << 16); }
__device__ inline float to_f32(F32, uint32_t v) { return __builtin_bit_cast(float, v); }
// Round to nearest even, once.
__device__ inline uint16_t from_f32(F16, float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }
__device__ inline uint16_t from_f32(BF16, float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }
__device__ inline uint32_t from_f32(F32, float v) { return __builtin_bit_cast(uint32_t, v); }

// Largest magnitude over dwords of T, as the bits of an fp32 (NaN and infinity
// keep an all-ones exponent): magnitudes order like their bit patterns.
template <typename T> __device__ inline uint32_t abs_max(uint32_t m, uint32_t w) {
    if constexpr (T::bytes == 2) {
        const u16x2_t a = __builtin_bit_cast(u16x2_t, m), b = __builtin_bit_cast(u16x2_t, w & 0x7FFF7FFFu);
        return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(a, b));
    } else {
        const uint32_t b = w & 0x7FFFFFFFu;
        return m > b ? m : b;
    }
}
template <typename T> __device__ inline uint32_t abs_max_f32_bits(uint32_t m) {
    if constexpr (T::bytes == 2) {
        const uint32_t lo = m & 0xFFFFu, hi = m >> 16, v = lo > hi ? lo : hi;
        return __builtin_bit_cast(uint32_t, to_f32(T{}, (uint16_t)v));
    } else {
        return m;
    }
}

// The scale byte of a block whose largest magnitude has these fp32 bits: its
// exponent less 2, the exponent of the largest code (6 = 1.5 * 2^2); magnitudes
// below 2^-125 share 2^-127; 255 when the block holds a NaN or an infinity.
__device__ inline uint32_t scale_byte(uint32_t amax_bits) {
    const uint32_t e = amax_bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}
// 2^(b - 127) as fp32, the divisor of the conversion (subnormal for b = 0).
__device__ inline float scale_value(uint32_t b) { return __builtin_bit_cast(float, b == 0u ? 0x00400000u : b << 23); }

// v_cvt_scalef32_pk_fp4_*: two values over `scale`, rounded to nearest even and
// saturated, into byte SEL of `old` (checked against the definition over every
// exponent, ties and subnormals included).
template <int SEL> __device__ inline uint32_t cvt_pair(F16, uint32_t old, uint32_t w, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, __builtin_bit_cast(f16x2_t, w), scale, SEL);
}
template <int SEL> __device__ inline uint32_t cvt_pair(BF16, uint32_t old, uint32_t w, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, __builtin_bit_cast(bf16x2_t, w), scale, SEL);
}
template <int SEL> __device__ inline uint32_t cvt_pair_f32(uint32_t old, uint32_t w0, uint32_t w1, float scale) {
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, __builtin_bit_cast(float, w0), __builtin_bit_cast(float, w1), scale, SEL);
}
// Eight values (4 dwords of a 16-bit type, 8 of fp32) to one dword of codes.
template <typename T> __device__ inline uint32_t cvt8(const uint32_t* w, float scale) {
    uint32_t r = 0;
    if constexpr (T::bytes == 2) {
        r = cvt_pair<0>(T{}, r, w[0], scale);
        r = cvt_pair<1>(T{}, r, w[1], scale);
        r = cvt_pair<2>(T{}, r, w[2], scale);
        r = cvt_pair<3>(T{}, r, w[3], scale);
    } else {
        r = cvt_pair_f32<0>(r, w[0], w[1], scale);
        r = cvt_pair_f32<1>(r, w[2], w[3], scale);
        r = cvt_pair_f32<2>(r, w[4], w[5], scale);
        r = cvt_pair_f32<3>(r, w[6], w[7], scale);
    }
    return r;
}

// D += A * B for 16 x 16 x 128; J selects the scale byte on both sides.
template <int J> __device__ inline f32x4_t mfma(const i32x4_t a, uint32_t sa, const i32x4_t b, uint32_t sb, f32x4_t c) {
    const i32x8_t a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, 4, 4, J, (int)sa, J, (int)sb);  // 4: E2M1
}

// D += A * B for 32 x 32 x 64: lane l holds row l % 32 and the (l / 32)th of the
// two blocks of 64 inputs; accumulator i is row 8 (i / 4) + 4 (l / 32) + i % 4 of
// the first operand against row l % 32 of the second.  One wave can issue this
// form at the matrix core's full rate (32 cycles each, 8.4 PFLOP/s measured over
// the card), the 16 x 16 x 128 form only every 29 cycles instead of 16.
template <int J> __device__ inline f32x16_t mfma32(const i32x4_t a, uint32_t sa, const i32x4_t b, uint32_t sb, f32x16_t c) {
    const i32x8_t a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a8, b8, c, 4, 4, J, (int)sa, J, (int)sb);
}

// Row tile `tile` of `bm` rows: its group, first row and row count.  With
// offsets, the groups' tiles follow each other, each group starting a new tile,
// then the rows behind the last group as group n_groups.  rows == 0: no such
// tile.  Every wave finds it alone: 64 groups at a time, a scan of their tile
// counts, the first whose running count passes the tile.  The offsets of 256 groups
// are asked for together: 64 rows in 1024 groups 1024 -> 1024 12 us against 20 with
// a wait for each scan's.
struct RowTile {
    int group, row0, rows;
};
__device__ inline int clamp_row(int v, int rows) { return v < 0 ? 0 : (v > rows ? rows : v); }

// Running sum over the lanes of a wave: DPP shifts inside rows of 16 lanes, then
// each row's last lane to the rows behind it.
__device__ inline int wave_scan(int v) {
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);   // row_shr:1
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);   // row_shr:2
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);   // row_shr:4
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);   // row_shr:8
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);  // row_bcast:15 into rows 1 and 3
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);  // row_bcast:31 into rows 2 and 3
    return v;
}

__device__ inline RowTile find_tile(const int* offsets, int n_groups, int rows, int tile, int bm) {
    if (!offsets) {
        const int row0 = tile * bm;
        return RowTile{0, row0, max(min(bm, rows - row0), 0)};
    }
    const int lane = threadIdx.x & 63;
    constexpr int U = 4;  // scans whose offsets are asked for together
    int before = 0;
    for (int g0 = 0; g0 <= n_groups; g0 += 64 * U) {
        int lo[U], hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + 64 * u + lane;
            lo[u] = hi[u] = 0;
            if (g <= n_groups) {
                lo[u] = offsets[g];
                hi[u] = g < n_groups ? offsets[g + 1] : rows;
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (g0 + 64 * u > n_groups) break;
            const int first = clamp_row(lo[u], rows), end = clamp_row(hi[u], rows);
            const int count = end > first ? end - first : 0;
            const int tiles = (count + bm - 1) / bm;
            const int sum = before + wave_scan(tiles);
            const uint64_t past = __ballot(sum > tile);
            if (past) {
                const int at = __ffsll((unsigned long long)past) - 1;
                const int within = (tile - __builtin_amdgcn_readlane(sum - tiles, at)) * bm;
                return RowTile{g0 + 64 * u + at, __builtin_amdgcn_readlane(first, at) + within,
                               min(bm, __builtin_amdgcn_readlane(count, at) - within)};
            }
            before = __builtin_amdgcn_readlane(sum, 63);
        }
    }
    return RowTile{0, 0, 0};
}

// Most row tiles that `rows` rows in n_groups groups and the rows behind them make.
inline int64_t max_row_tiles(bool grouped, int rows, int n_groups, int bm) {
    if (!grouped) return ((int64_t)rows + bm - 1) / bm;
    const int64_t parts = (int64_t)n_groups + 1 < rows ? (int64_t)n_groups + 1 : rows;
    return rows / bm + parts;
}

}  // namespace mx
}  // namespace exl3
