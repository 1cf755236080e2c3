// tile_device.hpp - what the products' tiles share: memory straight into LDS, stores
// of results, and which tile a workgroup takes (gfx950).
#pragma once
#include "mxfp4_device.hpp"

namespace exl3 {
namespace mx {

// Memory from `base` on, read at 32-bit offsets.
__device__ inline __amdgpu_buffer_rsrc_t buffer(const uint8_t* base, int64_t bytes) {
    const uint32_t n = bytes > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, n, 0x00020000);
}
// Straight into LDS: lane l's 16 bytes at dst + 16 l.
__device__ inline void load16_to_lds(__amdgpu_buffer_rsrc_t b, i32x4_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}
constexpr uint32_t OUTSIDE = 0x7FFFFFF0u;  // an offset past every buffer: the load gives zeros

__device__ inline void load4_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 4, voff, soff, 0, 0);
}

template <typename OT> __device__ inline void store4(void* y, int64_t at, int count, bool vec, const f32x4_t v) {
    typedef typename OT::raw raw;
    raw* dst = static_cast<raw*>(y) + at;
    if (vec && count >= 4) {
        if constexpr (OT::bytes == 2) {
            uint2 r;
            r.x = (uint32_t)from_f32(OT{}, v[0]) | ((uint32_t)from_f32(OT{}, v[1]) << 16);
            r.y = (uint32_t)from_f32(OT{}, v[2]) | ((uint32_t)from_f32(OT{}, v[3]) << 16);
            *reinterpret_cast<uint2*>(dst) = r;
        } else {
            *reinterpret_cast<f32x4_t*>(dst) = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) dst[i] = from_f32(OT{}, v[i]);
    }
}

// Workgroup b of a launch to tile index: units of 16 consecutive tiles go to the
// same XCD (workgroups go round the 8 XCDs one by one), so that the tiles that
// run together on an XCD share rows and weights in its L2.  Units of 8 to 32 and
// bands of 2 to 16 measure the same within 3 %, but for 4096 rows in 64 groups 2048
// -> 2816: 54 us against 61 with units of 32 in bands of 8 (empty tiles, which end
// at once, then come in longer runs of one XCD); units of 64 are 15 to 80 % slower.
constexpr int XCDS = 8, XCD_UNIT = 16;
__device__ inline int xcd_tile(int b) {
    const int xcd = b % XCDS, local = b / XCDS;
    return (local / XCD_UNIT * XCDS + xcd) * XCD_UNIT + local % XCD_UNIT;
}
// Tiles of a launch, padded to whole rounds of units.
inline int64_t xcd_padded(int64_t tiles) { return (tiles + XCDS * XCD_UNIT - 1) / (XCDS * XCD_UNIT) * (XCDS * XCD_UNIT); }
constexpr int BAND = 4;  // row tiles that share a run of output tiles
// Row tile and output tile of a tile index: bands of BAND row tiles, an output
// tile's row tiles after each other.  False behind the last tile.
__device__ inline bool tile_of(int tile, int row_tiles, int col_tiles, int* row, int* col) {
    const int band = tile / (BAND * col_tiles), height = min(BAND, row_tiles - band * BAND);
    if (height <= 0) return false;
    const int in_band = tile - band * BAND * col_tiles;
    *col = in_band / height;
    *row = band * BAND + in_band - *col * height;
    return *col < col_tiles;
}

}  // namespace mx
}  // namespace exl3
