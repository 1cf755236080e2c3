// pieces_device.hpp - rows of 16- and 32-bit values in pieces of 16 bytes (gfx950).
#pragma once
#include "mxfp4_device.hpp"

namespace exl3 {
namespace mx {

// 16 bytes of T in four registers.  VEC: rows are whole 16-byte pieces.  Otherwise
// one value at a time, `left` of them in the row, zeros behind.
template <typename T, bool VEC> __device__ inline u32x4_t load_piece(const void* base, int64_t at, int left) {
    typedef typename T::raw raw;
    const raw* src = static_cast<const raw*>(base) + at;
    if constexpr (VEC) return *reinterpret_cast<const u32x4_t*>(src);
    u32x4_t r = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16 / T::bytes; ++i) {
        const uint32_t v = i < left ? src[i] : 0;
        if constexpr (T::bytes == 2) r[i / 2] |= v << (16 * (i & 1));
        else r[i] = v;
    }
    return r;
}
template <typename T, bool VEC, bool STREAM> __device__ inline void store_piece(void* base, int64_t at, int left, const u32x4_t r) {
    typedef typename T::raw raw;
    raw* dst = static_cast<raw*>(base) + at;
    if constexpr (VEC) {
        if constexpr (STREAM) __builtin_nontemporal_store(r, reinterpret_cast<u32x4_t*>(dst));
        else *reinterpret_cast<u32x4_t*>(dst) = r;
    } else {
#pragma unroll
        for (int i = 0; i < 16 / T::bytes; ++i)
            if (i < left) dst[i] = (raw)(T::bytes == 2 ? r[i / 2] >> (16 * (i & 1)) : r[i]);
    }
}
// Value i of a piece, and a piece of values rounded to T.
template <typename T> __device__ inline float piece_value(const u32x4_t r, int i) {
    if constexpr (T::bytes == 2) return to_f32(T{}, (uint16_t)(r[i / 2] >> (16 * (i & 1))));
    else return to_f32(T{}, r[i]);
}
template <typename T> __device__ inline u32x4_t round_piece(const float (&v)[16 / T::bytes]) {
    u32x4_t r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (T::bytes == 2) r[i] = (uint32_t)from_f32(T{}, v[2 * i]) | ((uint32_t)from_f32(T{}, v[2 * i + 1]) << 16);
        else r[i] = from_f32(T{}, v[i]);
    }
    return r;
}

}  // namespace mx
}  // namespace exl3
