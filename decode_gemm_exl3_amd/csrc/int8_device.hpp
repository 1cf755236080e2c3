// int8_device.hpp - device building blocks of the 8-bit integer kernels (gfx950).
#pragma once
#include "lanes_device.hpp"
#include "pieces_device.hpp"
#include "tile_device.hpp"

namespace exl3 {
namespace i8 {

using namespace mx;  // element types, pieces, row tiles of groups

// Waits for all but `PENDING` of this wave's loads from memory; with LDS for its reads of LDS too.
template <int PENDING, bool LDS> __device__ inline void wait_loads() {
    static_assert(PENDING < 64, "a wait counts to 63");
    __builtin_amdgcn_s_waitcnt((LDS ? 0x0070 : 0x0F70) | (PENDING & 15) | ((PENDING >> 4) << 14));
}

// A product, rounded to fp32: without this a conversion to fp16 that follows would become one
// instruction with it and round the exact product, about 1 in 2^13 of them to another value.
__device__ inline float rounded(float v) {
    asm("" : "+v"(v));
    return v;
}

// Codes of N values u, in N / 4 dwords: 127 u / largest, rounded to the nearest, ties to even,
// exactly.  q = u * inverse with inverse = fl(127 / largest) is within 1.6e-5 of the quotient
// (two roundings of a number up to 127), so only a piece that holds a q nearer than 2^-15 to a
// tie is rounded again, from the quotient in 64 bits.  (127 u has at most 31 bits, so that a
// quotient that is a tie comes out as one, and any other is far enough away.)  Ties are common
// in 16-bit types: u = largest / 2 is one.
template <int N> __device__ inline void code_piece(const float (&u)[N], float largest, float inverse, uint32_t (&out)[N / 4]) {
    constexpr float ROUND = 12582912.f;  // 1.5 * 2^23: a sum's low byte is the rounded value
    uint32_t bits[N];
    float nearest = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float q = u[i] * inverse, m = q + ROUND;
        bits[i] = __builtin_bit_cast(uint32_t, m);
        nearest = fmaxf(nearest, fabsf(q - (m - ROUND)));
    }
    // largest below 2^-100: 127 / largest may be infinite
    if (nearest > 0.5f - 0x1p-15f || largest < 0x1p-100f) {
#pragma unroll
        for (int i = 0; i < N; ++i)
            bits[i] = largest > 0.f ? (uint32_t)(int)__builtin_rint(127.0 * (double)u[i] / (double)largest) : 0u;
    }
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        // bytes 0 of two, then of the other two on top
        const uint32_t lo = __builtin_amdgcn_perm(bits[i + 1], bits[i], 0x0C0C0400u), hi = __builtin_amdgcn_perm(bits[i + 3], bits[i + 2], 0x04000C0Cu);
        out[i / 4] = lo | hi;
    }
}

// The magnitudes' bits of a piece's values join `amax` (NaN and infinity have an all-ones
// exponent: magnitudes order like their bits).
template <int N> __device__ inline uint32_t amax_piece(uint32_t amax, const float (&u)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t b = __builtin_bit_cast(uint32_t, u[i]) & 0x7FFFFFFFu;
        amax = amax > b ? amax : b;
    }
    return amax;
}
constexpr uint32_t NOT_FINITE = 0x7F800000u;  // and above

// A row's scale from the bits of its largest magnitude; `root`: what a norm divides by.
__device__ inline float row_scale(uint32_t amax, double root) {
    if (amax >= NOT_FINITE) return __builtin_nanf("");
    return amax == 0 ? 0.f : (float)((double)__builtin_bit_cast(float, amax) / 127.0 / root);
}

__device__ inline uint32_t larger(uint32_t a, uint32_t b) { return a > b ? a : b; }

// Tile `index` of a product: its group, first row, row count and output tile, of tiles of bm rows in
// col_tiles runs of outputs.  rows == 0: no such tile.  With groups a group's tiles follow each
// other, in bands of row tiles as above, so that a weight comes from memory once (in bands
// over all groups' row tiles those that a band's border splits came twice: 16384 rows in 64 groups
// 2048 -> 2816 read 590 MB, of which the rows and weights are 403).
struct ProductTile {
    int group, row0, rows, col;
};
// Rows of 64 groups, one a lane: the first, and how many; the rows behind the last group are group n_groups.
struct GroupRows {
    int first, count;
};
__device__ inline GroupRows group_rows(int lo, int hi, int rows) {
    const int first = clamp_row(lo, rows), end = clamp_row(hi, rows);
    return GroupRows{first, end > first ? end - first : 0};
}
// The tile, if it is one of 64 groups from g0 on; `before`: row tiles of the groups before, to which these are added.
__device__ inline bool tile_of_groups(const GroupRows& g, int g0, int index, int bm, int col_tiles, int* before, ProductTile* t) {
    const int tiles = (g.count + bm - 1) / bm;
    const int sum = *before + wave_scan(tiles);
    const uint64_t past = __ballot((int64_t)sum * col_tiles > index);
    *before = __builtin_amdgcn_readlane(sum, 63);
    if (!past) return false;
    const int at = __ffsll((unsigned long long)past) - 1;
    const int mine = __builtin_amdgcn_readlane(tiles, at), start = __builtin_amdgcn_readlane(sum, at) - mine;
    int row;
    tile_of(index - start * col_tiles, mine, col_tiles, &row, &t->col);
    t->group = g0 + at;
    t->row0 = __builtin_amdgcn_readlane(g.first, at) + row * bm;
    t->rows = min(bm, __builtin_amdgcn_readlane(g.count, at) - row * bm);
    return true;
}

// The rows of groups, kept by a workgroup that looks for several tiles: of the first 128 with the rows
// behind the last.  (Read again for each tile, they would wait for all of its loads and stores: 16384 rows
// in 64 groups 2048 -> 2816 148 us against 144, 1024 rows in 8 groups 4096 -> 14336 129 against 125.)
constexpr int KEPT_GROUPS = 128;
struct KeptGroups {
    GroupRows rows[KEPT_GROUPS / 64];
};
__device__ inline KeptGroups keep_groups(const int* offsets, int n_groups, int rows) {
    KeptGroups k;
#pragma unroll
    for (int u = 0; u < KEPT_GROUPS / 64; ++u) {
        const int g = 64 * u + (threadIdx.x & 63);
        k.rows[u] = GroupRows{0, 0};
        if (offsets && g <= n_groups) k.rows[u] = group_rows(offsets[g], g < n_groups ? offsets[g + 1] : rows, rows);
    }
    return k;
}

__device__ inline ProductTile product_tile(const int* offsets, int n_groups, int rows, int index, int bm, int row_tiles, int col_tiles,
                                           const KeptGroups* kept = nullptr) {
    ProductTile t = {0, 0, 0, 0};
    if (!offsets) {
        int row;
        if (tile_of(index, row_tiles, col_tiles, &row, &t.col)) {
            t.row0 = row * bm;
            t.rows = max(min(bm, rows - t.row0), 0);
        }
        return t;
    }
    int before = 0;
    if (kept && n_groups < KEPT_GROUPS) {
#pragma unroll
        for (int u = 0; u < KEPT_GROUPS / 64; ++u)
            if (tile_of_groups(kept->rows[u], 64 * u, index, bm, col_tiles, &before, &t)) break;
        return t;
    }
    constexpr int U = 4;  // scans whose offsets are asked for together
    for (int g0 = 0; g0 <= n_groups; g0 += 64 * U) {
        int lo[U], hi[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int g = g0 + 64 * u + (threadIdx.x & 63);
            lo[u] = hi[u] = 0;
            if (g <= n_groups) {
                lo[u] = offsets[g];
                hi[u] = g < n_groups ? offsets[g + 1] : rows;
            }
        }
        wait_loads<0, false>();  // for those that are not used too: nothing waits for them behind this
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (tile_of_groups(group_rows(lo[u], hi[u], rows), g0 + 64 * u, index, bm, col_tiles, &before, &t)) return t;
    }
    return t;
}

}  // namespace i8
}  // namespace exl3
