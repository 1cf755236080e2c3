// int8_plan.hpp - how the few-rows product of 8-bit rows is laid out and split, and which
// kernel makes a product (host and device, no HIP in it).
#pragma once
#include <stdint.h>

#ifdef __HIPCC__
#define EXL3_I8_PLAN __host__ __device__ constexpr
#else
#define EXL3_I8_PLAN constexpr
#endif

namespace exl3 {
namespace i8 {

constexpr int BLOCK = 16;        // inputs of a 16-byte slot
constexpr int SPAN_BLOCKS = 16;  // blocks per span: 256 inputs
constexpr int CUS = 256, CU_LDS = 160 * 1024;

constexpr int SMALL_WAVES = 8, SMALL_RING = 2, SMALL_MAX_ROWS = 16;
constexpr int HELD_BLOCKS = 1024;  // 16-byte slots of held rows: with the rings half of a CU's LDS

EXL3_I8_PLAN int64_t spans_of(int n_in) { return ((int64_t)n_in + SPAN_BLOCKS * BLOCK - 1) / (SPAN_BLOCKS * BLOCK); }

// Rows of a tile whose codes HELD_BLOCKS hold (0: none fits).
EXL3_I8_PLAN int held_rows(int n_in) {
    const int64_t rows = HELD_BLOCKS / (spans_of(n_in) * SPAN_BLOCKS);
    return rows < SMALL_MAX_ROWS ? (int)rows : SMALL_MAX_ROWS;
}

// 16-byte slots of a workgroup: each wave's ring of spans of the weight (and of the rows, where none
// are held), then the held rows.
EXL3_I8_PLAN int small_slots(bool held) { return SMALL_WAVES * SMALL_RING * (held ? 1 : 2) * 256 + (held ? HELD_BLOCKS : 0); }
// Workgroups that a CU holds at once.
EXL3_I8_PLAN int small_per_cu(bool held) { return CU_LDS / (small_slots(held) * 16); }

// As many waves on a run of 16 outputs as the card holds at once, so that one round of workgroups
// starts up and quantises; where the rows are held and there is more than a round, two, as the
// last workgroups then have half as much to do (us: three tokens, two of eight experts each, 4096
// -> 14336 47.5 against 51.2, eight tokens 74.7 against 83.1; 4 waves 51.2 and 79.2).
EXL3_I8_PLAN int small_split(int64_t n_out, int64_t tiles, int n_in, bool held) {
    const int64_t resident = (int64_t)CUS * SMALL_WAVES * small_per_cu(held), runs = (n_out + 15) / 16;
    int split = 1;
    while (split < SMALL_WAVES && split < spans_of(n_in) && runs * tiles * split * 2 <= resident) split *= 2;
    return held && split == 1 && spans_of(n_in) >= 16 ? 2 : split;
}

// Rows that a group has on average, those behind the last group counted.
EXL3_I8_PLAN int64_t typical_rows(int64_t rows, int n_groups) { return (rows + n_groups - 1) / n_groups; }

// Does the product quantise its rows itself, without a launch and the codes' way through memory?
// Every workgroup does all of it, so few rows, and not for groups (us, with the quantisation: one row
// 4096 -> 4096 7.6 against 10.5, 14336 -> 4096 16.7 against 18.4; four rows 4096 -> 4096 10.4 against
// 10.9, 2048 -> 8192 9.2 against 11.9; eight rows 2048 -> 4096 11.4 against 10.0; six rows in eight
// groups 4096 -> 14336 55 against 50).
EXL3_I8_PLAN bool quantised_inside(int64_t rows, int n_groups, int n_in) {
    return n_groups == 1 && rows <= held_rows(n_in) && rows <= 4;
}

// ---- which kernel makes a product ----

constexpr int LARGE_COLS = 256;  // outputs of the largest tiles

struct ProductShape {
    bool grouped;
    int rows, n_groups, n_in, n_out;
};

// Row tiles of `high` rows that a product is expected to have: with groups, half a
// tile of each group (or row) is padding.
EXL3_I8_PLAN int64_t expected_tiles(const ProductShape& p, int high) {
    if (!p.grouped) return ((int64_t)p.rows + high - 1) / high;
    return p.rows / high + (p.n_groups < p.rows ? p.n_groups : p.rows) / 2 + 1;
}

// The time of a product in tiles, in us per 4096 inputs, by the rounds that 256 CUs take, as
// measured: 128 x 128 tiles 28 for one a CU and 39 for two at once; 128 x 256 36.7; 256 x 256 52.
EXL3_I8_PLAN double middle_time(const ProductShape& p) {
    const int64_t each = (expected_tiles(p, 128) * (((int64_t)p.n_out + 127) / 128) + CUS - 1) / CUS;
    return (double)(each / 2) * 39 + (double)(each % 2) * 28;
}
EXL3_I8_PLAN double large_time(const ProductShape& p, int rows, int64_t n_out) {
    const int64_t rounds = (expected_tiles(p, rows) * ((n_out + LARGE_COLS - 1) / LARGE_COLS) + CUS - 1) / CUS;
    return (double)rounds * (rows == 256 ? 52 : 36.7);
}

// small_kernel with held rows and with streamed ones, strips of 16, 32 and 64 outputs, 64 x 64 tiles in stages of
// 256 inputs and of 128, 128 x 128 tiles, 128 x 256, 256 x 256, and of these the first `cols` outputs with 128 x 256 for the rest.
enum ProductKernel { SMALL_STAGED, SMALL_STREAMED, STRIP_16, STRIP_32, STRIP_64, MEDIUM_LONG, MEDIUM_SHORT, MIDDLE, LARGE_128, LARGE_256, LARGE_BOTH };
struct ProductChoice {
    ProductKernel kernel;
    int cols;
};

// Rules by the average group, as the host doesn't know the route; times in us.
//
// Held rows: 128 rows in 64 groups 2048 -> 2816 52, streamed 62; 512 rows in 256 groups 1024 -> 1024 44 and 58; equal
// at as many rows as are held (8 a group 76.9 and 75.9).
// Streamed few-rows tiles while there is one of them a CU at most: against strips of 32 x 16 13 rows 14336 -> 4096 13.6 and
// 14.0, 64 rows 4096 -> 1024 5.1 and 6.0, 8192 -> 1024 6.3 and 8.9, but with more 17 rows 14336 -> 4096 16.7 and 14.3, 32 rows
// 20.0 and 16.9; against 32 x 32 ones 13 rows 4096 -> 6144 9.0 and 8.3; 32 rows in 8 groups 4096 -> 14336 101, in 64 x 64 tiles 91.
// Strips of 32 rows and 16, 32 or 64 outputs, the narrowest of which there is one a CU at most: 40 rows 4096 -> 4096 8.6, 7.4 and
// 9.3; 256 rows 4096 -> 1024 7.9, 6.5, 7.8; 128 rows 14336 -> 4096 44.3, 32.0, 26.9; 256 rows 4096 -> 2048 13.9, 9.1, 8.3; 64 x 64
// tiles instead of the last 35.3 and 11.9, but 160 rows 4096 -> 4096 (320 strips) 12.5 against 16.3.
// 64 x 64 tiles in stages of 256 inputs while there is one a CU, in stages of 128 where there are two: the latter
// against the former 512 rows 4096 -> 4096 20.5 and 23.1, 2048 rows 4096 -> 1024 17.1 and 22.6, but 256 rows
// 4096 -> 4096 14.3 and 12.7, 256 rows 14336 -> 4096 41.2 and 35.3.  128 x 128 ones beyond: 768 rows 4096 -> 4096
// 28.8, 64 x 64 ones 33.4.  Groups of up to 32 rows, which the weights' way from memory bounds, stay with 64 x 64 ones, two
// a CU: 2048 rows in 64 groups 2048 -> 2816 75.6, in 128 x 128 tiles 79.2, 128 x 256 77.9; 256 rows in 8 groups 4096 -> 14336 95.3, 115.6,
// 114.7; groups of 64 rows 116, 111 in 128 x 256 tiles.
// 128 x 128, 128 x 256 and 256 x 256 by the rounds that they take (the times above): 768 rows 4096 -> 4096 28.8, 31.5,
// 44.9; 2048 rows 38.9, 34.8, 46.5; 4096 rows 74, 67, 54; 1000 rows 4096 -> 28672 133, 126, 102; 8192^3 508, 465, 384; 16384 rows
// in 64 groups 2048 -> 2816 159, 143, 155.
// Whole rounds of 256 x 256 and the rest in 128 x 256 tiles: 2048 rows 8192 -> 28672 359, all of them large 366; only
// where it saves 5 %, for the second launch.
EXL3_I8_PLAN ProductChoice choose_product(const ProductShape& p) {
    const int64_t m = typical_rows(p.rows, p.n_groups), runs = ((int64_t)p.n_out + 15) / 16;
    if (p.grouped ? m < held_rows(p.n_in) : m <= held_rows(p.n_in)) return {SMALL_STAGED, 0};
    if (expected_tiles(p, 16) * runs <= CUS) return {SMALL_STREAMED, 0};
    if (expected_tiles(p, 32) * runs <= CUS) return {STRIP_16, 0};
    if (expected_tiles(p, 32) * (((int64_t)p.n_out + 31) / 32) <= CUS) return {STRIP_32, 0};
    const int64_t cols64 = ((int64_t)p.n_out + 63) / 64;
    if (expected_tiles(p, 32) * cols64 <= CUS) return {STRIP_64, 0};
    const int64_t tiles = expected_tiles(p, 64) * cols64;
    if (tiles <= CUS) return {MEDIUM_LONG, 0};
    if (tiles <= 2 * CUS || (p.grouped && m <= 32)) return {MEDIUM_SHORT, 0};
    const double middle = middle_time(p), low = large_time(p, 128, p.n_out), high = large_time(p, 256, p.n_out);
    // Whole rounds of 256 x 256 tiles, and 128 x 256 ones for the columns left over.
    const int64_t row_tiles = expected_tiles(p, 256), whole = row_tiles * (((int64_t)p.n_out + LARGE_COLS - 1) / LARGE_COLS) / CUS;
    const int64_t cols = whole * CUS / row_tiles * LARGE_COLS;
    if (!p.grouped && cols > 0 && cols < p.n_out) {
        const double both = large_time(p, 256, cols) + large_time(p, 128, p.n_out - cols);
        if (both < 0.95 * high && both < low && both < middle) return {LARGE_BOTH, (int)cols};
    }
    if (middle <= low && middle < high) return {MIDDLE, 0};
    return {low < high ? LARGE_128 : LARGE_256, 0};
}

}  // namespace i8
}  // namespace exl3
