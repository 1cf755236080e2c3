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

// Rules by the average group, as the host doesn't know the route; times in us, of one series of runs with the
// weights of several products in turn.
//
// Held rows: 128 rows in 64 groups 2048 -> 2816 55, streamed 64; 512 rows in 256 groups 1024 -> 1024 44 and 59; but as many a
// group as are held (8, 2048 -> 2816) 79, 64 x 64 tiles 69.
// Streamed few-rows tiles while there is one of them a CU at most: against strips of 32 x 16 13 rows 14336 -> 4096 13.6 and
// 13.9, 64 rows 4096 -> 1024 5.2 and 6.2, 8192 -> 1024 6.4 and 9.0, but with more 17 rows 14336 -> 4096 16.6 and 14.1, 32 rows
// 20.0 and 16.7.  Up to 16 rows of more outputs take strips as well: 16 rows 8192 -> 8192 15.1, streamed 16.4, 28672 -> 5120 36.6 and
// 40.3, 4096 -> 28672 26.2 and 29.5, though a few of them 28672 -> 8192 44.3 and 42.2, 28672 -> 16384 91 and 84, 13 rows 4096 -> 6144
// 7.5 and 7.3.
// Strips of 32 rows and 16, 32 or 64 outputs, the narrowest of which there is one a CU at most: 40 rows 4096 -> 4096 7.9, 6.7 and
// 7.9; 256 rows 4096 -> 1024 8.1, 6.6, 7.9; 128 rows 14336 -> 4096 44.0, 31.8, 26.8; 256 rows 4096 -> 2048 14.1, 9.3, 8.0; 64 x 64
// tiles instead of the last 35.0 and 12.0, but 160 rows 4096 -> 4096 (320 strips) 12.2 against 14.7.
// Beyond, few rows of long inputs keep to 32 x 32 strips, as larger tiles are slower for rows that are not there: up to 16
// of one weight from 4096 inputs on, against 64 x 64 and 128 x 256 tiles 16 rows 4096 -> 128256 97, 99 and 121, 4096 -> 40000 37, 40 and
// 44, two rows 20480 -> 20480 84 and 105 (16 rows 14336 -> 28672 77, 75 in the former; of 2048 inputs -> 28672 15.9 and 13.7); up to 8 a
// group from 8192 on, 16 rows in 8 groups 14336 -> 4096 67 and 72, 32 76.6 and 78.2.  More a group are faster in strips where
// they are shared out evenly (200 in 16 8192 -> 4096 92 and 102), but not where a few groups have them all (28 and 25 in two of the 16); shorter
// inputs are as fast (1024 in 64 groups 4096 -> 2048 101 and 102; 38 and 21 in four of the 64) or slower (384 in 64 2816 -> 2048 74 and 67).
// 64 x 64 tiles in stages of 256 inputs while there is one a CU, in stages of 128 where there are two: the latter
// against the former 512 rows 4096 -> 4096 16.9 and 22.7, 2048 rows 4096 -> 1024 16.9 and 22.7, but 256 rows
// 4096 -> 4096 13.8 and 12.2, 256 rows 14336 -> 4096 40.9 and 34.9.  128 x 128 ones beyond: 768 rows 4096 -> 4096
// 26.4, 64 x 64 ones 27.0.  Groups of up to 32 rows, which the weights' way from memory bounds, stay with 64 x 64 ones, two
// a CU: 2048 rows in 64 groups 2048 -> 2816 75.6, in 128 x 128 tiles 79.3, 128 x 256 77.6; 256 rows in 8 groups 4096 -> 14336 93.0, 110,
// 108; groups of 64 rows 97, 83.5 in 128 x 256 tiles.
// 128 x 128, 128 x 256 and 256 x 256 by the rounds that they take (the times above): 768 rows 4096 -> 4096 26.4, 28.6,
// 41.5; 2048 rows 36.9, 33.9, 41.1; 4096 rows 74, 66, 54; 1000 rows 4096 -> 28672 137, 127, 104; 8192^3 545, 477, 391; 16384 rows
// in 64 groups 2048 -> 2816 162, 150, 154.
// Whole rounds of 256 x 256 and the rest in 128 x 256 tiles: 2048 rows 8192 -> 28672 372, all of them large 377; only
// where it saves 5 % by these times, for the second launch.
EXL3_I8_PLAN ProductChoice choose_product(const ProductShape& p) {
    const int64_t m = typical_rows(p.rows, p.n_groups), runs = ((int64_t)p.n_out + 15) / 16;
    if (p.grouped ? m < held_rows(p.n_in) : m <= held_rows(p.n_in)) return {SMALL_STAGED, 0};
    if (expected_tiles(p, 16) * runs <= CUS) return {SMALL_STREAMED, 0};
    if (expected_tiles(p, 32) * runs <= CUS) return {STRIP_16, 0};
    const int64_t strips = expected_tiles(p, 32) * (((int64_t)p.n_out + 31) / 32), cols64 = ((int64_t)p.n_out + 63) / 64;
    if (strips <= CUS) return {STRIP_32, 0};
    if (expected_tiles(p, 32) * cols64 <= CUS) return {STRIP_64, 0};
    // (a launch takes 2^24 workgroups, and there may be twice the tiles that are expected)
    if (m <= (p.grouped ? 8 : 16) && p.n_in >= (p.grouped ? 8192 : 4096) && strips < (1 << 22)) return {STRIP_32, 0};
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
