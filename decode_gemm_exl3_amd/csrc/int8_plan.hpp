// int8_plan.hpp - how the few-rows product of 8-bit rows is laid out and split (host and
// device, no HIP in it).
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

}  // namespace i8
}  // namespace exl3
