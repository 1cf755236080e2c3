// mxfp4_plan.hpp - how the few-rows product is laid out and split (host and device,
// no HIP in it).
#pragma once
#include <stdint.h>

#ifdef __HIPCC__
#define EXL3_PLAN __host__ __device__ constexpr
#else
#define EXL3_PLAN constexpr
#endif

namespace exl3 {
namespace mx {

constexpr int BLOCK = 32;        // values per scale
constexpr int SPAN_BLOCKS = 16;  // blocks per span
constexpr int CUS = 256, CU_LDS = 160 * 1024;

constexpr int SMALL_WAVES = 8, SMALL_RING = 2, SMALL_MAX_ROWS = 16;
constexpr int HELD_SPANS = 32, MORE_HELD_SPANS = 64;

EXL3_PLAN int64_t spans_of(int n_in) { return ((int64_t)n_in + SPAN_BLOCKS * BLOCK - 1) / (SPAN_BLOCKS * BLOCK); }

// Rows of a tile that holds `spans` spans of them (0: none fits).
EXL3_PLAN int held_rows(int n_in, int spans) {
    const int rows = spans / (int)spans_of(n_in);
    return rows < SMALL_MAX_ROWS ? rows : SMALL_MAX_ROWS;
}

// Dwords of scales that a row of a span holds in LDS: its 16 bytes, or where rows
// start at any byte (not `whole`: n_in % 128 != 0) the aligned dwords that 16 bytes
// can touch.
EXL3_PLAN int small_scale_dwords(bool whole) { return whole ? 4 : 5; }
// 16-byte slots of a wave's span: the weight's codes and scales, and where no rows
// are held the rows' as well.
EXL3_PLAN int small_buf_slots(int held, bool whole) { return (held ? 1 : 2) * (16 * 16 + 4 * small_scale_dwords(whole)); }
// 16-byte slots of a workgroup: the waves' rings, then the held rows' codes and scales.
EXL3_PLAN int small_slots(int held, bool whole) { return SMALL_WAVES * SMALL_RING * small_buf_slots(held, whole) + held * 17; }
// Workgroups that a CU holds at once.
EXL3_PLAN int small_per_cu(int held, bool whole) { return CU_LDS / (small_slots(held, whole) * 16); }

// As many waves on a run of 16 outputs as the card holds at once, so that one round
// of workgroups starts up and quantises.
EXL3_PLAN int small_split(int64_t n_out, int64_t tiles, int n_in, int held) {
    const int64_t resident = (int64_t)CUS * SMALL_WAVES * small_per_cu(held, n_in % (4 * BLOCK) == 0), runs = (n_out + 15) / 16;
    int split = 1;
    while (split < SMALL_WAVES && split < spans_of(n_in) && runs * tiles * split * 2 <= resident) split *= 2;
    return split;
}

}  // namespace mx
}  // namespace exl3
