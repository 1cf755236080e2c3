// slots.hpp - a token's slots, shared out over the lanes that hold its logits (host and
// device, no HIP in it).
#pragma once
#include <stdint.h>

#ifdef __HIPCC__
#define EXL3_SLOTS __host__ __device__ inline
#else
#define EXL3_SLOTS inline
#endif

namespace exl3 {

// Lane `lane` of LANES takes slots lane, lane + LANES, ... of a token's top_k: the first, `id`, is there
// already (-1: none), load(j) brings slot j.
template <int LANES, typename LOAD, typename TAKE> EXL3_SLOTS void lane_slots(int top_k, int lane, int64_t id, LOAD load, TAKE take) {
    // By what is left, as the number of a slot behind the last may not fit 32 bits: 2^31 - 1 are allowed.
    for (int left = top_k - lane;;) {
        take(id);
        left -= LANES;
        if (left <= 0) break;
        id = load(top_k - left);
    }
}

}  // namespace exl3
