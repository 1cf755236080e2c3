// balance.hip - the loss that evens out a router's experts, their counts and the
// gradient to the logits (gfx950).
//
// With p_t the softmax of token t's logits, V the tokens that keep at least one of their k slots, c_e the kept
// slots of expert e and E experts:
//   loss = coefficient E sum_e c_e / (V k) * P_e,  P_e = 1 / V sum_t p_te over those tokens,
//   dlogits_te = dloss coefficient E / V * p_te (s_e - sum_f p_tf s_f),  s_e = c_e / (V k),
// as counts have no gradient.  One pass over the logits each way: the loss's first launch leaves each workgroup's
// sums and counts, its second adds them up; the backward pass makes the probabilities again, as reading
// them back would cost more than their exponentials.
#include <hip/hip_runtime.h>

#include "../../include/exl3_balance.h"
#include "lanes_device.hpp"
#include "pieces_device.hpp"
#include "slots.hpp"
#include "spans.hpp"

namespace exl3 {
namespace balance {

using namespace mx;  // element types, pieces

struct Params {
    const void* logits;
    const void* ids;
    int id_bytes, tokens, top_k, experts;
    double coefficient;
    int blocks;        // workgroups of the loss's first launch
    float* part;       // [blocks][experts]: sums of probabilities
    int* part_counts;  // [blocks][experts + 1]
    uint64_t* along;   // of the second launch's workgroups: counts times sums, as fp64
    int* arrived;      // how many of them are done
    float* loss;
    int* counts;
    const float* dloss;
    void* dlogits;
};

constexpr int SUM_THREADS = 1024, FINAL_THREADS = 1024, BACKWARD_THREADS = 256;
constexpr int MAX_BLOCKS = 256;          // workgroups of the loss's first launch
constexpr int FINAL_EXPERTS = 64;        // experts of a workgroup of its second

// A token's logits lie in LANES lanes (a power of two), Q pieces of N = 16 bytes each:
// piece q of lane l is columns (q * LANES + l) * N and on.  A wave holds 64 / LANES tokens.
// LANES * Q * N >= experts.

// 16 bytes of a row, or what is left of it.  Rows that are no whole pieces (VEC false) start at any
// value: unaligned loads and stores.
template <typename T, bool VEC> __device__ inline u32x4_t load_columns(const void* base, int64_t at, int left) {
    if constexpr (VEC) return load_piece<T, true>(base, at, left);
    if (left < 16 / T::bytes) return load_piece<T, false>(base, at, left);
    u32x4_t r;
    __builtin_memcpy(&r, static_cast<const char*>(base) + at * T::bytes, 16);
    return r;
}
template <typename T, bool VEC> __device__ inline void store_columns(void* base, int64_t at, int left, const u32x4_t r) {
    if constexpr (VEC) return store_piece<T, true, false>(base, at, left, r);
    if (left < 16 / T::bytes) return store_piece<T, false, false>(base, at, left, r);
    __builtin_memcpy(static_cast<char*>(base) + at * T::bytes, &r, 16);
}

// 4 bytes of -infinity.
template <typename T> constexpr uint32_t LOWEST = 0xFF800000u;
template <> constexpr uint32_t LOWEST<F16> = 0xFC00FC00u;
template <> constexpr uint32_t LOWEST<BF16> = 0xFF80FF80u;

// What a lane asks for of a token: its pieces of the logits, and the token's slot `lane`.
template <int Q> struct Asked {
    u32x4_t piece[Q];
    int64_t id;
};
__device__ inline int64_t load_id(const Params& p, int64_t at) {
    return p.id_bytes == 8 ? static_cast<const int64_t*>(p.ids)[at] : (int64_t) static_cast<const int*>(p.ids)[at];
}
template <typename T, int LANES, int Q, bool VEC> __device__ inline Asked<Q> ask(const Params& p, int token, int lane) {
    constexpr int N = 16 / T::bytes;
    Asked<Q> r;
    r.id = -1;
    if (token < p.tokens && lane < p.top_k) r.id = load_id(p, (int64_t)token * p.top_k + lane);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int c = (q * LANES + lane) * N;
        r.piece[q] = u32x4_t{LOWEST<T>, LOWEST<T>, LOWEST<T>, LOWEST<T>};  // columns behind the last
        if (token < p.tokens && c < p.experts) r.piece[q] = load_columns<T, VEC>(p.logits, (int64_t)token * p.experts + c, p.experts - c);
    }
    return r;
}

// Does the token have a slot that is kept?  All lanes of the wave come here; lanes of a
// token share its slots out.  COUNT: kept slots go into the histogram.
template <int LANES, bool COUNT> __device__ inline bool counts_token(const Params& p, int token, int64_t id, int lane, int* hist) {
    bool kept = false;
    lane_slots<LANES>(token < p.tokens ? p.top_k : 0, lane, id, [&](int j) { return load_id(p, (int64_t)token * p.top_k + j); }, [&](int64_t at) {
        if (at >= 0 && at < p.experts) {
            kept = true;
            if (COUNT) atomicAdd(&hist[(int)at], 1);
        }
    });
    if constexpr (LANES == 1) return kept;
    const uint64_t all = __ballot(kept);
    if constexpr (LANES == 64) return all != 0;
    const int first = (threadIdx.x & 63) / LANES * LANES;
    return ((all >> first) & ((1ull << (LANES & 63)) - 1)) != 0;
}

constexpr float INV_LN2 = 1.44269502f, INV_LN2_LOW = 1.92596299e-8f, LN2 = 0.693147182f;  // 1 / ln 2 in two parts

// e^d of d <= 0 to a step of fp32: 2^y with y = fl(d / ln 2), which is off by up to its own size times 2^-24,
// times 1 + (d / ln 2 - y) ln 2; 0 from 2^-126 (d = -87.3) down, as the instruction makes no subnormal numbers, which
// the 16-bit way below does neither.  (The largest of -104 keeps -infinity from becoming a NaN.)
__device__ inline float exp_below(float d) {
    d = fmaxf(d, -104.f);
    const float y = d * INV_LN2, e = __builtin_amdgcn_exp2f(y);
    const float rest = __builtin_fmaf(d, INV_LN2_LOW, __builtin_fmaf(d, INV_LN2, -y));
    return __builtin_fmaf(e * LN2, rest, e);
}

// The softmax of a token's logits: v times the result are the probabilities of this lane's columns, v
// is 0 behind the last.  VEC: pieces behind the last column hold -infinity, others lie whole before it.
//
// For 16-bit logits v = 2^y, y = fl(x / ln 2 - K) in one step, K the largest x / ln 2 rounded, which
// all of a token's v share: what K is off by cancels.  y is off by its own size times 2^-24, a relative
// 0.85 |y| 2^-24 of v: less than a tenth of a step of the gradients' types, and of the loss that far down (v
// = e^-10) 7e-7 a token.  (Four instructions more for fp32 logits, above.)  Largest logits of 2^20 and more,
// whose K is off by much, take the difference first.
template <typename T, bool VEC, int LANES, int Q> __device__ inline float softmax(const Params& p, const u32x4_t (&piece)[Q], int lane, float (&v)[Q][16 / T::bytes]) {
    constexpr int N = 16 / T::bytes;
    const float lowest = -__builtin_inff();
    float top = lowest;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[q][i] = VEC || (q * LANES + lane) * N + i < p.experts ? piece_value<T>(piece[q], i) : lowest;
            top = __builtin_elementwise_maximum(top, v[q][i]);  // a NaN stays one
        }
    top = over_lanes<LANES>(top, [](float a, float b) { return __builtin_elementwise_maximum(a, b); });
    const bool bad = !(top < __builtin_inff());  // a NaN or +infinity: all of the token's are NaN
    if (top == lowest) top = 0.f;                // nothing but -infinity: exp gives zeros
    float sum = 0.f;
    if (T::bytes == 2 && fabsf(top) < 0x1p20f) {
        const float k = top * INV_LN2;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i) v[q][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[q][i], INV_LN2, -k));
    } else {
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i) v[q][i] = exp_below(v[q][i] - top);
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) sum += v[q][i];
    sum = over_lanes<LANES>(sum, [](float a, float b) { return a + b; });
    // 1 / sum to a step of fp32: an estimate and one step of Newton's
    const float guess = __builtin_amdgcn_rcpf(sum), newton = __builtin_fmaf(__builtin_fmaf(-sum, guess, 1.f), guess, guess);
    return bad ? __builtin_nanf("") : sum == 0.f ? 0.f : newton;
}

// The loss, `along` the sum over the experts of count times sum of probabilities.
__device__ inline float loss_of(const Params& p, int tokens, double along) {
    if (tokens == 0) return 0.f;
    const double of = tokens;
    return (float)(p.coefficient * p.experts * along / (of * of * p.top_k));
}

// Sum over the threads of a workgroup, in each of them.
template <int COUNT> __device__ inline double block_sum(double v) {
    __shared__ double part[COUNT / 64];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    __syncthreads();  // a sum before this one is read
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < COUNT / 64; ++w) v += part[w];
    return v;
}

// Sums of probabilities and counts of the tokens of a workgroup: each lane adds up its
// columns over the wave's tokens in registers; the next token's logits and slots are on their
// way meanwhile.  One workgroup alone writes the results.
//
// 32768 tokens of 256 experts, 8 slots (18 MB of bf16 logits and ids, 3.6 us at a large copy's rate), take 8.8 us. The
// vector units are busy 0.61 of that, 5 us, with exponentials, sums and lane exchanges; the rest is the start, the first tokens'
// way from memory and the joins, which nothing covers (the waves wait 0.63 of their time).  16 waves a workgroup, so that a CU
// has enough to issue.
template <typename T, int LANES, int Q, bool VEC> __global__ __launch_bounds__(SUM_THREADS) void sum_kernel(const Params p) {
    constexpr int N = 16 / T::bytes, EACH = 64 / LANES, WAVES = SUM_THREADS / 64;
    __shared__ int hist[EXL3_MOE_MAX_EXPERTS + 1];
    __shared__ float sums[WAVES][LANES * Q * N];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & (LANES - 1), slot = (threadIdx.x & 63) / LANES;
    const int step = p.blocks * WAVES * EACH;
    int t0 = (blockIdx.x * WAVES + wave) * EACH;
    Asked<Q> next = ask<T, LANES, Q, VEC>(p, t0 + slot, lane);
    for (int e = threadIdx.x; e <= p.experts; e += SUM_THREADS) hist[e] = 0;
    if (blockIdx.x == 0 && threadIdx.x == 0 && p.blocks > 1) *p.arrived = 0;
    __syncthreads();
    float acc[Q][N];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[q][i] = 0.f;
    for (; t0 < p.tokens; t0 += step) {
        const Asked<Q> now = next;
        next = ask<T, LANES, Q, VEC>(p, t0 + step + slot, lane);
        const bool valid = counts_token<LANES, true>(p, t0 + slot, now.id, lane, hist);
        float v[Q][N];
        const float inverse = softmax<T, VEC, LANES, Q>(p, now.piece, lane, v);
        if (valid) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[q][i] = __builtin_fmaf(v[q][i], inverse, acc[q][i]);
            if (lane == 0) atomicAdd(&hist[p.experts], 1);
        }
    }
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) {
#pragma unroll
            for (int d = LANES; d < 64; d *= 2) acc[q][i] += __shfl_xor(acc[q][i], d);
            if (slot == 0) sums[wave][(q * LANES + lane) * N + i] = acc[q][i];
        }
    __syncthreads();
    double along = 0.0;
    for (int e = threadIdx.x; e < p.experts; e += SUM_THREADS) {
        float s = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) s += sums[w][e];
        if (p.blocks > 1) {
            p.part[(int64_t)blockIdx.x * p.experts + e] = s;
            p.part_counts[(int64_t)blockIdx.x * (p.experts + 1) + e] = hist[e];
        } else {
            along += (double)hist[e] * s;
            p.counts[e] = hist[e];
        }
    }
    if (p.blocks > 1) {
        if (threadIdx.x == 0) p.part_counts[(int64_t)blockIdx.x * (p.experts + 1) + p.experts] = hist[p.experts];
        return;
    }
    along = block_sum<SUM_THREADS>(along);
    if (threadIdx.x == 0) {
        p.counts[p.experts] = hist[p.experts];
        *p.loss = loss_of(p, hist[p.experts], along);
    }
}

// The workgroups' sums to the loss and the counts: a workgroup takes 64 experts, 16 threads each.
// The last one to arrive adds up what they made, in their order.  Latency bounds it: of 256 workgroups' sums of 256
// experts 7.4 us in four workgroups, whose waves wait 0.77 of their time, for the sums' way between XCDs and the arrivals'.
__global__ __launch_bounds__(FINAL_THREADS) void loss_kernel(const Params p) {
    constexpr int SLICES = FINAL_THREADS / FINAL_EXPERTS, EACH = MAX_BLOCKS / SLICES;
    static_assert(FINAL_EXPERTS == 64 && EXL3_MOE_MAX_EXPERTS / FINAL_EXPERTS <= 16, "an expert a lane, and a workgroup of 16");
    __shared__ float sums[SLICES][FINAL_EXPERTS];
    __shared__ int counts[SLICES][FINAL_EXPERTS];
    __shared__ int tokens;
    __shared__ bool last;
    __shared__ double sum_of_all;
    const int lane = threadIdx.x & 63, k = threadIdx.x >> 6, e = blockIdx.x * FINAL_EXPERTS + lane;
    const int groups = (p.experts + FINAL_EXPERTS - 1) / FINAL_EXPERTS;  // workgroups
    if (threadIdx.x == 0) tokens = 0;
    float part[EACH];
    int part_counts[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int b = k + i * SLICES;
        const bool in = e < p.experts && b < p.blocks;
        part[i] = in ? p.part[(int64_t)b * p.experts + e] : 0.f;
        part_counts[i] = in ? p.part_counts[(int64_t)b * (p.experts + 1) + e] : 0;
    }
    const int mine = threadIdx.x < p.blocks ? p.part_counts[(int64_t)threadIdx.x * (p.experts + 1) + p.experts] : 0;  // tokens
    float s = 0.f;
    int c = 0;
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        s += part[i];
        c += part_counts[i];
    }
    sums[k][lane] = s;
    counts[k][lane] = c;
    __syncthreads();
    if (mine) atomicAdd(&tokens, mine);
    if (threadIdx.x < 64) {
        s = 0.f;
        c = 0;
#pragma unroll
        for (int i = 0; i < SLICES; ++i) {
            s += sums[i][lane];
            c += counts[i][lane];
        }
        if (e < p.experts) p.counts[e] = c;
        double along = over_lanes<64>((double)c * s, [](double a, double b) { return a + b; });
        if (threadIdx.x == 0) {
            last = true;
            if (groups > 1) {
                __hip_atomic_store(&p.along[blockIdx.x], __builtin_bit_cast(uint64_t, along), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
                // The store has reached what all XCDs see before the arrival does: it is atomic itself, so a
                // wait for it is enough, without the write-back of the L2 that a release would add.
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
                last = __hip_atomic_fetch_add(p.arrived, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == groups - 1;
            }
        }
        if (groups > 1 && __builtin_amdgcn_readfirstlane(last)) {
            along = 0.0;
            if (lane < groups)
                along = __builtin_bit_cast(double, __hip_atomic_load(&p.along[threadIdx.x], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT));
            along = over_lanes<16>(along, [](double a, double b) { return a + b; });
        }
        if (lane == 0) sum_of_all = along;
    }
    __syncthreads();
    if (threadIdx.x == 0 && last) {
        p.counts[p.experts] = tokens;
        *p.loss = loss_of(p, tokens, sum_of_all);
    }
}

// dlogits: the shares of this lane's columns stay in registers over all its tokens.  They are taken less their mean, which
// s_e - sum_f p_f s_f does not see as probabilities sum to one: what rounding leaves of that sum then counts by the shares'
// differences, not by the shares, and a router whose experts have as many slots each has no gradient at all.  32768 tokens of 256 experts
// (35 MB, 6.9 us at a large copy's rate) take 14.1 us: the vector units are busy 0.54 of it, 7 us, and memory about as long; the
// two overlap little, as a wave has few tokens and only the next one on its way.  Up to 1024 workgroups: with 512 14.5 us in a graph,
// 1024 13.1, 2048 16.2.
template <typename T, int LANES, int Q, bool VEC> __global__ __launch_bounds__(BACKWARD_THREADS) void backward_kernel(const Params p) {
    constexpr int N = 16 / T::bytes, EACH = 64 / LANES, WAVES = BACKWARD_THREADS / 64;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & (LANES - 1), slot = (threadIdx.x & 63) / LANES;
    const int step = gridDim.x * WAVES * EACH;
    int t0 = (blockIdx.x * WAVES + wave) * EACH;
    Asked<Q> next = ask<T, LANES, Q, VEC>(p, t0 + slot, lane);
    int counts[Q][N];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (q * LANES + lane) * N + i;
            counts[q][i] = c < p.experts ? p.counts[c] : 0;
        }
    const int tokens = p.counts[p.experts];
    uint32_t kept = 0;  // below 2^31, as slots are
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) kept += counts[q][i];
    kept = over_lanes<LANES>(kept, [](uint32_t a, uint32_t b) { return a + b; });
    const double of = tokens > 0 ? tokens : 1, each = 1.0 / (of * p.top_k * p.experts);
    const float factor = (float)(*p.dloss * p.coefficient * (p.experts / of));
    float share[Q][N];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (q * LANES + lane) * N + i;
            share[q][i] = c < p.experts ? (float)((double)((int64_t)counts[q][i] * p.experts - kept) * each) : 0.f;
        }
    for (; t0 < p.tokens; t0 += step) {
        const int token = t0 + slot;
        const Asked<Q> now = next;
        next = ask<T, LANES, Q, VEC>(p, token + step, lane);
        const bool valid = counts_token<LANES, false>(p, token, now.id, lane, nullptr);
        float v[Q][N];
        const float inverse = softmax<T, VEC, LANES, Q>(p, now.piece, lane, v);
        float along = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i) along = __builtin_fmaf(v[q][i], share[q][i], along);
        along = over_lanes<LANES>(along, [](float a, float b) { return a + b; }) * inverse * inverse;
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = (q * LANES + lane) * N;
            float g[N];
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = factor * (v[q][i] * __builtin_fmaf(share[q][i], inverse, -along));
            if (token < p.tokens && c < p.experts) store_columns<T, VEC>(p.dlogits, (int64_t)token * p.experts + c, p.experts - c, valid ? round_piece<T>(g) : u32x4_t{0, 0, 0, 0});
        }
    }
}

// ---- launches ----

enum Op { LOSS, BACKWARD };

template <typename T, int LANES, int Q, bool VEC> hipError_t launch(Op op, const Params& p, hipStream_t s) {
    if (op == LOSS) {
        sum_kernel<T, LANES, Q, VEC><<<p.blocks, SUM_THREADS, 0, s>>>(p);
    } else {
        constexpr int EACH = BACKWARD_THREADS / LANES;
        const int64_t blocks = ((int64_t)p.tokens + EACH - 1) / EACH;
        backward_kernel<T, LANES, Q, VEC><<<(unsigned)(blocks < 1024 ? blocks : 1024), BACKWARD_THREADS, 0, s>>>(p);
    }
    return hipGetLastError();
}

template <typename T, bool VEC> hipError_t launch(Op op, const Params& p, hipStream_t s) {
    const int pieces = (p.experts * T::bytes + 15) / 16;
    if (pieces <= 1) return launch<T, 1, 1, VEC>(op, p, s);
    if (pieces <= 2) return launch<T, 2, 1, VEC>(op, p, s);
    if (pieces <= 4) return launch<T, 4, 1, VEC>(op, p, s);
    if (pieces <= 8) return launch<T, 8, 1, VEC>(op, p, s);
    if (pieces <= 16) return launch<T, 16, 1, VEC>(op, p, s);
    if (pieces <= 32) return launch<T, 32, 1, VEC>(op, p, s);
    if (pieces <= 64) return launch<T, 64, 1, VEC>(op, p, s);
    if (pieces <= 128) return launch<T, 64, 2, VEC>(op, p, s);
    if constexpr (T::bytes == 4) return launch<T, 64, 4, VEC>(op, p, s);
    return hipErrorInvalidValue;  // not reached: 1024 experts of 2 bytes are 128 pieces
}

template <typename T> hipError_t launch(Op op, const Params& p, hipStream_t s) {
    return p.experts * T::bytes % 16 == 0 ? launch<T, true>(op, p, s) : launch<T, false>(op, p, s);
}

hipError_t launch(int dtype, Op op, const Params& p, hipStream_t s) {
    switch (dtype) {
        case EXL3_F16: return launch<F16>(op, p, s);
        case EXL3_BF16: return launch<BF16>(op, p, s);
        default: return launch<F32>(op, p, s);
    }
}

// Workgroups of the first launch: one for few logits, else one for each 64 KB of fp32 logits, at most MAX_BLOCKS.
int plan_blocks(int tokens, int experts) {
    const int64_t blocks = ((int64_t)tokens * experts + 16383) / 16384;
    return blocks < 1 ? 1 : blocks > MAX_BLOCKS ? MAX_BLOCKS : (int)blocks;
}

bool misaligned(const void* ptr, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0; }
int64_t value_bytes(int dtype) { return dtype == EXL3_F32 ? 4 : 2; }
int64_t padded(int64_t bytes) { return (bytes + 255) & ~int64_t(255); }
int final_blocks(int experts) { return (experts + FINAL_EXPERTS - 1) / FINAL_EXPERTS; }
// The workspace's parts, one after the other: part, part_counts, along, arrived.
struct Parts {
    int64_t counts, along, arrived, bytes;
};
Parts parts(int blocks, int experts) {
    Parts w;
    w.counts = padded((int64_t)blocks * experts * 4);
    w.along = w.counts + padded((int64_t)blocks * (experts + 1) * 4);
    w.arrived = w.along + padded((int64_t)final_blocks(experts) * 8);
    w.bytes = w.arrived + 256;
    return w;
}

// Checks shared by both directions: <= 0 is the call's status.
int checks(const void* logits, int32_t dtype, const void* ids, int32_t id_bytes, int32_t n_tokens, int32_t top_k, int32_t n_experts,
           double coefficient) {
    if (dtype < EXL3_F16 || dtype > EXL3_F32 || (id_bytes != 4 && id_bytes != 8) || n_tokens < 0 || top_k < 1) return EXL3_EINVAL;
    if (n_experts < 1 || n_experts > EXL3_MOE_MAX_EXPERTS || !__builtin_isfinite(coefficient)) return EXL3_EINVAL;
    if (n_tokens > 0 && (!logits || !ids || misaligned(logits) || misaligned(ids))) return EXL3_EINVAL;
    if (n_tokens >= (1 << 24) || (int64_t)n_tokens * top_k > INT32_MAX) return EXL3_EUNSUPPORTED;
    return 1;
}

}  // namespace balance
}  // namespace exl3

extern "C" {

using exl3::apart;
using namespace exl3::balance;

int64_t exl3_moe_balance_workspace_bytes(int32_t n_tokens, int32_t n_experts) {
    if (n_tokens < 0 || n_experts < 1 || n_experts > EXL3_MOE_MAX_EXPERTS) return EXL3_EINVAL;
    const int blocks = plan_blocks(n_tokens, n_experts);
    return blocks == 1 ? 0 : parts(blocks, n_experts).bytes;
}

int exl3_moe_balance_loss(const void* logits, int32_t dtype, const void* ids, int32_t id_bytes, int32_t n_tokens,
                          int32_t top_k, int32_t n_experts, double coefficient, float* loss, int32_t* counts,
                          void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = checks(logits, dtype, ids, id_bytes, n_tokens, top_k, n_experts, coefficient);
    if (rc <= 0) return rc;
    if (!loss || !counts || misaligned(loss, 4) || misaligned(counts) || misaligned(workspace)) return EXL3_EINVAL;
    const int64_t need = exl3_moe_balance_workspace_bytes(n_tokens, n_experts), tokens = n_tokens;
    if (need > 0 && (!workspace || (int64_t)workspace_bytes < need)) return EXL3_EWORKSPACE;
    if (!apart({{loss, 4}, {counts, 4 * ((int64_t)n_experts + 1)}, {workspace, need}},
               {{logits, tokens * n_experts * value_bytes(dtype)}, {ids, tokens * top_k * id_bytes}}))
        return EXL3_EINVAL;
    const int blocks = plan_blocks(n_tokens, n_experts);
    char* const ws = static_cast<char*>(workspace);
    const Parts w = parts(blocks, n_experts);
    Params p = {logits, ids, id_bytes, n_tokens, top_k, n_experts, coefficient, blocks};
    p.loss = loss;
    p.counts = counts;
    if (blocks > 1) {
        p.part = reinterpret_cast<float*>(ws);
        p.part_counts = reinterpret_cast<int*>(ws + w.counts);
        p.along = reinterpret_cast<uint64_t*>(ws + w.along);
        p.arrived = reinterpret_cast<int*>(ws + w.arrived);
    }
    hipStream_t s = (hipStream_t)stream;
    if (launch(dtype, LOSS, p, s) != hipSuccess) return EXL3_EHIP;
    if (blocks > 1) loss_kernel<<<final_blocks(n_experts), FINAL_THREADS, 0, s>>>(p);
    return hipGetLastError() == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_moe_balance_loss_backward(const float* dloss, const void* logits, int32_t dtype, const void* ids,
                                   int32_t id_bytes, int32_t n_tokens, int32_t top_k, int32_t n_experts,
                                   const int32_t* counts, double coefficient, void* dlogits, void* stream) {
    const int rc = checks(logits, dtype, ids, id_bytes, n_tokens, top_k, n_experts, coefficient);
    if (rc <= 0) return rc;
    if (n_tokens == 0) return EXL3_OK;
    if (!dloss || !counts || !dlogits || misaligned(dloss, 4) || misaligned(counts) || misaligned(dlogits)) return EXL3_EINVAL;
    const int64_t size = (int64_t)n_tokens * n_experts * value_bytes(dtype);
    if (!apart({{dlogits, size}}, {{logits, size}, {ids, (int64_t)n_tokens * top_k * id_bytes}, {dloss, 4}, {counts, 4 * ((int64_t)n_experts + 1)}}))
        return EXL3_EINVAL;
    Params p = {logits, ids, id_bytes, n_tokens, top_k, n_experts, coefficient, 1};
    p.counts = const_cast<int*>(counts);
    p.dloss = dloss;
    p.dlogits = dlogits;
    return launch(dtype, BACKWARD, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

}  // extern "C"
