// balance.hip - the loss that evens out a router's experts, their counts and the
// gradient to the logits (gfx950).
#include <hip/hip_runtime.h>

#include "../../include/exl3_balance.h"
#include "pieces_device.hpp"
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
    float* loss;
    int* counts;
    const float* dloss;
    void* dlogits;
};

constexpr int THREADS = 256, WAVES = THREADS / 64;
constexpr int MAX_BLOCKS = 256;

// A token's logits lie in LANES lanes (a power of two), Q pieces of N = 16 bytes each:
// piece q of lane l is columns (q * LANES + l) * N and on.  A wave holds 64 / LANES tokens.
// LANES * Q * N >= experts.

// Does the token have a slot that is kept?  All lanes of the wave come here; lanes of a
// token share its slots out.  COUNT: kept slots go into the histogram.
template <int LANES, bool COUNT> __device__ inline bool counts_token(const Params& p, int token, bool live, int lane, int* hist) {
    bool kept = false;
    for (int j = lane; j < p.top_k; j += LANES) {
        if (!live) break;
        const int64_t at = (int64_t)token * p.top_k + j;
        const int64_t id = p.id_bytes == 8 ? static_cast<const int64_t*>(p.ids)[at] : (int64_t) static_cast<const int*>(p.ids)[at];
        if (id >= 0 && id < p.experts) {
            kept = true;
            if (COUNT) atomicAdd(&hist[(int)id], 1);
        }
    }
    if constexpr (LANES == 1) return kept;
    const uint64_t all = __ballot(kept);
    if constexpr (LANES == 64) return all != 0;
    const int first = (threadIdx.x & 63) / LANES * LANES;
    return ((all >> first) & ((1ull << (LANES & 63)) - 1)) != 0;
}

// The softmax of a token's logits: probabilities of this lane's columns, 0 behind the last.
template <typename T, int LANES, int Q, bool VEC>
__device__ inline void softmax(const Params& p, int token, bool live, int lane, float (&v)[Q][16 / T::bytes]) {
    constexpr int N = 16 / T::bytes;
    const float lowest = -__builtin_inff();
    float top = lowest;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        const int c = (q * LANES + lane) * N;
        u32x4_t r = {0, 0, 0, 0};
        const bool in = live && c < p.experts;
        if (in) r = load_piece<T, VEC>(p.logits, (int64_t)token * p.experts + c, p.experts - c);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[q][i] = in && c + i < p.experts ? piece_value<T>(r, i) : lowest;
            top = fmaxf(top, v[q][i]);
        }
    }
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
    if (top == lowest) top = 0.f;  // nothing but -infinity: exp gives zeros (a NaN stays one)
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            v[q][i] = expf(v[q][i] - top);
            sum += v[q][i];
        }
#pragma unroll
    for (int d = 1; d < LANES; d *= 2) sum += __shfl_xor(sum, d);
    const float inverse = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) v[q][i] *= inverse;
}

// The loss, `along` the sum over the experts of count times sum of probabilities.
__device__ inline float loss_of(const Params& p, int tokens, double along) {
    if (tokens == 0) return 0.f;
    const double of = tokens;
    return (float)(p.coefficient * p.experts * along / (of * of * p.top_k));
}

// Sum over the threads of a workgroup.
template <int COUNT> __device__ inline double block_sum(double v) {
    __shared__ double part[COUNT / 64];
#pragma unroll
    for (int d = 1; d < 64; d *= 2) v += __shfl_xor(v, d);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0;
#pragma unroll
    for (int w = 0; w < COUNT / 64; ++w) v += part[w];
    return v;
}

// Sums of probabilities and counts of the tokens of a workgroup: each lane adds up its
// columns over the wave's tokens in registers.  One workgroup alone writes the results.
template <typename T, int LANES, int Q, bool VEC> __global__ __launch_bounds__(THREADS) void sum_kernel(const Params p) {
    constexpr int N = 16 / T::bytes, EACH = 64 / LANES;
    __shared__ int hist[EXL3_MOE_MAX_EXPERTS + 1];
    __shared__ float sums[WAVES][LANES * Q * N];
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & (LANES - 1), slot = (threadIdx.x & 63) / LANES;
    for (int e = threadIdx.x; e <= p.experts; e += THREADS) hist[e] = 0;
    __syncthreads();
    float acc[Q][N];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[q][i] = 0.f;
    const int step = p.blocks * WAVES * EACH;
    for (int t0 = (blockIdx.x * WAVES + wave) * EACH; t0 < p.tokens; t0 += step) {
        const int token = t0 + slot;
        const bool live = token < p.tokens;
        const bool valid = counts_token<LANES, true>(p, token, live, lane, hist);
        float v[Q][N];
        softmax<T, LANES, Q, VEC>(p, token, live, lane, v);
        if (valid) {
#pragma unroll
            for (int q = 0; q < Q; ++q)
#pragma unroll
                for (int i = 0; i < N; ++i) acc[q][i] += v[q][i];
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
    for (int e = threadIdx.x; e < p.experts; e += THREADS) {
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
    along = block_sum<THREADS>(along);
    if (threadIdx.x == 0) {
        p.counts[p.experts] = hist[p.experts];
        *p.loss = loss_of(p, hist[p.experts], along);
    }
}

// The workgroups' sums to the loss and the counts, in the order of the workgroups.
constexpr int FINAL_THREADS = 1024;
__global__ __launch_bounds__(FINAL_THREADS) void loss_kernel(const Params p) {
    __shared__ float sums[FINAL_THREADS];
    __shared__ int counts[FINAL_THREADS];
    __shared__ int tokens;
    // `slices` threads an expert, each over every slices-th workgroup
    const int slices = FINAL_THREADS / p.experts, e = threadIdx.x / slices, k = threadIdx.x - e * slices;
    float s = 0.f;
    int c = 0;
    if (threadIdx.x == 0) tokens = 0;
    if (e < p.experts)
        for (int b = k; b < p.blocks; b += slices) {
            s += p.part[(int64_t)b * p.experts + e];
            c += p.part_counts[(int64_t)b * (p.experts + 1) + e];
        }
    sums[threadIdx.x] = s;
    counts[threadIdx.x] = c;
    __syncthreads();
    if (threadIdx.x < p.blocks) atomicAdd(&tokens, p.part_counts[(int64_t)threadIdx.x * (p.experts + 1) + p.experts]);
    double along = 0.0;
    if (threadIdx.x < p.experts) {
        s = 0.f;
        c = 0;
        for (int i = 0; i < slices; ++i) {
            s += sums[threadIdx.x * slices + i];
            c += counts[threadIdx.x * slices + i];
        }
        p.counts[threadIdx.x] = c;
        along = (double)c * s;
    }
    along = block_sum<FINAL_THREADS>(along);  // its barrier also ends the count of tokens
    if (threadIdx.x == 0) {
        p.counts[p.experts] = tokens;
        *p.loss = loss_of(p, tokens, along);
    }
}

// dlogits: the shares of this lane's columns stay in registers over all its tokens.
template <typename T, int LANES, int Q, bool VEC> __global__ __launch_bounds__(THREADS) void backward_kernel(const Params p) {
    constexpr int N = 16 / T::bytes, EACH = 64 / LANES;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & (LANES - 1), slot = (threadIdx.x & 63) / LANES;
    const int tokens = p.counts[p.experts];
    const double of = tokens > 0 ? tokens : 1;
    const float factor = (float)(*p.dloss * p.coefficient * (p.experts / of));
    float share[Q][N];
#pragma unroll
    for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int c = (q * LANES + lane) * N + i;
            share[q][i] = c < p.experts ? (float)(p.counts[c] / (of * p.top_k)) : 0.f;
        }
    const int step = gridDim.x * WAVES * EACH;
    for (int t0 = (blockIdx.x * WAVES + wave) * EACH; t0 < p.tokens; t0 += step) {
        const int token = t0 + slot;
        const bool live = token < p.tokens;
        const bool valid = counts_token<LANES, false>(p, token, live, lane, nullptr);
        float v[Q][N];
        softmax<T, LANES, Q, VEC>(p, token, live, lane, v);
        float along = 0.f;
#pragma unroll
        for (int q = 0; q < Q; ++q)
#pragma unroll
            for (int i = 0; i < N; ++i) along += v[q][i] * share[q][i];
#pragma unroll
        for (int d = 1; d < LANES; d *= 2) along += __shfl_xor(along, d);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
            const int c = (q * LANES + lane) * N;
            float g[N];
#pragma unroll
            for (int i = 0; i < N; ++i) g[i] = valid ? factor * (v[q][i] * (share[q][i] - along)) : 0.f;
            if (live && c < p.experts) store_piece<T, VEC, false>(p.dlogits, (int64_t)token * p.experts + c, p.experts - c, round_piece<T>(g));
        }
    }
}

// ---- launches ----

enum Op { LOSS, BACKWARD };

template <typename T, int LANES, int Q, bool VEC> hipError_t launch(Op op, const Params& p, hipStream_t s) {
    if (op == LOSS) {
        sum_kernel<T, LANES, Q, VEC><<<p.blocks, THREADS, 0, s>>>(p);
    } else {
        const int64_t blocks = ((int64_t)p.tokens + WAVES * (64 / LANES) - 1) / (WAVES * (64 / LANES));
        backward_kernel<T, LANES, Q, VEC><<<(unsigned)(blocks < 2048 ? blocks : 2048), THREADS, 0, s>>>(p);
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

// Workgroups of the first launch: one for few logits, else one for each 32 KB of fp32 logits, at most MAX_BLOCKS.
int plan_blocks(int tokens, int experts) {
    const int64_t blocks = ((int64_t)tokens * experts + 8191) / 8192;
    return blocks < 1 ? 1 : blocks > MAX_BLOCKS ? MAX_BLOCKS : (int)blocks;
}

bool misaligned(const void* ptr, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0; }
int64_t value_bytes(int dtype) { return dtype == EXL3_F32 ? 4 : 2; }
int64_t sums_bytes(int blocks, int experts) { return ((int64_t)blocks * experts * 4 + 255) & ~int64_t(255); }

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
    return blocks == 1 ? 0 : sums_bytes(blocks, n_experts) + (int64_t)blocks * (n_experts + 1) * 4;
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
    const Params p = {logits, ids, id_bytes, n_tokens, top_k, n_experts, coefficient, blocks, reinterpret_cast<float*>(ws),
                      reinterpret_cast<int*>(ws + (blocks > 1 ? sums_bytes(blocks, n_experts) : 0)), loss, counts, nullptr, nullptr};
    hipStream_t s = (hipStream_t)stream;
    if (launch(dtype, LOSS, p, s) != hipSuccess) return EXL3_EHIP;
    if (blocks > 1) loss_kernel<<<1, FINAL_THREADS, 0, s>>>(p);
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
    const Params p = {logits, ids, id_bytes, n_tokens, top_k, n_experts, coefficient, 1, nullptr, nullptr, nullptr, const_cast<int*>(counts), dloss, dlogits};
    return launch(dtype, BACKWARD, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

}  // extern "C"
