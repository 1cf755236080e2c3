// moe.hip - mixture-of-experts routing: the stable sort of slots by expert, the
// rows' gather, and their weighted sum with its gradients (gfx950).
#include <hip/hip_runtime.h>

#include "../../include/exl3_moe.h"
#include "mxfp4_device.hpp"
#include "spans.hpp"

namespace exl3 {
namespace moe {

using namespace mx;  // element types

// ---- sort ----
//
// A stable counting sort.  The slots are cut into chunks of consecutive slots, a
// workgroup each; count_kernel writes every chunk's count per expert, and
// place_kernel adds up the counts before its own (all experts before, then the
// same expert in the chunks before) and places its slots.  One chunk needs no
// first launch.  Latency bounds it: 10 slots 2.8 us, 65536 slots of 64 experts 4.9
// + 6.5 us, 1048576 slots 22 us.
constexpr int SORT_THREADS = 512, SORT_WAVES = SORT_THREADS / 64;
constexpr int SORT_MAX_CHUNKS = 256, SORT_MAX_COUNTS = 32768;
constexpr int SORT_ONE_CHUNK = 1024;  // slots one workgroup sorts alone (2 rounds, 4.9 us; two launches take 6.4)

struct SortParams {
    const void* ids;
    int id_bytes, slots, experts;
    int chunk, chunks;  // slots per chunk
    int* counts;        // [chunks][experts + 1]
    int* order;
    int* position;
    int* offsets;
};

// The bin of a slot: its expert, or `experts` when it is dropped.
__device__ inline int bin_of(const SortParams& p, int i) {
    if (p.id_bytes == 8) {
        const int64_t v = static_cast<const int64_t*>(p.ids)[i];
        return v >= 0 && v < p.experts ? (int)v : p.experts;
    }
    const int v = static_cast<const int*>(p.ids)[i];
    return v >= 0 && v < p.experts ? v : p.experts;
}

__device__ inline void count_chunk(const SortParams& p, int chunk, int* hist) {
    for (int e = threadIdx.x; e <= p.experts; e += SORT_THREADS) hist[e] = 0;
    __syncthreads();
    const int64_t end = min((int64_t)p.slots, (int64_t)(chunk + 1) * p.chunk);
    for (int64_t i = (int64_t)chunk * p.chunk + threadIdx.x; i < end; i += SORT_THREADS) atomicAdd(&hist[bin_of(p, (int)i)], 1);
    __syncthreads();
}

__global__ __launch_bounds__(SORT_THREADS) void count_kernel(const SortParams p) {
    __shared__ int hist[EXL3_MOE_MAX_EXPERTS + 1];
    count_chunk(p, blockIdx.x, hist);
    for (int e = threadIdx.x; e <= p.experts; e += SORT_THREADS) p.counts[(int64_t)blockIdx.x * (p.experts + 1) + e] = hist[e];
}

__global__ __launch_bounds__(SORT_THREADS) void place_kernel(const SortParams p) {
    __shared__ int next[EXL3_MOE_MAX_EXPERTS + 1];            // place of the next slot of each bin
    __shared__ int total[EXL3_MOE_MAX_EXPERTS + 1];           // a bin's count over all chunks
    __shared__ int in_wave[SORT_WAVES][EXL3_MOE_MAX_EXPERTS + 1];  // a bin's count in each wave's 64 slots
    __shared__ int wave_sum[SORT_WAVES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int bins = p.experts + 1;

    if (p.chunks == 1) {
        count_chunk(p, 0, total);
        for (int e = threadIdx.x; e < bins; e += SORT_THREADS) next[e] = 0;
    } else {
        for (int e = threadIdx.x; e < bins; e += SORT_THREADS) total[e] = next[e] = 0;
        __syncthreads();
        // the table's entries, row by row, over all threads; integer sums in any order
        constexpr int U = 8;
        const int entries = p.chunks * bins;
        for (int i0 = threadIdx.x; i0 < entries; i0 += U * SORT_THREADS) {
            int v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = i0 + u * SORT_THREADS < entries ? p.counts[i0 + u * SORT_THREADS] : 0;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int i = i0 + u * SORT_THREADS, c = i / bins, e = i - c * bins;
                if (v[u] == 0) continue;
                atomicAdd(&total[e], v[u]);
                if (c < (int)blockIdx.x) atomicAdd(&next[e], v[u]);
            }
        }
    }
    __syncthreads();
    // the bins' first places: an exclusive scan of the totals, SORT_THREADS bins at a time
    int carry = 0;
    for (int e0 = 0; e0 < bins; e0 += SORT_THREADS) {
        const int e = e0 + threadIdx.x;
        const int v = e < bins ? total[e] : 0;
        int sum = v;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const int up = __shfl_up(sum, d);
            if (lane >= d) sum += up;
        }
        if (lane == 63) wave_sum[wave] = sum;
        __syncthreads();
        int first = carry, all = 0;
        for (int w = 0; w < SORT_WAVES; ++w) {
            first += w < wave ? wave_sum[w] : 0;
            all += wave_sum[w];
        }
        carry += all;
        if (e < bins) {
            next[e] += first + sum - v;
            if (blockIdx.x == 0) p.offsets[e] = first + sum - v;
        }
        __syncthreads();
    }
    // 512 slots at a time: a slot's rank among the slots of its bin is the count
    // in the waves before plus the lanes before of its own wave
    int bits = 0;
    while ((1 << bits) < bins) ++bits;
    const int64_t begin = (int64_t)blockIdx.x * p.chunk, end = min((int64_t)p.slots, begin + p.chunk);
    for (int64_t i0 = begin; i0 < end; i0 += SORT_THREADS) {
        __syncthreads();  // the round before has read in_wave and moved next on
        for (int k = threadIdx.x; k < SORT_WAVES * bins; k += SORT_THREADS) in_wave[k / bins][k % bins] = 0;
        __syncthreads();
        const int64_t i = i0 + threadIdx.x;
        const bool live = i < end;
        const int e = live ? bin_of(p, (int)i) : 0;
        uint64_t same = __ballot(live);
        for (int b = 0; b < bits; ++b) {
            const uint64_t set = __ballot((e >> b) & 1);
            same &= (e >> b) & 1 ? set : ~set;
        }
        const int rank = __popcll(same & ((1ull << lane) - 1));
        if (live && rank == 0) in_wave[wave][e] = __popcll(same);
        __syncthreads();
        int place = rank;
        if (live) {
            place += next[e];
            for (int w = 0; w < wave; ++w) place += in_wave[w][e];
            p.order[place] = (int)i;
            p.position[i] = place;
        }
        __syncthreads();
        for (int k = threadIdx.x; k < bins; k += SORT_THREADS) {
            int n = 0;
            for (int w = 0; w < SORT_WAVES; ++w) n += in_wave[w][k];
            next[k] += n;
        }
    }
}

// ---- rows ----

struct RowParams {
    const void* in;    // x, or rows
    const void* in2;   // rows of the backward pass
    int tokens, top_k, n;
    const int* position;
    const int* kept;
    const void* weights;  // null: ones
    int weights_dtype;
    void* out;
    void* dweights;
    bool stream;  // the results' size asks for STREAM
};

// STREAM: results from 32 MiB on are stored past the L2s, which hold that much together and
// would write them back later, in the way of the next kernel (65536 rows of 4 KB
// gathered, then summed again: 121 us against 143; 4096 tokens of 8 KB combined and
// differentiated: 45 against 51).  Smaller ones stay there for their reader.
constexpr int64_t STREAM_BYTES = 32 << 20;

__device__ inline float load_weight(const RowParams& p, int64_t i) {
    if (!p.weights) return 1.f;
    if (p.weights_dtype == EXL3_F32) return static_cast<const float*>(p.weights)[i];
    const uint16_t v = static_cast<const uint16_t*>(p.weights)[i];
    return p.weights_dtype == EXL3_F16 ? to_f32(F16{}, v) : to_f32(BF16{}, v);
}

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

// The places (and weights) of up to 64 slots of a token, one a lane, loaded at
// once: the loops take them from the lanes, so that a token's rows are asked for
// without waiting for an index each.
struct Places {
    int at;
    float weight;
    __device__ inline int place(int j) const { return __builtin_amdgcn_readlane(at, j); }
    __device__ inline float factor(int j) const { return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, weight), j)); }
};
__device__ inline Places load_places(const RowParams& p, int64_t first, int count, bool weights) {
    const int lane = threadIdx.x & 63;
    Places s = {-1, 0.f};
    if (lane < count) {
        s.at = p.position[first + lane];
        if (weights) s.weight = load_weight(p, first + lane);
    }
    return s;
}

// rows[position[t][j]] = x[t]: a workgroup takes a token and 256 pieces of its
// row, reads them once and writes them top_k times.  Memory bounds it: 8192 tokens
// of 4 KB to 65536 rows in 47 us alone, 6.4 TB/s (58 with the sum below running after it).
template <typename T, bool VEC, bool STREAM> __global__ __launch_bounds__(256) void gather_kernel(const RowParams p) {
    constexpr int N = 16 / T::bytes;
    const int slots = p.tokens * p.top_k, kept = *p.kept;
    const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * N;
    const u32x4_t zero = {0, 0, 0, 0};
    const u32x4_t x = c < p.n ? load_piece<T, VEC>(p.in, (int64_t)t * p.n + c, p.n - c) : zero;
    for (int j0 = 0; j0 < p.top_k; j0 += 64) {
        const int count = min(64, p.top_k - j0);
        const Places s = load_places(p, (int64_t)t * p.top_k + j0, count, false);
        for (int j = 0; j < count; ++j) {
            const int at = s.place(j);
            if (at >= 0 && at < slots && c < p.n) store_piece<T, VEC, STREAM>(p.out, (int64_t)at * p.n + c, p.n - c, at < kept ? x : zero);
        }
    }
}

// y[t] = sum over j of weights[t][j] * rows[position[t][j]], U rows asked for
// together (a dropped slot's load goes to row 0 and is not used, so that no branch
// stands between the loads).  65536 rows of 4 KB to 8192 tokens in 53 us, 5.7 TB/s.
template <typename T, bool VEC, bool STREAM, int U> __global__ __launch_bounds__(256) void combine_kernel(const RowParams p) {
    constexpr int N = 16 / T::bytes;
    const int slots = p.tokens * p.top_k, kept = min(*p.kept, slots);
    const int t = blockIdx.x, c = (blockIdx.y * 256 + threadIdx.x) * N;
    const bool in = c < p.n;
    const int col = in ? c : 0;
    float sum[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.f;
    for (int j0 = 0; j0 < p.top_k; j0 += 64) {
        const Places s = load_places(p, (int64_t)t * p.top_k + j0, min(64, p.top_k - j0), true);
        for (int j = 0; j < 64 && j0 + j < p.top_k; j += U) {
            u32x4_t r[U];
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = s.place(j + k);  // -1 in lanes without a slot
                r[k] = load_piece<T, VEC>(p.in, (int64_t)(at >= 0 && at < kept ? at : 0) * p.n + col, p.n - col);
            }
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int at = s.place(j + k);
                if (at < 0 || at >= kept) continue;
                const float w = s.factor(j + k);
#pragma unroll
                for (int i = 0; i < N; ++i) sum[i] += w * piece_value<T>(r[k], i);
            }
        }
    }
    if (in) store_piece<T, VEC, STREAM>(p.out, (int64_t)t * p.n + c, p.n - c, round_piece<T>(sum));
}

// drows[position[t][j]] = weights[t][j] * dy[t] and dweights[t][j] = <rows[...], dy[t]>:
// one wave a slot, both in one pass over the rows.  A lane sums each value of its
// pieces apart, so that a sum's chain is n / (64 N) long and not n / 64 (67 x 3 rows
// of 1000 fp32 values are 0.9e-7 from 64 bits, 1.4e-7 with one sum a lane; no time).
// 8192 slots of 8 KB in 29 us: 5.7 TB/s of dy, rows and drows.
template <typename T, bool VEC, bool STREAM> __global__ __launch_bounds__(256) void combine_backward_kernel(const RowParams p) {
    constexpr int N = 16 / T::bytes;
    const int slots = p.tokens * p.top_k, kept = min(*p.kept, slots);
    const int lane = threadIdx.x & 63;
    const int64_t s = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if (s >= slots) return;
    const int64_t t = s / p.top_k;
    const int at = p.position[s];
    const bool live = at >= 0 && at < kept;
    const float w = live ? load_weight(p, s) : 0.f;
    float sums[N];
#pragma unroll
    for (int i = 0; i < N; ++i) sums[i] = 0.f;
    if (at >= 0 && at < slots) {
        for (int c = lane * N; c < p.n; c += 64 * N) {
            u32x4_t out = {0, 0, 0, 0};
            if (live) {
                const u32x4_t d = load_piece<T, VEC>(p.in, t * p.n + c, p.n - c);
                const u32x4_t r = load_piece<T, VEC>(p.in2, (int64_t)at * p.n + c, p.n - c);
                float g[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    g[i] = piece_value<T>(d, i);
                    sums[i] += g[i] * piece_value<T>(r, i);
                    g[i] *= w;
                }
                out = round_piece<T>(g);
            }
            store_piece<T, VEC, STREAM>(p.out, (int64_t)at * p.n + c, p.n - c, out);
        }
    }
#pragma unroll
    for (int d = N / 2; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < d; ++i) sums[i] += sums[i + d];
    float dot = sums[0];
#pragma unroll
    for (int d = 32; d > 0; d /= 2) dot += __shfl_xor(dot, d);
    if (lane == 0) {
        if (p.weights_dtype == EXL3_F32) static_cast<float*>(p.dweights)[s] = dot;
        else static_cast<uint16_t*>(p.dweights)[s] = p.weights_dtype == EXL3_F16 ? from_f32(F16{}, dot) : from_f32(BF16{}, dot);
    }
}

enum RowOp { GATHER, COMBINE, COMBINE_BACKWARD };

template <typename T, bool VEC, bool STREAM> hipError_t launch_rows(RowOp op, const RowParams& p, hipStream_t s) {
    const int pieces = (p.n * T::bytes + 15) / 16;
    const dim3 grid((unsigned)p.tokens, (unsigned)((pieces + 255) / 256));
    if (op == GATHER) gather_kernel<T, VEC, STREAM><<<grid, 256, 0, s>>>(p);
    else if (op == COMBINE && p.top_k <= 2) combine_kernel<T, VEC, STREAM, 2><<<grid, 256, 0, s>>>(p);
    else if (op == COMBINE && p.top_k <= 4) combine_kernel<T, VEC, STREAM, 4><<<grid, 256, 0, s>>>(p);
    else if (op == COMBINE) combine_kernel<T, VEC, STREAM, 8><<<grid, 256, 0, s>>>(p);
    else combine_backward_kernel<T, VEC, STREAM><<<(unsigned)(((int64_t)p.tokens * p.top_k + 3) / 4), 256, 0, s>>>(p);
    return hipGetLastError();
}

template <typename T> hipError_t launch_rows(RowOp op, const RowParams& p, hipStream_t s) {
    if ((int64_t)p.n * T::bytes % 16 != 0) return launch_rows<T, false, false>(op, p, s);
    return p.stream ? launch_rows<T, true, true>(op, p, s) : launch_rows<T, true, false>(op, p, s);
}

int rows_op(RowOp op, int dtype, const RowParams& p, hipStream_t s) {
    const hipError_t e = dtype == EXL3_F16 ? launch_rows<F16>(op, p, s) : dtype == EXL3_BF16 ? launch_rows<BF16>(op, p, s) : launch_rows<F32>(op, p, s);
    return e == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

bool misaligned(const void* ptr, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0; }
bool bad_dtype(int32_t d) { return d < EXL3_F16 || d > EXL3_F32; }

int64_t bytes_of(int64_t values, int32_t dtype) { return values * (dtype == EXL3_F32 ? 4 : 2); }

bool streams(int64_t tokens, int64_t rows_each, int64_t n, int dtype) {
    return bytes_of(tokens * rows_each * n, dtype) >= STREAM_BYTES;
}

// Checks shared by the three row operators: <= 0 is the call's status.
int row_checks(const void* in, int32_t dtype, int32_t n_tokens, int32_t top_k, int32_t n, const int32_t* position,
               const int32_t* kept, const void* out) {
    if (bad_dtype(dtype) || n_tokens < 0 || top_k < 1 || n < 1) return EXL3_EINVAL;
    if (n_tokens == 0) return EXL3_OK;
    if (!in || !position || !kept || !out) return EXL3_EINVAL;
    if (misaligned(in) || misaligned(position) || misaligned(kept, 4) || misaligned(out)) return EXL3_EINVAL;
    // a launch takes fewer than 2^32 threads: a workgroup a token, a wave a slot
    if (n_tokens >= (1 << 24) || (int64_t)n_tokens * top_k >= (1 << 26) - 4 || n > (1 << 24)) return EXL3_EUNSUPPORTED;
    return 1;
}

// One chunk while one workgroup sorts the slots alone, else at most
// SORT_MAX_CHUNKS chunks of whole rounds of SORT_THREADS slots; fewer where many
// experts make the table of counts long, as every chunk reads all of it.
void plan_sort(int slots, int experts, int* chunk, int* chunks) {
    if (slots <= SORT_ONE_CHUNK) {
        *chunk = SORT_ONE_CHUNK;
        *chunks = 1;
        return;
    }
    const int64_t rounds = ((int64_t)slots + SORT_THREADS - 1) / SORT_THREADS;
    const int64_t most = min(SORT_MAX_CHUNKS, SORT_MAX_COUNTS / (experts + 1));
    const int64_t per = (rounds + most - 1) / most;
    *chunk = (int)(per * SORT_THREADS);
    *chunks = (int)((rounds + per - 1) / per);
}

bool bad_sort(int32_t n_slots, int32_t n_experts) {
    return n_slots < 0 || n_experts < 1 || n_experts > EXL3_MOE_MAX_EXPERTS;
}

}  // namespace moe
}  // namespace exl3

extern "C" {

using exl3::apart;
using namespace exl3::moe;

int64_t exl3_moe_workspace_bytes(int32_t n_slots, int32_t n_experts) {
    if (bad_sort(n_slots, n_experts)) return EXL3_EINVAL;
    int chunk, chunks;
    plan_sort(n_slots, n_experts, &chunk, &chunks);
    return chunks == 1 ? 0 : (int64_t)chunks * (n_experts + 1) * 4;
}

int exl3_moe_sort(const void* ids, int32_t id_bytes, int32_t n_slots, int32_t n_experts, int32_t* order,
                  int32_t* position, int32_t* offsets, void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_sort(n_slots, n_experts) || (id_bytes != 4 && id_bytes != 8)) return EXL3_EINVAL;
    if (!offsets || misaligned(offsets)) return EXL3_EINVAL;
    if (n_slots > 0 && (!ids || !order || !position || misaligned(ids) || misaligned(order) || misaligned(position)))
        return EXL3_EINVAL;
    if (misaligned(workspace)) return EXL3_EINVAL;
    if (n_slots > (1 << 30)) return EXL3_EUNSUPPORTED;
    const int64_t need = exl3_moe_workspace_bytes(n_slots, n_experts);
    if (need > 0 && (!workspace || (int64_t)workspace_bytes < need)) return EXL3_EWORKSPACE;
    const int64_t slots = n_slots;
    if (!apart({{order, 4 * slots}, {position, 4 * slots}, {offsets, 4 * ((int64_t)n_experts + 1)}, {workspace, need}}, {{ids, id_bytes * slots}}))
        return EXL3_EINVAL;
    SortParams p = {ids, id_bytes, n_slots, n_experts, 0, 0, static_cast<int*>(workspace), order, position, offsets};
    plan_sort(n_slots, n_experts, &p.chunk, &p.chunks);
    hipStream_t s = (hipStream_t)stream;
    if (p.chunks > 1) {
        count_kernel<<<p.chunks, SORT_THREADS, 0, s>>>(p);
        if (hipGetLastError() != hipSuccess) return EXL3_EHIP;
    }
    place_kernel<<<p.chunks, SORT_THREADS, 0, s>>>(p);
    return hipGetLastError() == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_moe_gather(const void* x, int32_t dtype, int32_t n_tokens, int32_t top_k, int32_t n, const int32_t* position,
                    const int32_t* kept, void* rows, void* stream) {
    const int rc = row_checks(x, dtype, n_tokens, top_k, n, position, kept, rows);
    if (rc <= 0) return rc;
    const int64_t tokens = n_tokens, slots = tokens * top_k;
    if (!apart({{rows, bytes_of(slots * n, dtype)}}, {{x, bytes_of(tokens * n, dtype)}, {position, 4 * slots}, {kept, 4}})) return EXL3_EINVAL;
    const RowParams p = {x, nullptr, n_tokens, top_k, n, position, kept, nullptr, EXL3_F32, rows, nullptr, streams(n_tokens, top_k, n, dtype)};
    return rows_op(GATHER, dtype, p, (hipStream_t)stream);
}

int exl3_moe_combine(const void* rows, int32_t dtype, int32_t n_tokens, int32_t top_k, int32_t n,
                     const int32_t* position, const int32_t* kept, const void* weights, int32_t weights_dtype, void* y,
                     void* stream) {
    if (bad_dtype(weights_dtype)) return EXL3_EINVAL;
    const int rc = row_checks(rows, dtype, n_tokens, top_k, n, position, kept, y);
    if (rc <= 0) return rc;
    if (misaligned(weights)) return EXL3_EINVAL;
    const int64_t tokens = n_tokens, slots = tokens * top_k;
    if (!apart({{y, bytes_of(tokens * n, dtype)}}, {{rows, bytes_of(slots * n, dtype)}, {position, 4 * slots}, {kept, 4}, {weights, bytes_of(slots, weights_dtype)}}))
        return EXL3_EINVAL;
    const RowParams p = {rows, nullptr, n_tokens, top_k, n, position, kept, weights, weights_dtype, y, nullptr, streams(n_tokens, 1, n, dtype)};
    return rows_op(COMBINE, dtype, p, (hipStream_t)stream);
}

int exl3_moe_combine_backward(const void* dy, const void* rows, int32_t dtype, int32_t n_tokens, int32_t top_k,
                              int32_t n, const int32_t* position, const int32_t* kept, const void* weights,
                              int32_t weights_dtype, void* drows, void* dweights, void* stream) {
    if (bad_dtype(weights_dtype)) return EXL3_EINVAL;
    const int rc = row_checks(dy, dtype, n_tokens, top_k, n, position, kept, drows);
    if (rc <= 0) return rc;
    if (!rows || !weights || !dweights || misaligned(rows) || misaligned(weights) || misaligned(dweights)) return EXL3_EINVAL;
    const int64_t tokens = n_tokens, slots = tokens * top_k;
    if (!apart({{drows, bytes_of(slots * n, dtype)}, {dweights, bytes_of(slots, weights_dtype)}},
               {{dy, bytes_of(tokens * n, dtype)}, {rows, bytes_of(slots * n, dtype)}, {position, 4 * slots}, {kept, 4}, {weights, bytes_of(slots, weights_dtype)}}))
        return EXL3_EINVAL;
    const RowParams p = {dy, rows, n_tokens, top_k, n, position, kept, weights, weights_dtype, drows, dweights, streams(n_tokens, top_k, n, dtype)};
    return rows_op(COMBINE_BACKWARD, dtype, p, (hipStream_t)stream);
}

}  // extern "C"
