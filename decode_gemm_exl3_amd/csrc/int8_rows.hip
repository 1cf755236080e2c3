// int8_rows.hip - rows of values to 8-bit codes and scales, with a norm before them or
// without, and codes back to values (gfx950).
#include <hip/hip_runtime.h>

#include "int8_device.hpp"
#include "int8_internal.hpp"

namespace exl3 {
namespace i8 {

// ---- quantise, norm ----
//
// One pass over a row finds its largest magnitude A (and, for a norm, the sum of its
// squares), the codes follow from the values kept in registers.  A norm's codes are
// round(127 u / A) of u = h * weight: the row's 1 / rms is in u and A alike and cancels, so
// it enters the scale alone.
//
// Squares are summed in 64 bits: those of fp32 and bf16 values pass the range of fp32.
//
// Memory bounds it: 8192 rows of 8192 fp16 with a residual and their sum kept, 470 MB, take 95.8 us (4.9 TB/s;
// a large copy moves 5.0), 16384 rows of 2048 quantised 19.6 us.  A single row is launch and latencies: 2.9 us.

// N consecutive weights from column c on.
template <int N> __device__ inline void load_weights(const void* w, int dtype, int c, float (&out)[N]) {
    if (dtype == EXL3_F32) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(w) + c + i);
#pragma unroll
            for (int k = 0; k < 4; ++k) out[i + k] = v[k];
        }
    } else {
        uint32_t r[N / 2];
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(w) + c);
        if constexpr (N == 8) {
            const u32x4_t v = *reinterpret_cast<const u32x4_t*>(src);
#pragma unroll
            for (int k = 0; k < 4; ++k) r[k] = v[k];
        } else {
            const uint2 v = *reinterpret_cast<const uint2*>(src);
            r[0] = v.x;
            r[1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint16_t b = (uint16_t)(r[i / 2] >> (16 * (i & 1)));
            out[i] = dtype == EXL3_F16 ? to_f32(F16{}, b) : to_f32(BF16{}, b);
        }
    }
}

// THREADS threads a row (up to 64: 256 / THREADS rows a workgroup), P pieces of 16 bytes a thread;
// P == 0: longer rows, read once for the sums and again for the codes.
template <typename T, bool NORM, int THREADS, int P>
__global__ __launch_bounds__(THREADS <= 64 ? 256 : THREADS) void rows_kernel(const RowsParams p) {
    constexpr int N = 16 / T::bytes, KEPT = P > 0 ? P : 1, WAVES = THREADS / 64, LANES = THREADS <= 64 ? THREADS : 64;
    constexpr int ROWS = THREADS <= 64 ? 256 / THREADS : 1;  // of a workgroup
    __shared__ uint32_t wave_amax[2][WAVES > 0 ? WAVES : 1];
    __shared__ double wave_squares[2][WAVES > 0 ? WAVES : 1];
    const int thread = threadIdx.x % THREADS;  // of the row
    int parity = 0;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + threadIdx.x / THREADS; row < p.rows; row += (int64_t)gridDim.x * ROWS, parity ^= 1) {
        const int64_t x0 = row * p.ldx, r0 = row * p.ldr, o0 = row * p.n;
        float u[KEPT][N];
        uint32_t amax = 0;
        double squares = 0.0;
        // the values of a piece, before the weight; `first`: the sum is stored
        auto values = [&](int c, bool first, float (&v)[N]) {
            const u32x4_t a = load_piece<T, true>(p.x, x0 + c, N);
            if (NORM && p.residual) {
                const u32x4_t b = load_piece<T, true>(p.residual, r0 + c, N);
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = piece_value<T>(a, i) + piece_value<T>(b, i);
                const u32x4_t h = round_piece<T>(v);
                if (first) *reinterpret_cast<u32x4_t*>(static_cast<typename T::raw*>(p.added) + o0 + c) = h;
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = piece_value<T>(h, i);
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) v[i] = piece_value<T>(a, i);
            }
        };
        auto piece = [&](int c, bool first, float (&v)[N]) {
            values(c, first, v);
            if constexpr (NORM) {
                float w[N];
                load_weights<N>(p.weight, p.weight_dtype, c, w);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    if (first) squares = __builtin_fma((double)v[i], (double)v[i], squares);
                    v[i] *= w[i];
                }
            }
            amax = amax_piece<N>(amax, v);
        };
        if constexpr (P > 0) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const int c = (k * THREADS + thread) * N;
                if (c < p.n) piece(c, true, u[k]);
                else
#pragma unroll
                    for (int i = 0; i < N; ++i) u[k][i] = 0.f;
            }
        } else {
            for (int c = thread * N; c < p.n; c += THREADS * N) piece(c, true, u[0]);
        }
        amax = over_lanes<LANES>(amax, larger);
        if (NORM) squares = over_lanes<LANES>(squares, [](double a, double b) { return a + b; });
        if constexpr (WAVES > 1) {
            if ((threadIdx.x & 63) == 0) {
                wave_amax[parity][threadIdx.x >> 6] = amax;
                if (NORM) wave_squares[parity][threadIdx.x >> 6] = squares;
            }
            __syncthreads();
            amax = 0;
            squares = 0.0;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                amax = amax > wave_amax[parity][w] ? amax : wave_amax[parity][w];
                if (NORM) squares += wave_squares[parity][w];
            }
        }
        const bool bad = amax >= NOT_FINITE;
        const float largest = __builtin_bit_cast(float, amax), inverse = 127.f / largest;
        if (thread == 0) p.scales[row] = row_scale(amax, NORM ? sqrt(squares / p.n + p.eps) : 1.0);
        auto store = [&](int c, const float (&v)[N]) {
            uint32_t out[N / 4];
            if (bad) {
#pragma unroll
                for (int i = 0; i < N / 4; ++i) out[i] = 0;
            } else {
                code_piece<N>(v, largest, inverse, out);
            }
            uint32_t* dst = reinterpret_cast<uint32_t*>(p.codes + o0 + c);
            if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = uint2{out[0], out[1]};
            else *dst = out[0];
        };
        if constexpr (P > 0) {
#pragma unroll
            for (int k = 0; k < P; ++k) {
                const int c = (k * THREADS + thread) * N;
                if (c < p.n) store(c, u[k]);
            }
        } else {
            for (int c = thread * N; c < p.n; c += THREADS * N) {
                piece(c, false, u[0]);
                store(c, u[0]);
            }
        }
    }
}

// ---- dequantise ----
//
// A thread makes 16 bytes of values four times, 256 threads' apart, so that a wave's stores are whole lines.
// (Once where that leaves most CUs without a workgroup: 13 rows of 4096 2.0 us against 2.7.)
// Memory bounds it: 8192 rows of 8192 to fp16, 201 MB, take 33.1 us, 6.1 TB/s (codes just made are in the cache).
constexpr int DEQUANT_UNROLL = 4;

template <typename T, typename INDEX, int U>
__global__ __launch_bounds__(256) void dequantize_kernel(const int8_t* __restrict__ codes, const float* __restrict__ scales,
                                                         int64_t units, INDEX per_row, void* __restrict__ out) {
    constexpr int N = 16 / T::bytes;
    const int64_t base = (int64_t)blockIdx.x * 256 * U + threadIdx.x;
    uint32_t c[U][N / 4];
    float s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + u * 256;
        if (i >= units) continue;
        if constexpr (N == 8) {
            const uint2 v = reinterpret_cast<const uint2*>(codes)[i];
            c[u][0] = v.x;
            c[u][1] = v.y;
        } else {
            c[u][0] = reinterpret_cast<const uint32_t*>(codes)[i];
        }
        s[u] = scales[(INDEX)i / per_row];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + u * 256;
        if (i >= units) continue;
        float v[N];
#pragma unroll
        for (int e = 0; e < N; ++e) v[e] = rounded((float)((int)(c[u][e / 4] << (24 - 8 * (e & 3))) >> 24) * s[u]);
        reinterpret_cast<u32x4_t*>(out)[i] = round_piece<T>(v);
    }
}

// ---- launches ----

template <typename T, bool NORM, int THREADS, int P> hipError_t launch(const RowsParams& p, hipStream_t s) {
    constexpr int ROWS = THREADS <= 64 ? 256 / THREADS : 1;
    const int64_t groups = (p.rows + ROWS - 1) / ROWS;
    rows_kernel<T, NORM, THREADS, P><<<(unsigned)(groups < MAX_GRID ? groups : MAX_GRID), THREADS <= 64 ? 256 : THREADS, 0, s>>>(p);
    return hipGetLastError();
}

// Threads a row and pieces a thread (us): as few pieces as there are where rows are few, since a
// row is then one latency after the other (256 rows of 2048 bf16, norm: 3.4 with 4 waves of one piece,
// 6.8 with one wave of 4; one row of 4096 3.3 with 8 x 1, 4.1 with 4 x 4); where they are many, two
// pieces of four waves or eight (16384 rows of 2048, quantised: 19.6 with 2 x 2, 23.0 with 1 x 4; 2048
// rows of 8192, norm: 26.9 with 8 x 2, 30.4 with 4 x 4; 2048 rows of 16384: 54.7 with 8 x 4, 65.9 with 16 x 4).
template <typename T, bool NORM> hipError_t launch_rows(const RowsParams& p, hipStream_t s) {
    const int pieces = p.n * T::bytes / 16;  // n <= 2^24
    const bool few = p.rows <= 512;
    if (pieces <= 4) return launch<T, NORM, 4, 1>(p, s);
    if (pieces <= 8) return launch<T, NORM, 8, 1>(p, s);
    if (pieces <= 16) return launch<T, NORM, 16, 1>(p, s);
    if (pieces <= 32) return launch<T, NORM, 32, 1>(p, s);
    if (pieces <= 64) return launch<T, NORM, 64, 1>(p, s);
    if (pieces <= 128) return launch<T, NORM, 64, 2>(p, s);
    if (pieces <= 256) return NORM || few ? launch<T, NORM, 256, 1>(p, s) : launch<T, NORM, 128, 2>(p, s);
    if (pieces <= 512) return few ? launch<T, NORM, 512, 1>(p, s) : launch<T, NORM, 256, 2>(p, s);
    if (pieces <= 1024) return launch<T, NORM, 512, 2>(p, s);
    if (pieces <= 2048) return few ? launch<T, NORM, 1024, 2>(p, s) : launch<T, NORM, 512, 4>(p, s);
    if (pieces <= 4096) return launch<T, NORM, 1024, 4>(p, s);
    return launch<T, NORM, 1024, 0>(p, s);
}

template <bool NORM> hipError_t launch_rows(int dtype, const RowsParams& p, hipStream_t s) {
    switch (dtype) {
        case EXL3_F16: return launch_rows<F16, NORM>(p, s);
        case EXL3_BF16: return launch_rows<BF16, NORM>(p, s);
        default: return launch_rows<F32, NORM>(p, s);
    }
}

hipError_t launch_quantize(int dtype, const RowsParams& p, hipStream_t s) { return launch_rows<false>(dtype, p, s); }

template <typename T, int U> hipError_t launch_dequantize(const int8_t* codes, const float* scales, int64_t units, int per_row, void* out, hipStream_t s) {
    const unsigned grid = (unsigned)((units + 256 * U - 1) / (256 * U));
    if (units < (1ll << 32)) dequantize_kernel<T, uint32_t, U><<<grid, 256, 0, s>>>(codes, scales, units, (uint32_t)per_row, out);
    else dequantize_kernel<T, int64_t, U><<<grid, 256, 0, s>>>(codes, scales, units, (int64_t)per_row, out);
    return hipGetLastError();
}
template <typename T> hipError_t launch_dequantize(const int8_t* codes, const float* scales, int64_t rows, int n, void* out, hipStream_t s) {
    constexpr int N = 16 / T::bytes;
    const int64_t units = rows * (n / N);
    if (units < 256 * 256 * DEQUANT_UNROLL) return launch_dequantize<T, 1>(codes, scales, units, n / N, out, s);
    return launch_dequantize<T, DEQUANT_UNROLL>(codes, scales, units, n / N, out, s);
}

}  // namespace i8
}  // namespace exl3

extern "C" {

using exl3::apart;
using exl3::Span;
using namespace exl3::i8;

int exl3_int8_quantize(const void* x, int32_t dtype, int64_t rows, int32_t n, int64_t ldx, int8_t* codes,
                       float* scales, void* stream) {
    if (bad_dtype(dtype) || bad_row(n) || rows < 0 || bad_ld(ldx, n, dtype)) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!x || !codes || !scales || misaligned(x) || misaligned(codes) || misaligned(scales, 4)) return EXL3_EINVAL;
    if (too_many(rows, n)) return EXL3_EUNSUPPORTED;
    if (!apart({{codes, rows * n}, {scales, rows * 4}}, {values(x, dtype, rows, n, ldx)})) return EXL3_EINVAL;
    const RowsParams p = {x, ldx, nullptr, 0, nullptr, 0, 0.0, rows, n, codes, scales, nullptr};
    return launch_quantize(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_int8_dequantize(const int8_t* codes, const float* scales, int64_t rows, int32_t n, void* out, int32_t dtype,
                         void* stream) {
    if (bad_dtype(dtype) || bad_row(n) || rows < 0) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!out || !codes || !scales || misaligned(out) || misaligned(codes) || misaligned(scales, 4)) return EXL3_EINVAL;
    // a launch takes fewer than 2^32 threads: 2^24 - 1 workgroups, of at least 4096 values
    if (too_many(rows, n) || rows * n > (int64_t)0xFFFFFF * 4096) return EXL3_EUNSUPPORTED;
    if (!apart({values(out, dtype, 1, rows * n, rows * n)}, {{codes, rows * n}, {scales, rows * 4}})) return EXL3_EINVAL;
    hipStream_t s = (hipStream_t)stream;
    const hipError_t e = dtype == EXL3_F16    ? launch_dequantize<exl3::mx::F16>(codes, scales, rows, n, out, s)
                         : dtype == EXL3_BF16 ? launch_dequantize<exl3::mx::BF16>(codes, scales, rows, n, out, s)
                                              : launch_dequantize<exl3::mx::F32>(codes, scales, rows, n, out, s);
    return e == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_int8_rms_norm(const void* x, int32_t dtype, int64_t rows, int32_t n, int64_t ldx, const void* residual,
                       int64_t ldr, const void* weight, int32_t weight_dtype, double eps, int8_t* codes, float* scales,
                       void* added, void* stream) {
    if (bad_dtype(dtype) || bad_dtype(weight_dtype) || bad_row(n) || rows < 0 || bad_ld(ldx, n, dtype)) return EXL3_EINVAL;
    if (!(eps >= 0.0 && eps <= 1.7976931348623157e308) || !residual != !added || (residual && bad_ld(ldr, n, dtype))) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!x || !weight || !codes || !scales || misaligned(x) || misaligned(residual) || misaligned(weight) || misaligned(codes) ||
        misaligned(scales, 4) || misaligned(added))
        return EXL3_EINVAL;
    if (too_many(rows, n)) return EXL3_EUNSUPPORTED;
    if (!apart({{codes, rows * n}, {scales, rows * 4}, values(added, dtype, 1, rows * n, rows * n)},
               {values(x, dtype, rows, n, ldx), values(residual, dtype, rows, n, ldr), values(weight, weight_dtype, 1, n, n)}))
        return EXL3_EINVAL;
    const RowsParams p = {x, ldx, residual, ldr, weight, weight_dtype, eps, rows, n, codes, scales, added};
    return launch_rows<true>(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

}  // extern "C"
