// int8_internal.hpp - what the 8-bit integer operators share between their files: the
// row operators' launch and the checks of arguments (host).
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/exl3_int8.h"
#include "spans.hpp"

namespace exl3 {
namespace i8 {

constexpr int MAX_ROW = 1 << 24;                // values of a row that the row operators take
constexpr int64_t MAX_ROWS = (int64_t)1 << 40;
constexpr int64_t MAX_VALUES = (int64_t)1 << 56;  // rows times values: their bytes stay within 64 bits
constexpr int64_t MAX_GRID = 1 << 20;           // workgroups of a row operator, which take row after row

// Rows to codes and scales; with a weight, after the norm.
struct RowsParams {
    const void* x;
    int64_t ldx;
    const void* residual;  // or null
    int64_t ldr;
    const void* weight;
    int weight_dtype;
    double eps;
    int64_t rows;
    int n;
    int8_t* codes;
    float* scales;
    void* added;
};
hipError_t launch_quantize(int dtype, const RowsParams& p, hipStream_t s);

inline bool misaligned(const void* ptr, uintptr_t to = 16) { return (reinterpret_cast<uintptr_t>(ptr) & (to - 1)) != 0; }
inline bool bad_dtype(int32_t d) { return d < EXL3_F16 || d > EXL3_F32; }
inline int64_t dtype_bytes(int32_t d) { return d == EXL3_F32 ? 4 : 2; }
inline bool bad_row(int32_t n) { return n < EXL3_INT8_PIECE || n % EXL3_INT8_PIECE != 0; }
inline bool too_many(int64_t rows, int32_t n) { return n > MAX_ROW || rows > MAX_ROWS || rows > MAX_VALUES / n; }
inline bool bad_ld(int64_t ldx, int32_t n, int32_t dtype) { return ldx < n || ldx * dtype_bytes(dtype) % 16 != 0; }

// `rows` rows of n values of dtype.
inline Span values(const void* at, int32_t dtype, int64_t rows, int64_t n, int64_t ld) {
    const int64_t size = dtype_bytes(dtype);
    return Span{at, n * size, rows, (rows > 1 ? ld : n) * size};
}

}  // namespace i8
}  // namespace exl3
