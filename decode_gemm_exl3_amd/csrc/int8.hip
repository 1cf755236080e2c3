// int8.hip - products of 8-bit rows with 8-bit weights (gfx950).
#include <hip/hip_runtime.h>

#include "int8_internal.hpp"
#include "tile_device.hpp"

namespace exl3 {
namespace i8 {

using namespace mx;  // element types, row tiles of groups, tile order

typedef int i32x16_t __attribute__((ext_vector_type(16)));

struct ProductParams {
    const int8_t* xc;  // quantised rows
    const float* xs;
    const int* offsets;  // null: one group of all rows
    int n_groups, rows;
    const int8_t* wc;
    const float* ws;
    int n_in, n_out;
    void* y;
};

constexpr int PIECE = EXL3_INT8_PIECE;

__device__ inline __amdgpu_buffer_rsrc_t buffer(const int8_t* base, int64_t bytes) {
    return mx::buffer(reinterpret_cast<const uint8_t*>(base), bytes);
}

// A wave's results, 32 RT rows from `row0` and 32 CT outputs from `col0`, of which
// `rows` rows are written.  A lane holds 4 consecutive outputs of a row; the sums take
// both scales (xs: of this lane's rows, ws: of the outputs, in LDS) and 32 rows at a time
// go through LDS (`part`, the wave's own), so that a store writes whole pieces of a row.
template <typename OT, int CT> constexpr int store_part_bytes() { return 32 * (32 * CT * OT::bytes + 16); }

template <typename OT, int RT, int CT>
__device__ inline void store_tile(const i32x16_t (&acc)[RT][CT], const float (&xs)[RT], const float* ws, char* part, const ProductParams& p,
                                  int row0, int rows, int col0) {
    typedef typename OT::raw raw;
    constexpr int PITCH = 32 * CT * OT::bytes + 16;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int cols = min(32 * CT, p.n_out - col0);
    const bool vec = ((int64_t)p.n_out * OT::bytes) % 16 == 0;
    raw* y = static_cast<raw*>(p.y);
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        const int live = min(32, rows - 32 * m);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4_t w = *reinterpret_cast<const f32x4_t*>(ws + 32 * c + 8 * g + 4 * h);
                f32x4_t v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = rounded((float)acc[m][c][4 * g + i] * xs[m] * w[i]);
                store4<OT>(part + r * PITCH, 32 * c + 8 * g + 4 * h, 4, true, v);
            }
        __builtin_amdgcn_wave_barrier();
        const int64_t y0 = (int64_t)(row0 + 32 * m) * p.n_out + col0;
        if (vec) {
            constexpr int PER = 16 / OT::bytes, LANES = 32 * CT / PER;  // outputs of a lane, lanes of a row
#pragma unroll
            for (int i = 0; i < 32; i += 64 / LANES) {
                const int row = i + lane / LANES, o = lane % LANES * PER;
                const i32x4_t v = *reinterpret_cast<const i32x4_t*>(part + row * PITCH + o * OT::bytes);
                if (row < live && o < cols) *reinterpret_cast<i32x4_t*>(y + y0 + (int64_t)row * p.n_out + o) = v;
            }
        } else {
            for (int i = lane; i < live * 32 * CT; i += 64) {
                const int row = i / (32 * CT), o = i % (32 * CT);
                const raw v = reinterpret_cast<const raw*>(part + row * PITCH)[o];
                if (o < cols) y[y0 + (int64_t)row * p.n_out + o] = v;
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// A workgroup of four waves owns 64 RT rows and 64 CT outputs, each wave a quarter of
// them.  Stages of 128 inputs of both sides go straight from memory into LDS, double
// buffered.  Block c (16 inputs) of row r sits in 16-byte slot c ^ (r / 2 & 7) of the
// row's 128 bytes: the 16 lanes that LDS serves together (0-3, 12-15, 20-23, 24-27
// and so on) then read 16 different slots of its 256-byte width.
//
// v_mfma_i32_32x32x32_i8 takes, per lane, 16 codes of row lane % 32, of the first or the
// second 16 inputs by lane / 32; accumulator i is row 8 (i / 4) + 4 (lane / 32) + i % 4 of
// the first operand (an output) against row lane % 32 of the second.
constexpr int STAGE_BLOCKS = 8;

template <typename OT, int RT, int CT>
__global__ __launch_bounds__(256, RT * CT > 4 ? 1 : 2) void tile_kernel(const ProductParams p, int row_tiles, int col_tiles) {
    constexpr int BM = 64 * RT, BN = 64 * CT;
    constexpr int STAGE = (BM + BN) * STAGE_BLOCKS;  // 16-byte slots: the rows', then the weight's
    constexpr int ROW_LOADS = BM / 32, W_LOADS = BN / 32;  // a wave's loads per stage, 8 rows each
    constexpr int PART = store_part_bytes<OT, CT>();
    constexpr int SLOTS = 2 * STAGE * 16 > 4 * PART ? 2 * STAGE : 4 * PART / 16;
    __shared__ i32x4_t lds[SLOTS + BN / 4];  // the buffers (later the waves' parts), then the outputs' scales
    float* const lds_scales = reinterpret_cast<float*>(lds + SLOTS);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, wy = wave >> 1, wx = wave & 1;
    int row_tile, col;
    if (!tile_of(xcd_tile(blockIdx.x), row_tiles, col_tiles, &row_tile, &col)) return;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, row_tile, BM);
    if (t.rows == 0) return;
    const int n0 = col * BN, cols = min(BN, p.n_out - n0);
    const int nb = p.n_in / PIECE, stages = (nb + STAGE_BLOCKS - 1) / STAGE_BLOCKS;

    i32x16_t acc[RT][CT];
    float xs[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        xs[m] = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][c][i] = 0;
    }
    if (t.group < p.n_groups) {
        const int64_t w0 = (int64_t)t.group * p.n_out + n0;
        const __amdgpu_buffer_rsrc_t bx = buffer(p.xc + (int64_t)t.row0 * p.n_in, (int64_t)t.rows * p.n_in);
        const __amdgpu_buffer_rsrc_t bw = buffer(p.wc + w0 * p.n_in, (int64_t)cols * p.n_in);
#pragma unroll
        for (int m = 0; m < RT; ++m) xs[m] = p.xs[t.row0 + min((wy * RT + m) * 32 + r, t.rows - 1)];
        for (int i = threadIdx.x; i < BN; i += 256) lds_scales[i] = p.ws[w0 + min(i, cols - 1)];
        // Rows behind the tile re-read its last (never stored).  Load i of a wave brings
        // rows 32 i + 8 wave .. + 7, lane l slot l % 8 of row l / 8.
        const int srow = 8 * wave + (lane >> 3), sblock = (lane & 7) ^ ((srow >> 1) & 7);
        uint32_t xat[ROW_LOADS], wat[W_LOADS];
#pragma unroll
        for (int i = 0; i < ROW_LOADS; ++i) xat[i] = (uint32_t)min(32 * i + srow, t.rows - 1) * p.n_in + 16 * sblock;
#pragma unroll
        for (int i = 0; i < W_LOADS; ++i) wat[i] = (uint32_t)min(32 * i + srow, cols - 1) * p.n_in + 16 * sblock;
        auto ask = [&](int st) {  // blocks behind the end: zeros
            const bool in = st * STAGE_BLOCKS + sblock < nb;
            i32x4_t* dst = lds + (st & 1) * STAGE + wave * 64;
#pragma unroll
            for (int i = 0; i < ROW_LOADS; ++i) load16_to_lds(bx, dst + i * 256, in ? xat[i] : OUTSIDE, (uint32_t)st * 128);
#pragma unroll
            for (int i = 0; i < W_LOADS; ++i) load16_to_lds(bw, dst + BM * 8 + i * 256, in ? wat[i] : OUTSIDE, (uint32_t)st * 128);
        };
        ask(0);
        for (int st = 0; st < stages; ++st) {
            __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0): this stage has landed, the one before it is read
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            if (st + 1 < stages) ask(st + 1);
            const i32x4_t* const buf = lds + (st & 1) * STAGE;
#pragma unroll
            for (int j = 0; j < STAGE_BLOCKS / 2; ++j) {
                const int slot = r * 8 + ((2 * j + h) ^ ((r >> 1) & 7));
                i32x4_t xv[RT], wv[CT];
#pragma unroll
                for (int m = 0; m < RT; ++m) xv[m] = buf[(wy * RT + m) * 256 + slot];
#pragma unroll
                for (int c = 0; c < CT; ++c) wv[c] = buf[BM * 8 + (wx * CT + c) * 256 + slot];
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[m][c] = __builtin_amdgcn_mfma_i32_32x32x32_i8(wv[c], xv[m], acc[m][c], 0, 0, 0);
            }
        }
    } else {
        for (int i = threadIdx.x; i < BN; i += 256) lds_scales[i] = 0.f;
    }
    __syncthreads();
    store_tile<OT, RT, CT>(acc, xs, lds_scales + wx * CT * 32, reinterpret_cast<char*>(lds) + wave * PART, p, t.row0 + wy * RT * 32,
                           t.rows - wy * RT * 32, n0 + wx * CT * 32);
}

// ---- launches ----

template <typename OT, int RT, int CT> hipError_t launch_tiles(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 64 * RT), cols = (p.n_out + 64 * CT - 1) / (64 * CT);
    tile_kernel<OT, RT, CT><<<(unsigned)xcd_padded(rows * cols), 256, 0, s>>>(p, (int)rows, (int)cols);
    return hipGetLastError();
}

template <typename OT> hipError_t launch_product(const ProductParams& p, hipStream_t s) {
    return launch_tiles<OT, 1, 1>(p, s);
}

hipError_t product(int dtype, const ProductParams& p, hipStream_t s) {
    switch (dtype) {
        case EXL3_F16: return launch_product<F16>(p, s);
        case EXL3_BF16: return launch_product<BF16>(p, s);
        default: return launch_product<F32>(p, s);
    }
}

// ---- argument checks ----

int64_t codes_bytes(int64_t rows, int32_t n) { return (rows * n + 255) & ~int64_t(255); }

int product_checks(int32_t rows, const int32_t* offsets, int32_t n_groups, const int8_t* codes, const float* scales,
                   int32_t n_in, int32_t n_out, const void* y, int32_t dtype) {
    if (bad_dtype(dtype) || bad_row(n_in) || n_out < 1 || rows < 0 || n_groups < 1) return EXL3_EINVAL;
    if (!offsets && n_groups != 1) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!codes || !scales || !y) return EXL3_EINVAL;
    if (misaligned(codes) || misaligned(scales, 4) || misaligned(y) || misaligned(offsets, 4)) return EXL3_EINVAL;
    // codes are -128 .. 127: fewer than 2^17 products of at most 2^14 stay below 2^31
    if (n_in >= (1 << 17) || n_groups > 4096 || rows > (1 << 23) || n_out > (1 << 24)) return EXL3_EUNSUPPORTED;
    // a launch takes fewer than 2^32 threads: 2^24 workgroups of the smallest tile that many outputs come in
    if ((((int64_t)rows >> 6) + n_groups + 2) * (((int64_t)n_out >> 6) + 1) >= (1 << 24) - XCDS * XCD_UNIT) return EXL3_EUNSUPPORTED;
    return 1;  // proceed
}

}  // namespace i8
}  // namespace exl3

extern "C" {

using exl3::apart;
using namespace exl3::i8;

int64_t exl3_int8_workspace_bytes(int32_t rows, int32_t n_groups, int32_t n_in) {
    if (rows < 0 || n_groups < 1 || bad_row(n_in)) return EXL3_EINVAL;
    return codes_bytes(rows, n_in) + (((int64_t)rows * 4 + 255) & ~int64_t(255));
}

int exl3_int8_matmul(const int8_t* x_codes, const float* x_scales, int32_t rows, const int32_t* offsets,
                     int32_t n_groups, const int8_t* codes, const float* scales, int32_t n_in, int32_t n_out, void* y,
                     int32_t dtype, void* stream) {
    const int rc = product_checks(rows, offsets, n_groups, codes, scales, n_in, n_out, y, dtype);
    if (rc <= 0) return rc;
    if (!x_codes || !x_scales || misaligned(x_codes) || misaligned(x_scales, 4)) return EXL3_EINVAL;
    const int64_t in = rows, w = (int64_t)n_groups * n_out, size = (int64_t)rows * n_out;
    if (!apart({values(y, dtype, 1, size, size)}, {{x_codes, in * n_in}, {x_scales, in * 4}, {codes, w * n_in}, {scales, w * 4},
               {offsets, 4 * ((int64_t)n_groups + 1)}}))
        return EXL3_EINVAL;
    const ProductParams p = {x_codes, x_scales, offsets, n_groups, rows, codes, scales, n_in, n_out, y};
    return product(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_int8_linear(const void* x, int32_t dtype, int32_t rows, int64_t ldx, const int32_t* offsets, int32_t n_groups,
                     const int8_t* codes, const float* scales, int32_t n_in, int32_t n_out, void* y, void* workspace,
                     size_t workspace_bytes, void* stream) {
    const int rc = product_checks(rows, offsets, n_groups, codes, scales, n_in, n_out, y, dtype);
    if (rc < 0) return rc;
    if (bad_ld(ldx, n_in, dtype)) return EXL3_EINVAL;
    if (rc == 0) return rc;
    if (!x || misaligned(x) || misaligned(workspace)) return EXL3_EINVAL;
    const int64_t need = exl3_int8_workspace_bytes(rows, n_groups, n_in);
    if (need > 0 && (!workspace || (int64_t)workspace_bytes < need)) return EXL3_EWORKSPACE;
    const int64_t w = (int64_t)n_groups * n_out, size = (int64_t)rows * n_out;
    if (!apart({values(y, dtype, 1, size, size), {workspace, need}}, {values(x, dtype, rows, n_in, ldx), {codes, w * n_in}, {scales, w * 4},
               {offsets, 4 * ((int64_t)n_groups + 1)}}))
        return EXL3_EINVAL;
    int8_t* const xc = static_cast<int8_t*>(workspace);
    float* const xs = reinterpret_cast<float*>(xc + codes_bytes(rows, n_in));
    const RowsParams q = {x, ldx, nullptr, 0, nullptr, 0, 0.0, rows, n_in, xc, xs, nullptr};
    if (launch_quantize(dtype, q, (hipStream_t)stream) != hipSuccess) return EXL3_EHIP;
    const ProductParams p = {xc, xs, offsets, n_groups, rows, codes, scales, n_in, n_out, y};
    return product(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

}  // extern "C"
