// mxfp4.hip - MXFP4 quantisation, dequantisation and products (gfx950).
#include <hip/hip_runtime.h>

#include "../../include/exl3_mxfp4.h"
#include "mxfp4_device.hpp"

namespace exl3 {
namespace mx {

// ---- quantise: values to codes and scales ----
//
// A lane takes 8 consecutive values, four lanes a block: the block's largest
// magnitude is a maximum over the quad (two DPP moves), then each lane converts
// its own values to one dword of codes, so codes leave a wave as 256 consecutive
// bytes.
constexpr int QUANT_UNROLL = 4;

template <typename T, bool FLAT>
__global__ __launch_bounds__(256) void quantize_kernel(const void* __restrict__ xv, int64_t rows, int n, int64_t ldx,
                                                       uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    constexpr int NW = T::bytes == 2 ? 4 : 8;  // dwords of 8 values
    const int64_t units = rows * (n / 8);
    const int64_t base = (int64_t)blockIdx.x * 256 * QUANT_UNROLL + threadIdx.x;
    uint32_t w[QUANT_UNROLL][NW];
#pragma unroll
    for (int u = 0; u < QUANT_UNROLL; ++u) {
        const int64_t i = base + u * 256;
        if (i >= units) continue;
        int64_t at = i * 8;
        if (!FLAT) {
            const int64_t r = i / (n / 8);
            at = r * ldx + (i - r * (n / 8)) * 8;
        }
        const u32x4_t* src = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(xv) + at * T::bytes);
#pragma unroll
        for (int c = 0; c < NW / 4; ++c) {
            const u32x4_t v = src[c];
#pragma unroll
            for (int e = 0; e < 4; ++e) w[u][4 * c + e] = v[e];
        }
    }
#pragma unroll
    for (int u = 0; u < QUANT_UNROLL; ++u) {
        const int64_t i = base + u * 256;
        if (i >= units) continue;  // whole quads: units is a multiple of 4
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < NW; ++e) m = abs_max<T>(m, w[u][e]);
        uint32_t a = abs_max_f32_bits<T>(m);
        uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
        a = a > o ? a : o;
        o = (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
        a = a > o ? a : o;
        const uint32_t b = scale_byte(a);
        const uint32_t c = cvt8<T>(w[u], scale_value(b));
        codes[i] = b == 255u ? 0u : c;
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
    }
}

// ---- dequantise: codes and scales to values ----
template <typename T>
__global__ __launch_bounds__(256) void dequantize_kernel(const uint32_t* __restrict__ codes,
                                                         const uint8_t* __restrict__ scales, int64_t units,
                                                         void* __restrict__ out) {
    const int64_t base = (int64_t)blockIdx.x * 256 * QUANT_UNROLL + threadIdx.x;
    uint32_t c[QUANT_UNROLL], b[QUANT_UNROLL];
#pragma unroll
    for (int u = 0; u < QUANT_UNROLL; ++u) {
        const int64_t i = base + u * 256;
        if (i >= units) continue;
        c[u] = codes[i];
        b[u] = scales[i >> 2];
    }
#pragma unroll
    for (int u = 0; u < QUANT_UNROLL; ++u) {
        const int64_t i = base + u * 256;
        if (i >= units) continue;
        // 2^(b - 127); b = 255 makes an infinity, and its blocks are NaN
        const float s = scale_value(b[u]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const uint32_t code = (c[u] >> (4 * e)) & 15u;
            // magnitude: 0 and .5 without an implied bit, (1 + mantissa / 2) * 2^(exponent - 1) else
            const uint32_t mag = code & 7u;
            const float f = mag < 2u ? 0.5f * (float)mag : __builtin_bit_cast(float, (((mag >> 1) + 126u) << 23) | ((mag & 1u) << 22));
            v[e] = b[u] == 255u ? __builtin_nanf("") : (code & 8u ? -f : f) * s;
        }
        if constexpr (T::bytes == 2) {
            u32x4_t r;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                r[e] = (uint32_t)from_f32(T{}, v[2 * e]) | ((uint32_t)from_f32(T{}, v[2 * e + 1]) << 16);
            static_cast<u32x4_t*>(out)[i] = r;
        } else {
            u32x4_t r0, r1;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                r0[e] = from_f32(T{}, v[e]);
                r1[e] = from_f32(T{}, v[4 + e]);
            }
            static_cast<u32x4_t*>(out)[2 * i] = r0;
            static_cast<u32x4_t*>(out)[2 * i + 1] = r1;
        }
    }
}

// ---- products ----

struct ProductParams {
    const void* x;  // rows of values (quantised inside), or null
    int64_t ldx;
    const uint8_t* xc;  // quantised rows
    const uint8_t* xs;
    const int* offsets;  // null: one group of all rows
    int n_groups, rows;
    const uint8_t* wc;
    const uint8_t* ws;
    int n_in, n_out;
    void* y;
};

// This lane's four scales of a span: bytes at s[0..3], `left` of them in the row
// (others read as 1).  whole: every row has a multiple of 4 blocks, so the dword
// is aligned and all in the row or all behind it.
__device__ inline uint32_t load_scales(const uint8_t* s, int left, bool whole) {
    uint32_t v = UNIT_SCALES;
    if (whole) {
        if (left > 0) v = *reinterpret_cast<const uint32_t*>(s);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < left) v = (v & ~(0xFFu << (8 * j))) | ((uint32_t)s[j] << (8 * j));
    }
    return v;
}
// This lane's four blocks of codes, zeros behind the row's end.
__device__ inline void load_codes(const uint8_t* c, int left, i32x4_t (&v)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[j] = i32x4_t{0, 0, 0, 0};
        if (j < left) v[j] = reinterpret_cast<const i32x4_t*>(c)[j];
    }
}

// One block of 32 values to an operand: its 16 bytes of codes and scale byte.
template <typename T> __device__ inline i32x4_t quantize_block(const uint32_t (&w)[8 * T::bytes], uint32_t& b) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8 * T::bytes; ++e) m = abs_max<T>(m, w[e]);
    b = scale_byte(abs_max_f32_bits<T>(m));
    const float s = scale_value(b);
    i32x4_t c;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
        const uint32_t v = cvt8<T>(w + d * 2 * T::bytes, s);
        c[d] = b == 255u ? 0 : (int)v;
    }
    return c;
}

template <typename OT> __device__ inline void store4(void* y, int64_t at, int count, bool vec, const f32x4_t v) {
    typedef typename OT::raw raw;
    raw* dst = static_cast<raw*>(y) + at;
    if (vec && count >= 4) {
        if constexpr (OT::bytes == 2) {
            uint2 r;
            r.x = (uint32_t)from_f32(OT{}, v[0]) | ((uint32_t)from_f32(OT{}, v[1]) << 16);
            r.y = (uint32_t)from_f32(OT{}, v[2]) | ((uint32_t)from_f32(OT{}, v[3]) << 16);
            *reinterpret_cast<uint2*>(dst) = r;
        } else {
            *reinterpret_cast<f32x4_t*>(dst) = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < count) dst[i] = from_f32(OT{}, v[i]);
    }
}

// Few rows: a workgroup owns 16 NS outputs for a tile of 16 MT rows; its W waves
// share the spans of the input (wave w takes spans w, w + W, ...) and read the
// weight from memory straight into the operand, once.  The rows come quantised,
// or (FUSED) as values that each lane quantises into the operand it needs: a
// lane's block is its own, so this takes no exchange.  The waves' sums meet in
// LDS and are added in the order of the waves.
template <typename OT, bool FUSED, int MT, int NS, int W>
__global__ __launch_bounds__(W * 64) void skinny_kernel(const ProductParams p) {
    __shared__ f32x4_t red[W][NS * MT][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, blockIdx.y, 16 * MT);
    if (t.rows == 0) return;
    const int n0 = blockIdx.x * 16 * NS;
    const int nb = p.n_in / BLOCK, spans = (nb + SPAN_BLOCKS - 1) / SPAN_BLOCKS;
    const bool whole = (nb & 3) == 0, vec = (p.n_out & 3) == 0;

    f32x4_t acc[NS][MT];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[s][m] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    if (t.group < p.n_groups) {
        const uint8_t *wc[NS], *ws[NS];
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const int64_t o = (int64_t)t.group * p.n_out + min(n0 + 16 * s + r, p.n_out - 1);
            wc[s] = p.wc + o * (p.n_in / 2) + 64 * q;
            ws[s] = p.ws + o * nb + 4 * q;
        }
        for (int sp = wave; sp < spans; sp += W) {
            const int left = nb - sp * SPAN_BLOCKS - 4 * q;
            i32x4_t wv[NS][4];
            uint32_t wsc[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                load_codes(wc[s] + sp * 256, left, wv[s]);
                wsc[s] = load_scales(ws[s] + sp * 16, left, whole);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int row = t.row0 + 16 * m + r;
                const bool live = 16 * m + r < t.rows;
                i32x4_t xv[4];
                uint32_t xsc = UNIT_SCALES;
                if constexpr (FUSED) {
                    const char* x = static_cast<const char*>(p.x) + ((int64_t)row * p.ldx + sp * 512 + 128 * q) * OT::bytes;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        xv[j] = i32x4_t{0, 0, 0, 0};
                        if (live && j < left) {
                            uint32_t w[8 * OT::bytes];
#pragma unroll
                            for (int c = 0; c < 2 * OT::bytes; ++c) {
                                const u32x4_t v = reinterpret_cast<const u32x4_t*>(x + j * BLOCK * OT::bytes)[c];
#pragma unroll
                                for (int e = 0; e < 4; ++e) w[4 * c + e] = v[e];
                            }
                            uint32_t b;
                            xv[j] = quantize_block<OT>(w, b);
                            xsc = (xsc & ~(0xFFu << (8 * j))) | (b << (8 * j));
                        }
                    }
                } else {
                    const int xleft = live ? left : 0;
                    load_codes(p.xc + (int64_t)row * (p.n_in / 2) + sp * 256 + 64 * q, xleft, xv);
                    xsc = load_scales(p.xs + (int64_t)row * nb + sp * 16 + 4 * q, xleft, whole);
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    acc[s][m] = mfma<0>(wv[s][0], wsc[s], xv[0], xsc, acc[s][m]);
                    acc[s][m] = mfma<1>(wv[s][1], wsc[s], xv[1], xsc, acc[s][m]);
                    acc[s][m] = mfma<2>(wv[s][2], wsc[s], xv[2], xsc, acc[s][m]);
                    acc[s][m] = mfma<3>(wv[s][3], wsc[s], xv[3], xsc, acc[s][m]);
                }
            }
        }
    }
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
        for (int m = 0; m < MT; ++m) red[wave][s * MT + m][lane] = acc[s][m];
    __syncthreads();
    for (int i = threadIdx.x; i < NS * MT * 64; i += W * 64) {
        const int l = i & 63, sm = i >> 6, s = sm / MT, m = sm - s * MT;
        f32x4_t v = red[0][sm][l];
#pragma unroll
        for (int w = 1; w < W; ++w) v += red[w][sm][l];
        const int row = 16 * m + (l & 15), o = n0 + 16 * s + 4 * (l >> 4);
        if (row < t.rows && o < p.n_out) store4<OT>(p.y, (int64_t)(t.row0 + row) * p.n_out + o, p.n_out - o, vec, v);
    }
}

// Many rows: a workgroup of four waves owns 16 RT rows and 256 outputs, wave w
// all the rows and outputs 64 w .. 64 w + 63.  The quantised rows of a span (256
// bytes each) are staged in LDS, double buffered and loaded there directly; the
// weight goes from memory into the operands, as no other wave needs it.  Block c
// of row r sits in 16-byte slot c ^ (r & 15) of the row's 256 bytes: the 16 rows
// of an operand then read 16 different slots.
template <typename OT, int RT>
__global__ __launch_bounds__(256, 1) void gemm_kernel(const ProductParams p) {
    constexpr int BM = 16 * RT;
    __shared__ i32x4_t As[2][BM * 16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, q = lane >> 4;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, blockIdx.y, BM);
    if (t.rows == 0) return;
    const int n0 = blockIdx.x * 256 + wave * 64;
    const int nb = p.n_in / BLOCK, spans = (nb + SPAN_BLOCKS - 1) / SPAN_BLOCKS;
    const bool whole = (nb & 3) == 0, vec = (p.n_out & 3) == 0;
    const int half = p.n_in / 2;

    f32x4_t acc[RT][4];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    if (t.group < p.n_groups) {
        // load i of a wave brings 4 rows: lane l writes slot l % 16 of row l / 16.
        // Rows behind the tile re-read its last, blocks behind the row's end its last
        // block: what they multiply is zero or never stored.
        const uint8_t* xc = p.xc + (int64_t)t.row0 * half;
        auto stage = [&](int sp, int buf) {
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                const int row = (i * 4 + wave) * 4 + (lane >> 4);
                const int c = min((lane & 15) ^ (row & 15), nb - 1 - sp * SPAN_BLOCKS);
                const uint8_t* src = xc + (int64_t)min(row, t.rows - 1) * half + sp * 256 + c * 16;
                __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                                 (__attribute__((address_space(3))) void*)(&As[buf][(i * 4 + wave) * 64]), 16, 0, 0);
            }
        };
        const uint8_t *wc[4], *ws[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int64_t o = (int64_t)t.group * p.n_out + min(n0 + 16 * c + r, p.n_out - 1);
            wc[c] = p.wc + o * half + 64 * q;
            ws[c] = p.ws + o * nb + 4 * q;
        }
        stage(0, 0);
        for (int sp = 0; sp < spans; ++sp) {
            const int left = nb - sp * SPAN_BLOCKS - 4 * q;
            i32x4_t wv[4][4];
            uint32_t wsc[4], xsc[RT];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                load_codes(wc[c] + sp * 256, left, wv[c]);
                wsc[c] = load_scales(ws[c] + sp * 16, left, whole);
            }
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                const int row = t.row0 + min(16 * m + r, t.rows - 1);
                xsc[m] = load_scales(p.xs + (int64_t)row * nb + sp * 16 + 4 * q, left, whole);
            }
            __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): this span's rows have landed
            __syncthreads();
            if (sp + 1 < spans) stage(sp + 1, (sp + 1) & 1);
            const i32x4_t* a = As[sp & 1];
#pragma unroll
            for (int m = 0; m < RT; ++m) {
                i32x4_t xv[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[j] = a[(16 * m + r) * 16 + ((4 * q + j) ^ r)];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    acc[m][c] = mfma<0>(wv[c][0], wsc[c], xv[0], xsc[m], acc[m][c]);
                    acc[m][c] = mfma<1>(wv[c][1], wsc[c], xv[1], xsc[m], acc[m][c]);
                    acc[m][c] = mfma<2>(wv[c][2], wsc[c], xv[2], xsc[m], acc[m][c]);
                    acc[m][c] = mfma<3>(wv[c][3], wsc[c], xv[3], xsc[m], acc[m][c]);
                }
            }
            __syncthreads();  // the buffer is free for the span after next
        }
    }
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            const int row = 16 * m + r, o = n0 + 16 * c + 4 * q;
            if (row < t.rows && o < p.n_out)
                store4<OT>(p.y, (int64_t)(t.row0 + row) * p.n_out + o, p.n_out - o, vec, acc[m][c]);
        }
}

// ---- launches ----

template <typename T> hipError_t launch_quantize(const void* x, int64_t rows, int n, int64_t ldx, uint8_t* codes,
                                                 uint8_t* scales, hipStream_t s) {
    const int64_t units = rows * (n / 8);
    const dim3 grid((unsigned)((units + 256 * QUANT_UNROLL - 1) / (256 * QUANT_UNROLL)));
    if (ldx == n || rows == 1)
        quantize_kernel<T, true><<<grid, 256, 0, s>>>(x, rows, n, ldx, reinterpret_cast<uint32_t*>(codes), scales);
    else
        quantize_kernel<T, false><<<grid, 256, 0, s>>>(x, rows, n, ldx, reinterpret_cast<uint32_t*>(codes), scales);
    return hipGetLastError();
}

// Rows above which the staged product takes over from the few-rows one.
constexpr int SKINNY_MAX_ROWS = 64;

template <typename OT, bool FUSED, int MT, int NS> hipError_t launch_skinny(const ProductParams& p, hipStream_t s) {
    constexpr int W = 8;
    const dim3 grid((unsigned)((p.n_out + 16 * NS - 1) / (16 * NS)),
                    (unsigned)max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 16 * MT));
    skinny_kernel<OT, FUSED, MT, NS, W><<<grid, W * 64, 0, s>>>(p);
    return hipGetLastError();
}

// Rows that a group has on average: what a tile's height is chosen by.
inline int64_t typical_rows(int64_t rows, int n_groups) { return (rows + n_groups - 1) / n_groups; }
// Whether a product quantises its rows itself.
inline bool fused(int64_t rows, int n_groups) { return typical_rows(rows, n_groups) <= 16; }

template <typename OT> hipError_t launch_product(const ProductParams& p, hipStream_t s) {
    const int64_t m = typical_rows(p.rows, p.n_groups);
    if (p.x) return launch_skinny<OT, true, 1, 1>(p, s);
    if (m <= 16) return launch_skinny<OT, false, 1, 1>(p, s);
    if (m <= 32) return launch_skinny<OT, false, 2, 1>(p, s);
    if (m <= SKINNY_MAX_ROWS) return launch_skinny<OT, false, 4, 1>(p, s);
    if (m <= 128) {
        const dim3 grid((unsigned)((p.n_out + 255) / 256), (unsigned)max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 128));
        gemm_kernel<OT, 8><<<grid, 256, 0, s>>>(p);
    } else {
        const dim3 grid((unsigned)((p.n_out + 255) / 256), (unsigned)max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 256));
        gemm_kernel<OT, 16><<<grid, 256, 0, s>>>(p);
    }
    return hipGetLastError();
}

hipError_t product(int dtype, const ProductParams& p, hipStream_t s) {
    switch (dtype) {
        case EXL3_F16: return launch_product<F16>(p, s);
        case EXL3_BF16: return launch_product<BF16>(p, s);
        default: return launch_product<F32>(p, s);
    }
}

hipError_t quantize(int dtype, const void* x, int64_t rows, int n, int64_t ldx, uint8_t* codes, uint8_t* scales, hipStream_t s) {
    switch (dtype) {
        case EXL3_F16: return launch_quantize<F16>(x, rows, n, ldx, codes, scales, s);
        case EXL3_BF16: return launch_quantize<BF16>(x, rows, n, ldx, codes, scales, s);
        default: return launch_quantize<F32>(x, rows, n, ldx, codes, scales, s);
    }
}

// ---- argument checks ----

bool misaligned(const void* ptr) { return (reinterpret_cast<uintptr_t>(ptr) & 15) != 0; }
bool bad_dtype(int32_t d) { return d < EXL3_F16 || d > EXL3_F32; }
int dtype_bytes(int32_t d) { return d == EXL3_F32 ? 4 : 2; }
bool bad_row(int32_t n) { return n < BLOCK || n % BLOCK != 0; }
bool bad_ld(int64_t ldx, int32_t n, int32_t dtype) { return ldx < n || ldx * dtype_bytes(dtype) % 16 != 0; }

int64_t codes_bytes(int64_t rows, int32_t n) { return (rows * (n / 2) + 255) & ~int64_t(255); }

// Workgroups that one launch takes of quantise and dequantise: 2^31 - 1.
bool too_many_units(int64_t rows, int32_t n) {
    return rows > ((int64_t)1 << 40) || rows * (n / 8) > (int64_t)0x7FFFFFFF * 256 * QUANT_UNROLL;
}

int product_checks(int32_t rows, const int32_t* offsets, int32_t n_groups, const uint8_t* codes, const uint8_t* scales,
                   int32_t n_in, int32_t n_out, const void* y, int32_t dtype) {
    if (bad_dtype(dtype) || bad_row(n_in) || n_out < 1 || rows < 0 || n_groups < 1) return EXL3_EINVAL;
    if (!offsets && n_groups != 1) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!codes || !scales || !y) return EXL3_EINVAL;
    if (misaligned(codes) || misaligned(scales) || misaligned(y) || (reinterpret_cast<uintptr_t>(offsets) & 3)) return EXL3_EINVAL;
    if (n_in > (1 << 20) || n_groups > 4096 || rows > (1 << 23) || n_out > (1 << 24)) return EXL3_EUNSUPPORTED;
    return 1;  // proceed
}

}  // namespace mx
}  // namespace exl3

extern "C" {

using namespace exl3::mx;

int exl3_mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int32_t n, int64_t ldx, uint8_t* codes,
                        uint8_t* scales, void* stream) {
    if (bad_dtype(dtype) || bad_row(n) || rows < 0 || bad_ld(ldx, n, dtype)) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!x || !codes || !scales || misaligned(x) || misaligned(codes) || misaligned(scales)) return EXL3_EINVAL;
    if (too_many_units(rows, n)) return EXL3_EUNSUPPORTED;
    return quantize(dtype, x, rows, n, ldx, codes, scales, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t n, void* out,
                          int32_t dtype, void* stream) {
    if (bad_dtype(dtype) || bad_row(n) || rows < 0) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!out || !codes || !scales || misaligned(out) || misaligned(codes) || misaligned(scales)) return EXL3_EINVAL;
    if (too_many_units(rows, n)) return EXL3_EUNSUPPORTED;
    const int64_t units = rows * (n / 8);
    const dim3 grid((unsigned)((units + 256 * QUANT_UNROLL - 1) / (256 * QUANT_UNROLL)));
    const uint32_t* c = reinterpret_cast<const uint32_t*>(codes);
    hipStream_t s = (hipStream_t)stream;
    if (dtype == EXL3_F16) dequantize_kernel<F16><<<grid, 256, 0, s>>>(c, scales, units, out);
    else if (dtype == EXL3_BF16) dequantize_kernel<BF16><<<grid, 256, 0, s>>>(c, scales, units, out);
    else dequantize_kernel<F32><<<grid, 256, 0, s>>>(c, scales, units, out);
    return hipGetLastError() == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int64_t exl3_mxfp4_workspace_bytes(int32_t rows, int32_t n_groups, int32_t n_in) {
    if (rows < 0 || n_groups < 1 || bad_row(n_in)) return EXL3_EINVAL;
    return fused(rows, n_groups) ? 0 : codes_bytes(rows, n_in) + (((int64_t)rows * (n_in / BLOCK) + 255) & ~int64_t(255));
}

int exl3_mxfp4_matmul(const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows, const int32_t* offsets,
                      int32_t n_groups, const uint8_t* codes, const uint8_t* scales, int32_t n_in, int32_t n_out,
                      void* y, int32_t dtype, void* stream) {
    const int rc = product_checks(rows, offsets, n_groups, codes, scales, n_in, n_out, y, dtype);
    if (rc <= 0) return rc;
    if (!x_codes || !x_scales || misaligned(x_codes) || misaligned(x_scales) || y == x_codes || y == x_scales)
        return EXL3_EINVAL;
    const ProductParams p = {nullptr, 0, x_codes, x_scales, offsets, n_groups, rows, codes, scales, n_in, n_out, y};
    return product(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_mxfp4_linear(const void* x, int32_t dtype, int32_t rows, int64_t ldx, const int32_t* offsets,
                      int32_t n_groups, const uint8_t* codes, const uint8_t* scales, int32_t n_in, int32_t n_out,
                      void* y, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = product_checks(rows, offsets, n_groups, codes, scales, n_in, n_out, y, dtype);
    if (rc < 0) return rc;
    if (bad_ld(ldx, n_in, dtype)) return EXL3_EINVAL;
    if (rc == 0) return rc;
    if (!x || misaligned(x) || misaligned(workspace) || x == y) return EXL3_EINVAL;
    const int64_t need = exl3_mxfp4_workspace_bytes(rows, n_groups, n_in);
    if (need > 0 && (!workspace || (int64_t)workspace_bytes < need)) return EXL3_EWORKSPACE;
    ProductParams p = {x, ldx, nullptr, nullptr, offsets, n_groups, rows, codes, scales, n_in, n_out, y};
    if (need > 0) {
        uint8_t* xc = static_cast<uint8_t*>(workspace);
        uint8_t* xs = xc + codes_bytes(rows, n_in);
        if (quantize(dtype, x, rows, n_in, ldx, xc, xs, (hipStream_t)stream) != hipSuccess) return EXL3_EHIP;
        p.x = nullptr;
        p.xc = xc;
        p.xs = xs;
    }
    return product(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

}  // extern "C"
