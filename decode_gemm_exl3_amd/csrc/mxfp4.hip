// mxfp4.hip - MXFP4 quantisation, dequantisation and products (gfx950).
#include <hip/hip_runtime.h>

#include <type_traits>

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
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
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

// Many rows: a workgroup of four waves owns 64 RT rows and 256 outputs, each wave
// a quarter of them, 32 RT rows and 128 outputs.  Stages of 256 inputs (128 bytes
// of codes a row) of both sides go straight from memory into LDS, double
// buffered; the waves read their operands from there.  (A weight operand read
// from memory by its lanes would touch 64 cache lines for 1 KB.)
//
// Block c of row r sits in 16-byte slot c ^ (r / 2 & 7) of the row's 128 bytes:
// the 16 lanes that LDS serves together (0-3, 12-15, 20-23, 24-27 and so on) then
// read 16 different slots of its 256-byte width.
//
// A stage is four steps of 64 inputs; lane half h holds blocks 4h .. 4h + 3 of the
// stage's eight, one dword of scales, and feeds block 4h + j to step j.
//
// The scales of two stages (16 bytes a row) go through LDS as well, four lanes a
// row: read by the lanes that use them they would be one dword from each of 64
// places, 64 cycles of the address unit a load and twice the time of all codes.
// Where rows start at any byte (WHOLE false: n_in % 128 != 0) the eight aligned
// dwords that hold them are staged and two of them meet in an alignbyte.

// Workgroup b of a launch to tile index: units of 32 consecutive tiles go to the
// same XCD (workgroups go round the 8 XCDs one by one), so that the tiles that
// run together on an XCD share rows and weights in its L2.
constexpr int XCDS = 8, XCD_UNIT = 32;
__device__ inline int xcd_tile(int b) {
    const int xcd = b % XCDS, local = b / XCDS;
    return (local / XCD_UNIT * XCDS + xcd) * XCD_UNIT + local % XCD_UNIT;
}
// Tiles of a launch, padded to whole rounds of units.
inline int64_t xcd_padded(int64_t tiles) { return (tiles + XCDS * XCD_UNIT - 1) / (XCDS * XCD_UNIT) * (XCDS * XCD_UNIT); }
constexpr int BAND = 8;  // row tiles that share a run of output tiles

// Memory from `base` on, read at 32-bit offsets.
__device__ inline __amdgpu_buffer_rsrc_t buffer(const uint8_t* base, int64_t bytes) {
    const uint32_t n = bytes > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, n, 0x00020000);
}
__device__ inline i32x4_t load16(__amdgpu_buffer_rsrc_t b, uint32_t voff, uint32_t soff) {
    return __builtin_bit_cast(i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, 0));
}
// Straight into LDS: lane l's 16 bytes at dst + 16 l.
__device__ inline void load16_to_lds(__amdgpu_buffer_rsrc_t b, i32x4_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}
constexpr uint32_t OUTSIDE = 0x7FFFFFF0u;  // an offset past every buffer: the load gives zeros

__device__ inline void load4_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 4, voff, soff, 0, 0);
}

constexpr int STAGE_BLOCKS = 8;

template <typename OT, int RT, bool WHOLE>
__global__ __launch_bounds__(256, 1) void gemm_kernel(const ProductParams p, int row_tiles, int col_tiles) {
    constexpr int BM = 64 * RT, BN = 256;
    constexpr int STAGE = (BM + BN) * 8;  // 16-byte slots: the rows', then the weight's
    constexpr int ROW_LOADS = BM / 32, W_LOADS = BN / 32;  // a wave's loads per stage, 8 rows each
    constexpr int SDW = WHOLE ? 4 : 8;    // dwords of scales a row holds in LDS
    constexpr int SPAIR = (BM + BN) * SDW, SCALE_LOADS = (BM + BN) * SDW / 256;
    __shared__ i32x4_t lds[2 * STAGE + SPAIR / 2];  // one object: the compiler then keeps loads into it in flight over reads of it
    uint32_t* const lds_scales = reinterpret_cast<uint32_t*>(lds + 2 * STAGE);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, wy = wave >> 1, wx = wave & 1;
    const int tile = xcd_tile(blockIdx.x);
    const int band = tile / (BAND * col_tiles), band_rows = min(BAND, row_tiles - band * BAND);
    if (band_rows <= 0) return;
    const int in_band = tile - band * BAND * col_tiles;
    const int col = in_band / band_rows;
    if (col >= col_tiles) return;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, band * BAND + in_band - col * band_rows, BM);
    if (t.rows == 0) return;
    const int n0 = col * BN, cols = min(BN, p.n_out - n0);
    const int nb = p.n_in / BLOCK, stages = (nb + STAGE_BLOCKS - 1) / STAGE_BLOCKS;
    const int half = p.n_in / 2;

    f32x16_t acc[RT][4];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[m][c][i] = 0.f;

    if (t.group < p.n_groups) {
        const int64_t w0 = (int64_t)t.group * p.n_out + n0;
        // scales from the 16-byte border at or before the tile's first
        const int64_t xs0 = (int64_t)t.row0 * nb, ws0 = w0 * nb;
        const __amdgpu_buffer_rsrc_t bxc = buffer(p.xc + (int64_t)t.row0 * half, (int64_t)t.rows * half);
        const __amdgpu_buffer_rsrc_t bwc = buffer(p.wc + w0 * half, (int64_t)cols * half);
        const __amdgpu_buffer_rsrc_t bxs = buffer(p.xs + (xs0 & ~int64_t(15)), ((xs0 & 15) + (int64_t)t.rows * nb + 3) & ~int64_t(3));
        const __amdgpu_buffer_rsrc_t bws = buffer(p.ws + (ws0 & ~int64_t(15)), ((ws0 & 15) + (int64_t)cols * nb + 3) & ~int64_t(3));
        // Byte offsets of this lane from those.  Rows behind the tile re-read its
        // last, outputs behind the last re-read that one (never stored).  Load i
        // of a wave brings rows 32 i + 8 wave .. + 7, lane l slot l % 8 of row l / 8.
        const int srow = 8 * wave + (lane >> 3), sblock = (lane & 7) ^ ((srow >> 1) & 7);
        uint32_t rc[ROW_LOADS], wc[W_LOADS], so[SCALE_LOADS];
#pragma unroll
        for (int i = 0; i < ROW_LOADS; ++i) rc[i] = (uint32_t)min(32 * i + srow, t.rows - 1) * half;
#pragma unroll
        for (int i = 0; i < W_LOADS; ++i) wc[i] = (uint32_t)min(32 * i + srow, cols - 1) * half;
        // load i of a wave brings the scales of 64 / SDW rows
        const int sdw = lane % SDW;
#pragma unroll
        for (int i = 0; i < SCALE_LOADS; ++i) {
            const int row = (4 * i + wave) * (64 / SDW) + lane / SDW;
            const uint32_t first = row < BM ? (uint32_t)min(row, t.rows - 1) * nb + (uint32_t)(xs0 & 15)
                                            : (uint32_t)min(row - BM, cols - 1) * nb + (uint32_t)(ws0 & 15);
            so[i] = (first & ~3u) + 4 * sdw;
        }
        // Load k of a wave for stage st.  Rows: blocks behind the end re-read the
        // last (any codes: the weight's are zeros there).
        auto ask_codes = [&](int k, int st, int buf) {
            const int rest = nb - st * STAGE_BLOCKS;
            const uint32_t soff = (uint32_t)st * 128;
            i32x4_t* dst = lds + buf * STAGE + wave * 64;
            if (k < ROW_LOADS) load16_to_lds(bxc, dst + k * 256, rc[k] + 16 * min(sblock, rest - 1), soff);
            else load16_to_lds(bwc, dst + BM * 8 + (k - ROW_LOADS) * 256, sblock < rest ? wc[k - ROW_LOADS] + 16 * sblock : OUTSIDE, soff);
        };
        // Load k of a wave for the scales of stages 2 pair and 2 pair + 1.
        auto ask_scales = [&](int k, uint32_t off, int pair) {
            const bool in = pair * SPAN_BLOCKS + 4 * sdw < nb + (WHOLE ? 0 : 4);
            load4_to_lds((4 * k + wave) * (64 / SDW) < BM ? bxs : bws, lds_scales + (pair & 1) * SPAIR + (4 * k + wave) * 64,
                         in ? off : OUTSIDE, (uint32_t)pair * SPAN_BLOCKS);
        };
        // The dword of this lane's four blocks of stage st, of staged row `row`.
        auto scales = [&](int row, int shift, int st, int par) {  // par = st & 1
            const uint32_t* s = lds_scales + (st >> 1 & 1) * SPAIR + row * SDW + 2 * par + h;
            if constexpr (WHOLE) return s[0];
            const int left = nb - st * STAGE_BLOCKS - 4 * h;  // the bytes of the next row, which may be NaN, give way to zeros
            const uint32_t v = __builtin_amdgcn_alignbyte(s[1], s[0], shift);
            return left >= 4 ? v : (left > 0 ? v & ((1u << (8 * left)) - 1u) : 0u);
        };
        uint32_t xshift[RT], wshift[4];  // bytes from an aligned dword to a row's scales
#pragma unroll
        for (int m = 0; m < RT; ++m) xshift[m] = ((uint32_t)min((wy * RT + m) * 32 + r, t.rows - 1) * nb + (uint32_t)(xs0 & 15)) & 3;
#pragma unroll
        for (int c = 0; c < 4; ++c) wshift[c] = ((uint32_t)min((wx * 4 + c) * 32 + r, cols - 1) * nb + (uint32_t)(ws0 & 15)) & 3;
        // slot of this lane's block of step j in row r of a 32-row tile
        int frag[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) frag[j] = r * 8 + ((4 * h + j) ^ ((r >> 1) & 7));

        // Operands run one step ahead, across the stages' borders: a stage's barrier
        // comes before its last step, when that step's operands are in registers (so
        // the buffer is free) and the next stage has landed.  From there on the last
        // step reads the next stage's first operands and scales and asks for half of
        // the stage after next; the next stage's first step asks for the other half.
        // The loads go between the MFMAs: a wave that issues them in a row waits for
        // the address unit with the matrix core idle.  Stages behind the last re-read it.
        constexpr int MFMAS = 4 * RT, READS = 4 + RT, CODES = (ROW_LOADS + W_LOADS) / 2, EACH = (SCALE_LOADS + 1) / 2;
        const int last = stages - 1;
        i32x4_t xv[2][RT], wv[2][4];
        uint32_t wsc[4], xsc[RT], wsn[4], xsn[RT];  // scales of this stage and the next
        auto read_operand = [&](int k, int j, int par, int to) {  // operand k of step j of a stage of this parity
            const i32x4_t* a = lds + par * STAGE + frag[j];
            if (k < 4) wv[to][k] = a[BM * 8 + (wx * 4 + k) * 256];
            else xv[to][k - 4] = a[(wy * RT + k - 4) * 256];
        };
        auto read_scale = [&](int k, int st, int par) {
            if (k < 4) wsn[k] = scales(BM + (wx * 4 + k) * 32 + r, wshift[k], st, par);
            else xsn[k - 4] = scales((wy * RT + k - 4) * 32 + r, xshift[k - 4], st, par);
        };
#pragma unroll
        for (int k = 0; k < 2 * CODES; ++k) ask_codes(k, 0, 0);
#pragma unroll
        for (int k = 0; k < SCALE_LOADS; ++k) ask_scales(k, so[k], 0);
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < CODES; ++k) ask_codes(k, min(1, last), 1);
#pragma unroll
        for (int k = 0; k < EACH; ++k) ask_scales(k, so[k], 1);
#pragma unroll
        for (int k = 0; k < READS; ++k) {
            read_operand(k, 0, 0, 0);
            read_scale(k, 0, 0);
        }
        for (int st = 0; st < stages; ++st) {
            const int par = st & 1;
#pragma unroll
            for (int c = 0; c < 4; ++c) wsc[c] = wsn[c];
#pragma unroll
            for (int m = 0; m < RT; ++m) xsc[m] = xsn[m];
            auto step = [&](auto jc) {
                constexpr int j = decltype(jc)::value;
                if constexpr (j == 3) {
                    // this step's operands are here, the next stage has landed, in every wave
                    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
                    __builtin_amdgcn_s_barrier();
                    __builtin_amdgcn_sched_barrier(0);
                }
#pragma unroll
                for (int i = 0; i < MFMAS; ++i) {
#pragma unroll
                    for (int k = i * READS / MFMAS; k < (i + 1) * READS / MFMAS; ++k) {
                        read_operand(k, (j + 1) & 3, j == 3 ? par ^ 1 : par, (j + 1) & 1);
                        if constexpr (j == 3) read_scale(k, st + 1, par ^ 1);
                    }
                    if constexpr (j == 0 || j == 3) {
#pragma unroll
                        for (int k = i * CODES / MFMAS; k < (i + 1) * CODES / MFMAS; ++k) {
                            if (j == 3) ask_codes(k, min(st + 2, last), par);
                            else ask_codes(CODES + k, min(st + 1, last), par ^ 1);
                        }
                    }
                    if constexpr (j == 3) {
                        // scales of pair p + 1: one half at stage 2p - 1, the other at 2p
#pragma unroll
                        for (int k = i * EACH / MFMAS; k < (i + 1) * EACH / MFMAS; ++k) {
                            constexpr int end = SCALE_LOADS - 1;
                            ask_scales(par ? k : min(EACH + k, end), par ? so[k] : so[EACH + k < end ? EACH + k : end], ((st + 1) >> 1) + 1);
                        }
                    }
                    acc[i / 4][i % 4] = mfma32<j>(wv[j & 1][i % 4], wsc[i % 4], xv[j & 1][i / 4], xsc[i / 4], acc[i / 4][i % 4]);
                    __builtin_amdgcn_sched_barrier(0);
                }
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            step(std::integral_constant<int, 2>{});
            step(std::integral_constant<int, 3>{});
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the last stage's second copy is here
        __builtin_amdgcn_s_barrier();        // and the buffers are read
    }
    // Results: a lane holds 4 consecutive outputs of a row.  32 rows at a time they
    // go through LDS (this wave's own part), so that a store writes 256 bytes and
    // more of a row.
    constexpr int PITCH = 128 * OT::bytes + 16;
    static_assert(4 * 32 * PITCH <= (int)sizeof(lds), "the waves' parts fit");
    char* part = reinterpret_cast<char*>(lds) + wave * 32 * PITCH;
    const int wcols = min(128, cols - wx * 128);
    const bool vec = (p.n_out * OT::bytes) % 16 == 0;
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        const int mrow = (wy * RT + m) * 32, live = min(32, t.rows - mrow);
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4_t v = {acc[m][c][4 * g], acc[m][c][4 * g + 1], acc[m][c][4 * g + 2], acc[m][c][4 * g + 3]};
                store4<OT>(part + r * PITCH, 32 * c + 8 * g + 4 * h, 4, true, v);
            }
        __builtin_amdgcn_wave_barrier();
        const int64_t y0 = (int64_t)(t.row0 + mrow) * p.n_out + n0 + wx * 128;
        typedef typename OT::raw raw;
        raw* y = static_cast<raw*>(p.y);
        if (vec) {
            constexpr int PER = 16 / OT::bytes, LANES = 128 / PER;  // outputs of a lane, lanes of a row
#pragma unroll
            for (int i = 0; i < 32; i += 64 / LANES) {
                const int row = i + lane / LANES, o = lane % LANES * PER;
                const i32x4_t v = *reinterpret_cast<const i32x4_t*>(part + row * PITCH + o * OT::bytes);
                if (row < live && o < wcols) *reinterpret_cast<i32x4_t*>(y + y0 + (int64_t)row * p.n_out + o) = v;
            }
        } else {
            for (int row = 0; row < live; ++row)
#pragma unroll
                for (int o = 0; o < 128; o += 64) {
                    const raw v = reinterpret_cast<const raw*>(part + row * PITCH)[o + lane];
                    if (o + lane < wcols) y[y0 + (int64_t)row * p.n_out + o + lane] = v;
                }
        }
        __builtin_amdgcn_wave_barrier();
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

template <typename OT, int RT> hipError_t launch_gemm(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 64 * RT), cols = (p.n_out + 255) / 256;
    const int64_t tiles = xcd_padded(rows * cols);
    if (tiles > 0x7FFFFFFF) return hipErrorInvalidConfiguration;
    if (p.n_in % (4 * BLOCK) == 0) gemm_kernel<OT, RT, true><<<(unsigned)tiles, 256, 0, s>>>(p, (int)rows, (int)cols);
    else gemm_kernel<OT, RT, false><<<(unsigned)tiles, 256, 0, s>>>(p, (int)rows, (int)cols);
    return hipGetLastError();
}

template <typename OT> hipError_t launch_product(const ProductParams& p, hipStream_t s) {
    const int64_t m = typical_rows(p.rows, p.n_groups);
    if (p.x) return launch_skinny<OT, true, 1, 1>(p, s);
    if (m <= 16) return launch_skinny<OT, false, 1, 1>(p, s);
    if (m <= 32) return launch_skinny<OT, false, 2, 1>(p, s);
    if (m <= SKINNY_MAX_ROWS) return launch_skinny<OT, false, 4, 1>(p, s);
    if (m <= 128) return launch_gemm<OT, 2>(p, s);
    return launch_gemm<OT, 4>(p, s);
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
