// mxfp4.hip - MXFP4 quantisation, dequantisation and products (gfx950).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../../include/exl3_mxfp4.h"
#include "mxfp4_device.hpp"
#include "spans.hpp"

namespace exl3 {
namespace mx {

// ---- quantise: values to codes and scales ----
//
// A lane takes 8 consecutive values, four lanes a block: the block's largest
// magnitude is a maximum over the quad (two DPP moves), then each lane converts
// its own values to one dword of codes, so codes leave a wave as 256 consecutive
// bytes.  Memory bounds it: 28672 x 8192 fp16 values in 127 us, 4.7 TB/s of reads
// and writes (a copy reaches 5.2).
template <typename T> __device__ inline uint32_t quantize_quad(const uint32_t (&w)[2 * T::bytes], uint32_t& b) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 2 * T::bytes; ++e) m = abs_max<T>(m, w[e]);
    uint32_t a = abs_max_f32_bits<T>(m);
    uint32_t o = (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true);  // lanes 1 0 3 2
    a = a > o ? a : o;
    o = (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, true);  // lanes 2 3 0 1
    a = a > o ? a : o;
    b = scale_byte(a);
    const uint32_t c = cvt8<T>(w, scale_value(b));
    return b == 255u ? 0u : c;
}

// Loads in flight a thread: four, or one where that leaves most CUs without a
// workgroup (13 x 14336 bf16 values: 1 us less; 1.9 from a graph, 2.8 traced).
constexpr int QUANT_UNROLL = 4;

template <typename T, bool FLAT, int U>
__global__ __launch_bounds__(256) void quantize_kernel(const void* __restrict__ xv, int64_t rows, int n, int64_t ldx,
                                                       uint32_t* __restrict__ codes, uint8_t* __restrict__ scales) {
    constexpr int NW = T::bytes == 2 ? 4 : 8;  // dwords of 8 values
    const int64_t units = rows * (n / 8);
    const int64_t base = (int64_t)blockIdx.x * 256 * U + threadIdx.x;
    uint32_t w[U][NW];
#pragma unroll
    for (int u = 0; u < U; ++u) {
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
    for (int u = 0; u < U; ++u) {
        const int64_t i = base + u * 256;
        if (i >= units) continue;  // whole quads: units is a multiple of 4
        uint32_t b;
        codes[i] = quantize_quad<T>(w[u], b);
        if ((i & 3) == 0) scales[i >> 2] = (uint8_t)b;
    }
}

// ---- dequantise: codes and scales to values ----
//
// A lane makes 8 values of one dword of codes.  28672 x 8192 fp16 values in 117 us,
// 5.1 TB/s.
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
    int ldy;  // outputs from a row of y to the next: n_out, or more where this launch makes some of the columns
};

// Memory from `base` on, read at 32-bit offsets.
__device__ inline __amdgpu_buffer_rsrc_t buffer(const uint8_t* base, int64_t bytes) {
    const uint32_t n = bytes > 0x7FFFFFFF ? 0x7FFFFFFFu : (uint32_t)bytes;
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(base), 0, n, 0x00020000);
}
// Straight into LDS: lane l's 16 bytes at dst + 16 l.
__device__ inline void load16_to_lds(__amdgpu_buffer_rsrc_t b, i32x4_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}
constexpr uint32_t OUTSIDE = 0x7FFFFFF0u;  // an offset past every buffer: the load gives zeros

__device__ inline void load4_to_lds(__amdgpu_buffer_rsrc_t b, uint32_t* dst, uint32_t voff, uint32_t soff) {
    __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (__attribute__((address_space(3))) void*)dst, 4, voff, soff, 0, 0);
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

// Dwords of scales that a row of a span holds in LDS: its 16 bytes, or where rows
// start at any byte (WHOLE false: n_in % 128 != 0) the aligned dwords around them.
template <bool WHOLE> constexpr int SCALE_DWORDS = WHOLE ? 4 : 8;

// Four scale bytes out of staged dwords: s[0], or with a row that starts `shift`
// bytes into a dword s[0] and s[1].  `left` blocks of the row are left from the
// first of these on; bytes of the next row, which may stand for NaN, give way to zeros.
template <bool WHOLE> __device__ inline uint32_t staged_scales(const uint32_t* s, uint32_t shift, int left) {
    if constexpr (WHOLE) return s[0];
    const uint32_t v = __builtin_amdgcn_alignbyte(s[1], s[0], shift);
    return left >= 4 ? v : (left > 0 ? v & ((1u << (8 * left)) - 1u) : 0u);
}
// The offset of dword `dw` of a span's staged scales, or OUTSIDE behind the row's end.
template <bool WHOLE> __device__ inline uint32_t scale_offset(uint32_t row_first, int dw, int span, int nb) {
    return span * SPAN_BLOCKS + 4 * dw < nb + (WHOLE ? 0 : 4) ? (row_first & ~3u) + 4 * dw : OUTSIDE;
}

// A tile of one side of a product: codes and scales of `rows` rows from row
// `first` of a matrix of nb blocks a row.
struct Side {
    __amdgpu_buffer_rsrc_t codes, scales;
    uint32_t lead;  // bytes from the scale buffer's 16-byte border to the first row's
    int rows;
};
__device__ inline Side side(const uint8_t* codes, const uint8_t* scales, int64_t first, int rows, int nb) {
    const int64_t at = first * nb;
    return Side{buffer(codes + at * 16, (int64_t)rows * nb * 16),
                buffer(scales + (at & ~int64_t(15)), ((at & 15) + (int64_t)rows * nb + 3) & ~int64_t(3)), (uint32_t)(at & 15), rows};
}

// Few rows: eight waves, `split` of them on each run of 16 outputs (8 / split runs
// a workgroup), for up to 16 rows; of a run's waves, wave w takes the spans w,
// w + split, ... of the input.  Each wave brings its spans of the weight straight
// into a ring of its own in LDS, four rows of 256 bytes a load, and waits for
// nobody (a weight operand read from memory by its lanes would be 64 places for
// 1 KB, 64 cycles of the address unit instead of 16).  The rows come quantised, the
// same way (STREAMED), or, up to HELD spans of them, all rows together, the
// workgroup brings them into LDS first, while the weight is on its way: quantised
// ones (STAGED), or values that it quantises (QUANTISED).  With HELD_SPANS two
// workgroups fit a CU: 2048 rows in 256 groups 1024 -> 1024 35 us staged against 57
// streamed; where scales start at any byte too, as they take 5 dwords a row (one row
// 4128 -> 14336 10.4 us; 12.4 with 8 dwords and one workgroup a CU, 9.5 for 4096).
// A run's sums meet in LDS and are added in the order of its waves.
//
// Block b of row r sits in 16-byte slot b ^ swizzle(r): the 16 lanes that LDS
// serves together (rows 0-3 and 12-15 of one quarter, 4-11 of the next) then
// read 16 different slots of its 256-byte width.
//
// The weight's bytes bound it where there are many: one row 8192 -> 28672 in 25.3
// us, 5.0 TB/s; three tokens through two of eight experts 4096 -> 14336 in 23 us.
// A short launch is its start, the rows' and the weight's latency and the sums:
// one row 4096 -> 4096 in 4.7 us, of which 1.7 are the weight's at the copy rate.
enum Rows { STREAMED, STAGED, QUANTISED };

__device__ inline int small_swizzle(int row) {  // rows / 4: 0 1 2 3 -> 0 2 3 1
    return (row & 3) | (((0x78 >> (row >> 2 << 1)) & 3) << 2);
}

template <typename OT, Rows ROWS, int HELD, bool WHOLE>
__global__ __launch_bounds__(SMALL_WAVES * 64) void small_kernel(const ProductParams p, int split) {
    constexpr int SDW = small_scale_dwords(WHOLE), SIDES = HELD ? 1 : 2, SCALE_LOADS = (16 * SDW + 63) / 64, LOADS = SIDES * (4 + SCALE_LOADS);
    constexpr int BUF = small_buf_slots(HELD, WHOLE);  // slots: codes of each side, then scales
    constexpr int RING = SMALL_WAVES * SMALL_RING * BUF;
    __shared__ i32x4_t lds[small_slots(HELD, WHOLE)];  // the rings, and the held rows: codes, scales
    static_assert(HELD != HELD_SPANS || small_per_cu(HELD, WHOLE) == 2, "two workgroups a CU");
    static_assert(SMALL_RING * BUF >= 64, "the sums of a wave fit its ring");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, blockIdx.y, HELD ? held_rows(p.n_in, HELD) : SMALL_MAX_ROWS);
    if (t.rows == 0) return;
    const int first = wave % split;  // of the run's spans
    const int n0 = (blockIdx.x * (SMALL_WAVES / split) + wave / split) * 16, cols = min(16, p.n_out - n0);
    const int nb = p.n_in / BLOCK, spans = (nb + SPAN_BLOCKS - 1) / SPAN_BLOCKS;
    i32x4_t* const ring = lds + wave * SMALL_RING * BUF;

    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    if (t.group < p.n_groups) {
        const int mine = cols > 0 ? (spans - first + split - 1) / split : 0;  // spans of this wave
        Side sides[SIDES];
        sides[0] = side(p.wc, p.ws, (int64_t)t.group * p.n_out + (cols > 0 ? n0 : 0), max(cols, 1), nb);
        if constexpr (!HELD) sides[1] = side(p.xc, p.xs, t.row0, t.rows, nb);
        uint32_t row_at[SIDES][4], scale_at[SIDES][SCALE_LOADS], shift[SIDES];
        // load i of a side's scales: 64 of its 16 SDW dwords; the second of 80 brings
        // some of the first's again rather than run over the end
        auto scale_first = [](int i) { return min(64 * i, 16 * SDW - 64); };
#pragma unroll
        for (int s = 0; s < SIDES; ++s) {
            // load i: row 4 i + lane / 16, slot lane % 16; rows behind the tile re-read its last
#pragma unroll
            for (int i = 0; i < 4; ++i) row_at[s][i] = (uint32_t)min(4 * i + (lane >> 4), sides[s].rows - 1) * (nb * 16);
#pragma unroll
            for (int i = 0; i < SCALE_LOADS; ++i)
                scale_at[s][i] = (uint32_t)min((scale_first(i) + lane) / SDW, sides[s].rows - 1) * nb + sides[s].lead;
            shift[s] = ((uint32_t)min(r, sides[s].rows - 1) * nb + sides[s].lead) & 3u;
        }
        // The loads of this wave's kth span; behind its last they give zeros.
        auto ask = [&](int k) {
            const int sp = k < mine ? first + k * split : spans;
            i32x4_t* const buf = ring + k % SMALL_RING * BUF;
#pragma unroll
            for (int s = 0; s < SIDES; ++s) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int block = (lane & 15) ^ small_swizzle(4 * i + (lane >> 4));
                    load16_to_lds(sides[s].codes, buf + s * 256 + i * 64, sp * SPAN_BLOCKS + block < nb ? row_at[s][i] + 16 * block : OUTSIDE,
                                  (uint32_t)sp * 256);
                }
#pragma unroll
                for (int i = 0; i < SCALE_LOADS; ++i)
                    load4_to_lds(sides[s].scales, reinterpret_cast<uint32_t*>(buf + SIDES * 256 + s * 4 * SDW) + scale_first(i),
                                 scale_offset<WHOLE>(scale_at[s][i], (scale_first(i) + lane) % SDW, sp, nb), (uint32_t)sp * SPAN_BLOCKS);
            }
        };
        auto scales = [&](int s, int k, int left) {
            const uint32_t* at = reinterpret_cast<const uint32_t*>(ring + k % SMALL_RING * BUF + SIDES * 256 + s * 4 * SDW);
            return staged_scales<WHOLE>(at + r * SDW + q, shift[s], left);
        };
        auto operand = [&](int s, int k, int j) { return ring[k % SMALL_RING * BUF + s * 256 + r * 16 + ((4 * q + j) ^ small_swizzle(r))]; };
        i32x4_t* const xq = lds + RING;  // [row][spans * 16], block b of row r at b ^ small_swizzle(r)
        uint8_t* const xq_scales = reinterpret_cast<uint8_t*>(xq + HELD * 16);
#pragma unroll
        for (int k = 0; k < SMALL_RING; ++k) ask(k);
        if constexpr (ROWS == STAGED) {
            // a block a thread; zeros behind a row's end
            static_assert(HELD * SPAN_BLOCKS <= SMALL_WAVES * 64, "a thread for each");
            const int row = threadIdx.x / (spans * SPAN_BLOCKS), block = threadIdx.x - row * spans * SPAN_BLOCKS;
            if (row < t.rows) {
                const int64_t at = (int64_t)(t.row0 + row) * nb + block;
                i32x4_t c = {0, 0, 0, 0};
                uint8_t b = 0;
                if (block < nb) {
                    c = *reinterpret_cast<const i32x4_t*>(p.xc + at * 16);
                    b = p.xs[at];
                }
                xq[row * spans * 16 + (block ^ small_swizzle(row))] = c;
                xq_scales[row * spans * 16 + block] = b;
            }
            __syncthreads();
        }
        if constexpr (ROWS == QUANTISED) {
            // eight values a thread and round, four threads a block, as quantize_kernel
            constexpr int THREADS = SMALL_WAVES * 64, ROUNDS = 4, NW = 2 * OT::bytes;
            const int per_row = spans * 64, units = t.rows * per_row;
            for (int u0 = threadIdx.x; u0 < units; u0 += ROUNDS * THREADS) {
                uint32_t w[ROUNDS][NW];
#pragma unroll
                for (int i = 0; i < ROUNDS; ++i) {
                    const int u = u0 + i * THREADS, row = u / per_row, at = u - row * per_row;
#pragma unroll
                    for (int e = 0; e < NW; ++e) w[i][e] = 0;
                    if (u < units && at < nb * 4) {
                        const int64_t from = (int64_t)(t.row0 + row) * p.ldx + 8 * at;
                        const u32x4_t* src = reinterpret_cast<const u32x4_t*>(static_cast<const char*>(p.x) + from * OT::bytes);
#pragma unroll
                        for (int c = 0; c < NW / 4; ++c) {
                            const u32x4_t v = src[c];
#pragma unroll
                            for (int e = 0; e < 4; ++e) w[i][4 * c + e] = v[e];
                        }
                    }
                }
#pragma unroll
                for (int i = 0; i < ROUNDS; ++i) {
                    const int u = u0 + i * THREADS, row = u / per_row, at = u - row * per_row;
                    if (u < units) {  // whole quads
                        uint32_t b;
                        const uint32_t c = quantize_quad<OT>(w[i], b);
                        const int slot = row * spans * 16 + ((at >> 2) ^ small_swizzle(row));
                        reinterpret_cast<uint32_t*>(xq + slot)[at & 3] = c;
                        if ((at & 3) == 0) xq_scales[row * spans * 16 + (at >> 2)] = (uint8_t)b;
                    }
                }
            }
            __syncthreads();
        }
        for (int k = 0; k < mine; ++k) {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0x0F70 | ((SMALL_RING - 1) * LOADS & 15) | (((SMALL_RING - 1) * LOADS >> 4) << 14));  // vmcnt
            __builtin_amdgcn_sched_barrier(0);
            const int sp = first + k * split, left = nb - sp * SPAN_BLOCKS - 4 * q;
            i32x4_t wv[4], xv[4];
            uint32_t xsc;
#pragma unroll
            for (int j = 0; j < 4; ++j) wv[j] = operand(0, k, j);
            const uint32_t wsc = scales(0, k, left);
            if constexpr (HELD) {
                const int row = min(r, t.rows - 1);  // rows behind the tile re-read its last
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[j] = xq[(row * spans + sp) * 16 + ((4 * q + j) ^ small_swizzle(row))];
                xsc = reinterpret_cast<const uint32_t*>(xq_scales)[(row * spans + sp) * 4 + q];
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) xv[j] = operand(1, k, j);
                xsc = scales(1, k, left);
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read
            __builtin_amdgcn_sched_barrier(0);
            ask(k + SMALL_RING);
            acc = mfma<0>(wv[0], wsc, xv[0], xsc, acc);
            acc = mfma<1>(wv[1], wsc, xv[1], xsc, acc);
            acc = mfma<2>(wv[2], wsc, xv[2], xsc, acc);
            acc = mfma<3>(wv[3], wsc, xv[3], xsc, acc);
        }
        __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): nothing is on its way into LDS any more
    }
    // each wave's sums over its own ring
    ring[lane] = __builtin_bit_cast(i32x4_t, acc);
    __syncthreads();
    if (first == 0) {
        f32x4_t v = acc;
        for (int w = 1; w < split; ++w) v += __builtin_bit_cast(f32x4_t, ring[w * SMALL_RING * BUF + lane]);
        const int o = n0 + 4 * q;
        if (r < t.rows && o < p.n_out) store4<OT>(p.y, (int64_t)(t.row0 + r) * p.ldy + o, p.n_out - o, (p.ldy & 3) == 0, v);
    }
}

// Workgroup b of a launch to tile index: units of 16 consecutive tiles go to the
// same XCD (workgroups go round the 8 XCDs one by one), so that the tiles that
// run together on an XCD share rows and weights in its L2.  Units of 8 to 32 and
// bands of 2 to 16 measure the same within 3 %, but for 4096 rows in 64 groups 2048
// -> 2816: 54 us against 61 with units of 32 in bands of 8 (empty tiles, which end
// at once, then come in longer runs of one XCD); units of 64 are 15 to 80 % slower.
constexpr int XCDS = 8, XCD_UNIT = 16;
__device__ inline int xcd_tile(int b) {
    const int xcd = b % XCDS, local = b / XCDS;
    return (local / XCD_UNIT * XCDS + xcd) * XCD_UNIT + local % XCD_UNIT;
}
// Tiles of a launch, padded to whole rounds of units.
inline int64_t xcd_padded(int64_t tiles) { return (tiles + XCDS * XCD_UNIT - 1) / (XCDS * XCD_UNIT) * (XCDS * XCD_UNIT); }
constexpr int BAND = 4;  // row tiles that share a run of output tiles
// Row tile and output tile of a tile index: bands of BAND row tiles, an output
// tile's row tiles after each other.  False behind the last tile.
__device__ inline bool tile_of(int tile, int row_tiles, int col_tiles, int* row, int* col) {
    const int band = tile / (BAND * col_tiles), height = min(BAND, row_tiles - band * BAND);
    if (height <= 0) return false;
    const int in_band = tile - band * BAND * col_tiles;
    *col = in_band / height;
    *row = band * BAND + in_band - *col * height;
    return *col < col_tiles;
}

// A wave's results, 32 RT rows from `row0` and 32 CT outputs from `col0`, of which
// `rows` rows are written.  A lane holds 4 consecutive outputs of a row; 32 rows
// at a time they go through LDS (`part`, the wave's own), so that a store writes
// whole pieces of a row, 64 CT bytes and more.
template <typename OT, int CT> constexpr int store_part_bytes() { return 32 * (32 * CT * OT::bytes + 16); }

template <typename OT, int RT, int CT>
__device__ inline void store_tile(const f32x16_t (&acc)[RT][CT], char* part, const ProductParams& p, int row0, int rows, int col0) {
    typedef typename OT::raw raw;
    constexpr int PITCH = 32 * CT * OT::bytes + 16;
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int cols = min(32 * CT, p.n_out - col0);
    const bool vec = ((int64_t)p.ldy * OT::bytes) % 16 == 0 && p.n_out % (16 / OT::bytes) == 0;
    raw* y = static_cast<raw*>(p.y);
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        const int live = min(32, rows - 32 * m);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const f32x4_t v = {acc[m][c][4 * g], acc[m][c][4 * g + 1], acc[m][c][4 * g + 2], acc[m][c][4 * g + 3]};
                store4<OT>(part + r * PITCH, 32 * c + 8 * g + 4 * h, 4, true, v);
            }
        __builtin_amdgcn_wave_barrier();
        const int64_t y0 = (int64_t)(row0 + 32 * m) * p.ldy + col0;
        if (vec) {
            constexpr int PER = 16 / OT::bytes, LANES = 32 * CT / PER;  // outputs of a lane, lanes of a row
#pragma unroll
            for (int i = 0; i < 32; i += 64 / LANES) {
                const int row = i + lane / LANES, o = lane % LANES * PER;
                const i32x4_t v = *reinterpret_cast<const i32x4_t*>(part + row * PITCH + o * OT::bytes);
                if (row < live && o < cols) *reinterpret_cast<i32x4_t*>(y + y0 + (int64_t)row * p.ldy + o) = v;
            }
        } else {
            for (int i = lane; i < live * 32 * CT; i += 64) {
                const int row = i / (32 * CT), o = i % (32 * CT);
                const raw v = reinterpret_cast<const raw*>(part + row * PITCH)[o];
                if (o < cols) y[y0 + (int64_t)row * p.ldy + o] = v;
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

// Some rows, or few tiles: a workgroup of four waves owns T rows and T outputs.
// Stages of a span (256 bytes of codes a row of both sides) go straight into a
// ring in LDS, all but one of it ahead: a stage is little work, so it is the bytes
// in flight that count.  T = 64: each wave a quarter of the tile, 8 MFMAs a stage.
// T = 32: each wave the whole tile over a quarter of the stage's inputs, and the
// waves' sums meet in LDS at the end; four times the workgroups where 64 x 64
// tiles would leave most of the card idle.  Block b of row r sits in slot
// b ^ (r & 15) of the row's 256 bytes.
//
// 256 rows 4096 -> 4096 in 9.0 us (256 tiles, one a CU): 5 us of it is start and
// first latency, the rest 0.5 us a stage, where 100 KB in flight a CU meet a latency
// of 1.5 us.  64 rows 14336 -> 4096 in 15 us (T = 32).
template <int T> constexpr int MEDIUM_RING = T == 64 ? 4 : 8;

template <typename OT, int T, bool WHOLE>
__global__ __launch_bounds__(256) void medium_kernel(const ProductParams p, int row_tiles, int col_tiles) {
    constexpr int SDW = SCALE_DWORDS<WHOLE>, RING = MEDIUM_RING<T>;
    constexpr int CODE_LOADS = T / 8, SCALE_LOADS = T * SDW / 128, LOADS = CODE_LOADS + SCALE_LOADS;  // of a wave and stage
    constexpr int BUF = 2 * T * 16 + 2 * T * SDW / 4;  // slots: codes (rows, then weight rows), then scales
    constexpr int STEPS = T == 64 ? 8 : 2;             // MFMAs of a wave and stage
    static_assert(store_part_bytes<OT, 1>() * 4 <= RING * BUF * 16, "the waves' parts fit");
    __shared__ i32x4_t lds[RING * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, wy = T == 64 ? wave >> 1 : 0, wx = T == 64 ? wave & 1 : 0;
    int row_tile, col;
    if (!tile_of(xcd_tile(blockIdx.x), row_tiles, col_tiles, &row_tile, &col)) return;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, row_tile, T);
    if (t.rows == 0) return;
    const int n0 = col * T, cols = min(T, p.n_out - n0);
    const int nb = p.n_in / BLOCK, stages = (nb + SPAN_BLOCKS - 1) / SPAN_BLOCKS;

    f32x16_t acc[1][1];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[0][0][i] = 0.f;

    if (t.group < p.n_groups) {
        const Side x = side(p.xc, p.xs, t.row0, t.rows, nb), w = side(p.wc, p.ws, (int64_t)t.group * p.n_out + n0, cols, nb);
        // Rows of both sides together, the weight's from T on.  Load i of a wave: row
        // 16 i + 4 wave + lane / 16, slot lane % 16; rows behind a side's end re-read its last.
        const int srow = 4 * wave + (lane >> 4), block = (lane & 15) ^ srow;
        uint32_t row_at[CODE_LOADS], scale_at[SCALE_LOADS];
#pragma unroll
        for (int i = 0; i < CODE_LOADS; ++i) {
            const int row = 16 * i + srow;
            row_at[i] = (uint32_t)(16 * i < T ? min(row, x.rows - 1) : min(row - T, w.rows - 1)) * (nb * 16) + 16 * block;
        }
#pragma unroll
        for (int i = 0; i < SCALE_LOADS; ++i) {
            const int row = (4 * i + wave) * (64 / SDW) + lane / SDW;
            scale_at[i] = row < T ? (uint32_t)min(row, x.rows - 1) * nb + x.lead : (uint32_t)min(row - T, w.rows - 1) * nb + w.lead;
        }
        const uint32_t xshift = ((uint32_t)min(wy * 32 + r, x.rows - 1) * nb + x.lead) & 3u;
        const uint32_t wshift = ((uint32_t)min(wx * 32 + r, w.rows - 1) * nb + w.lead) & 3u;
        auto ask = [&](int st) {  // behind the last stage: zeros
            i32x4_t* const buf = lds + st % RING * BUF;
#pragma unroll
            for (int i = 0; i < CODE_LOADS; ++i)
                load16_to_lds(16 * i < T ? x.codes : w.codes, buf + i * 256 + wave * 64, st * SPAN_BLOCKS + block < nb ? row_at[i] : OUTSIDE,
                              (uint32_t)st * 256);
#pragma unroll
            for (int i = 0; i < SCALE_LOADS; ++i)
                load4_to_lds((4 * i + wave) * (64 / SDW) < T ? x.scales : w.scales, reinterpret_cast<uint32_t*>(buf + 2 * T * 16) + (4 * i + wave) * 64,
                             scale_offset<WHOLE>(scale_at[i], lane % SDW, st, nb), (uint32_t)st * SPAN_BLOCKS);
        };
#pragma unroll
        for (int k = 0; k < RING - 1; ++k) ask(k);
        for (int st = 0; st < stages; ++st) {
            // this stage has landed in every wave, and the one before it is read
            constexpr int PENDING = (RING - 2) * LOADS;
            static_assert(PENDING < 64, "a wait counts to 63");
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_waitcnt(0x0070 | (PENDING & 15) | ((PENDING >> 4) << 14));  // lgkmcnt(0), vmcnt(PENDING)
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            ask(st + RING - 1);
            // This lane's blocks: T = 64, the 8 of its half, two dwords of scales; T = 32,
            // two of the wave's four, h and h + 2, so that one dword holds the scales.
            const i32x4_t* const buf = lds + st % RING * BUF;
            const int first = T == 64 ? 8 * h : 4 * wave, left = nb - st * SPAN_BLOCKS - first;
            const uint32_t* const xs = reinterpret_cast<const uint32_t*>(buf + 2 * T * 16) + (wy * 32 + r) * SDW + first / 4;
            const uint32_t* const ws = reinterpret_cast<const uint32_t*>(buf + 2 * T * 16) + (T + wx * 32 + r) * SDW + first / 4;
            uint32_t xsc[T / 32], wsc[T / 32];
#pragma unroll
            for (int e = 0; e < T / 32; ++e) {
                xsc[e] = staged_scales<WHOLE>(xs + e, xshift, left - 4 * e);
                wsc[e] = staged_scales<WHOLE>(ws + e, wshift, left - 4 * e);
            }
            if constexpr (T == 32) {  // bytes h and h + 2 to 0 and 2
                xsc[0] >>= 8 * h;
                wsc[0] >>= 8 * h;
            }
            auto step = [&](auto jc) {
                constexpr int j = decltype(jc)::value;
                const int slot = (T == 64 ? 8 * h + j : first + h + 2 * j) ^ (r & 15);
                const i32x4_t xv = buf[(wy * 32 + r) * 16 + slot], wv = buf[(T + wx * 32 + r) * 16 + slot];
                acc[0][0] = mfma32<T == 64 ? j & 3 : 2 * j>(wv, wsc[T == 64 ? j >> 2 : 0], xv, xsc[T == 64 ? j >> 2 : 0], acc[0][0]);
            };
            step(std::integral_constant<int, 0>{});
            step(std::integral_constant<int, 1>{});
            if constexpr (STEPS == 8) {
                step(std::integral_constant<int, 2>{});
                step(std::integral_constant<int, 3>{});
                step(std::integral_constant<int, 4>{});
                step(std::integral_constant<int, 5>{});
                step(std::integral_constant<int, 6>{});
                step(std::integral_constant<int, 7>{});
            }
        }
        __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0): nothing is on its way, the ring is read
        __builtin_amdgcn_s_barrier();
    }
    if constexpr (T == 32) {
        // the four waves' sums, added in order by wave 0
        f32x16_t* const sums = reinterpret_cast<f32x16_t*>(lds);
        if (wave > 0) sums[(wave - 1) * 64 + lane] = acc[0][0];
        __syncthreads();
        if (wave > 0) return;
#pragma unroll
        for (int v = 0; v < 3; ++v) acc[0][0] += sums[v * 64 + lane];
        __builtin_amdgcn_wave_barrier();
    }
    constexpr int PART = store_part_bytes<OT, 1>();
    store_tile<OT, 1, 1>(acc, reinterpret_cast<char*>(lds) + wave * PART, p, t.row0 + wy * 32, t.rows - wy * 32, n0 + wx * 32);
}

// Many rows: a workgroup of four waves owns 64 RT rows and 64 CT outputs, each wave
// a quarter of them, 32 RT rows and 32 CT outputs.  Stages of 256 inputs (128
// bytes of codes a row) of both sides go straight from memory into LDS, double
// buffered; the waves read their operands from there.  (A weight operand read from
// memory by its lanes would touch 64 cache lines for 1 KB.)
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
//
// 256 x 256 tiles (one workgroup a CU): 8192^3 in 260 us, 4.2 PFLOP/s, half of the
// 8.4 that the matrix cores issue alone; 2048 rows 8192 -> 28672 in 260 us with the
// 128 x 128 tiles of the last columns.  The matrix cores are busy 57 % of the cycles
// at 1.66 GHz: one wave a SIMD waits at each stage's border with nothing else to
// run, and the clock falls under load (zeros for codes: 2.11 GHz, 15 % faster).
// 128 x 128 tiles (two a CU): 16384 rows in 64 groups 2048 -> 2816 in 105 to 131 us.
// No unit is full (matrix cores busy 26 %, address units 57 %); waves wait for data or
// a barrier 44 % of their time, as a stage's loads have one stage to land.

constexpr int STAGE_BLOCKS = 8;

template <typename OT, int RT, int CT, bool WHOLE>
__global__ __launch_bounds__(256, RT * CT > 4 ? 1 : 2) void gemm_kernel(const ProductParams p, int row_tiles, int col_tiles) {
    constexpr int BM = 64 * RT, BN = 64 * CT;
    constexpr int STAGE = (BM + BN) * 8;  // 16-byte slots: the rows', then the weight's
    constexpr int ROW_LOADS = BM / 32, W_LOADS = BN / 32;  // a wave's loads per stage, 8 rows each
    constexpr int SDW = WHOLE ? 4 : 8;    // dwords of scales a row holds in LDS
    constexpr int SPAIR = (BM + BN) * SDW, SCALE_LOADS = (BM + BN) * SDW / 256;
    __shared__ i32x4_t lds[2 * STAGE + SPAIR / 2];  // one object: the compiler then keeps loads into it in flight over reads of it
    uint32_t* const lds_scales = reinterpret_cast<uint32_t*>(lds + 2 * STAGE);
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 31, h = lane >> 5, wy = wave >> 1, wx = wave & 1;
    int row_tile, col;
    if (!tile_of(xcd_tile(blockIdx.x), row_tiles, col_tiles, &row_tile, &col)) return;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, row_tile, BM);
    if (t.rows == 0) return;
    const int n0 = col * BN, cols = min(BN, p.n_out - n0);
    const int nb = p.n_in / BLOCK, stages = (nb + STAGE_BLOCKS - 1) / STAGE_BLOCKS;
    const int half = p.n_in / 2;

    f32x16_t acc[RT][CT];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c)
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
        uint32_t xshift[RT], wshift[CT];  // bytes from an aligned dword to a row's scales
#pragma unroll
        for (int m = 0; m < RT; ++m) xshift[m] = ((uint32_t)min((wy * RT + m) * 32 + r, t.rows - 1) * nb + (uint32_t)(xs0 & 15)) & 3;
#pragma unroll
        for (int c = 0; c < CT; ++c) wshift[c] = ((uint32_t)min((wx * CT + c) * 32 + r, cols - 1) * nb + (uint32_t)(ws0 & 15)) & 3;
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
        constexpr int MFMAS = CT * RT, READS = CT + RT, CODES = (ROW_LOADS + W_LOADS) / 2, EACH = (SCALE_LOADS + 1) / 2;
        const int last = stages - 1;
        i32x4_t xv[2][RT], wv[2][CT];
        uint32_t wsc[CT], xsc[RT], wsn[CT], xsn[RT];  // scales of this stage and the next
        auto read_operand = [&](int k, int j, int par, int to) {  // operand k of step j of a stage of this parity
            const i32x4_t* a = lds + par * STAGE + frag[j];
            if (k < CT) wv[to][k] = a[BM * 8 + (wx * CT + k) * 256];
            else xv[to][k - CT] = a[(wy * RT + k - CT) * 256];
        };
        auto read_scale = [&](int k, int st, int par) {
            if (k < CT) wsn[k] = scales(BM + (wx * CT + k) * 32 + r, wshift[k], st, par);
            else xsn[k - CT] = scales((wy * RT + k - CT) * 32 + r, xshift[k - CT], st, par);
        };
        // both buffers are asked for before the first is waited for
#pragma unroll
        for (int k = 0; k < 2 * CODES; ++k) ask_codes(k, 0, 0);
#pragma unroll
        for (int k = 0; k < SCALE_LOADS; ++k) ask_scales(k, so[k], 0);
#pragma unroll
        for (int k = 0; k < 2 * CODES; ++k) ask_codes(k, min(1, last), 1);
#pragma unroll
        for (int k = 0; k < EACH; ++k) ask_scales(k, so[k], 1);
        constexpr int YOUNGER = 2 * CODES + EACH;
        static_assert(YOUNGER < 64, "a wait counts to 63");
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_waitcnt(0x0F70 | (YOUNGER & 15) | ((YOUNGER >> 4) << 14));  // vmcnt(YOUNGER)
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int k = 0; k < READS; ++k) {
            read_operand(k, 0, 0, 0);
            read_scale(k, 0, 0);
        }
        for (int st = 0; st < stages; ++st) {
            const int par = st & 1;
#pragma unroll
            for (int c = 0; c < CT; ++c) wsc[c] = wsn[c];
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
                            else if (st > 0) ask_codes(CODES + k, min(st + 1, last), par ^ 1);
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
                    acc[i / CT][i % CT] = mfma32<j>(wv[j & 1][i % CT], wsc[i % CT], xv[j & 1][i / CT], xsc[i / CT], acc[i / CT][i % CT]);
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
    constexpr int PART = store_part_bytes<OT, CT>();
    static_assert(4 * PART <= (int)sizeof(lds), "the waves' parts fit");
    store_tile<OT, RT, CT>(acc, reinterpret_cast<char*>(lds) + wave * PART, p, t.row0 + wy * RT * 32, t.rows - wy * RT * 32, n0 + wx * CT * 32);
}

// ---- launches ----

template <typename T, int U> hipError_t launch_quantize(const void* x, int64_t rows, int n, int64_t ldx, uint8_t* codes,
                                                        uint8_t* scales, hipStream_t s) {
    const dim3 grid((unsigned)((rows * (n / 8) + 256 * U - 1) / (256 * U)));
    uint32_t* const c = reinterpret_cast<uint32_t*>(codes);
    if (ldx == n || rows == 1) quantize_kernel<T, true, U><<<grid, 256, 0, s>>>(x, rows, n, ldx, c, scales);
    else quantize_kernel<T, false, U><<<grid, 256, 0, s>>>(x, rows, n, ldx, c, scales);
    return hipGetLastError();
}

template <typename T> hipError_t launch_quantize(const void* x, int64_t rows, int n, int64_t ldx, uint8_t* codes,
                                                 uint8_t* scales, hipStream_t s) {
    const bool few = rows * (n / 8) < 256 * 256 * QUANT_UNROLL;
    return few ? launch_quantize<T, 1>(x, rows, n, ldx, codes, scales, s) : launch_quantize<T, QUANT_UNROLL>(x, rows, n, ldx, codes, scales, s);
}

// Rows that a group has on average, those behind the last group counted: what a
// tile's height is chosen by, as the host knows no more of a route.  An uneven one
// takes the same height: all of 256 rows in one of 64 groups 4096 -> 2816 34 us, 64
// tiles of 4 rows that each read that group's weight (77 for an even route, which
// reads every weight; 11 for a product of one weight), 512 rows 2048 -> 2816 24 (42;
// 13), 2048 rows 20 (55; 20).
inline int64_t typical_rows(int64_t rows, int n_groups) { return (rows + n_groups - 1) / n_groups; }

// The spans that a product's workgroups hold in LDS, where a tile of them holds a
// group's rows; 0 where it holds none.  A product of values then quantises them
// itself, without a launch and the codes' way through memory (us, with the
// quantisation: one row 4096 -> 4096 5.0 against 7.0, 8192 -> 28672 25.6 against 31;
// 4 rows of each of 64 groups 2048 -> 2816 32 against 39; equal at 8, and 16 rows of
// each of 512 groups 1024 -> 1024 115 against 93).  More than HELD_SPANS: 5 rows
// 4096 -> 14336 9.1 against 11.0, 8 rows 9.9 against 10.9, but 12 rows (96 spans)
// 11.4 against 11.1, 8192 -> 4096 4 rows 8.6 against 9.2 and 6 rows (96) 9.9.  These
// leave a CU one workgroup, so they are for one row tile, which one round of
// workgroups covers: groups, a tile or more each, take several (512 rows in 64
// 4096 -> 2816 110 against 89).
inline int held_spans(int64_t rows, int n_groups, int n_in) {
    const int64_t m = typical_rows(rows, n_groups);
    if (n_groups > 1 && m > 8) return 0;
    if (m <= held_rows(n_in, HELD_SPANS)) return HELD_SPANS;
    return n_groups == 1 && m <= held_rows(n_in, MORE_HELD_SPANS) ? MORE_HELD_SPANS : 0;
}

template <typename OT, Rows ROWS, int HELD> hipError_t launch_small(const ProductParams& p, hipStream_t s) {
    const int64_t runs = (p.n_out + 15) / 16, tiles = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, HELD ? held_rows(p.n_in, HELD) : SMALL_MAX_ROWS);
    // As many waves a run as the card holds at once: one row 4096 -> 14336 takes 9.0
    // us at 4 waves a run and 11.2 at 8, 8192 -> 28672 25.6 at 2, 29.9 at 4 and 30.2
    // at 1, 14336 -> 4096 9.5 at 8 and 11.1 at 4; 64 rows in 64 groups 2048 -> 2816 19
    // at 1 and 63 at 8.
    const int split = small_split(p.n_out, tiles, p.n_in, HELD);
    const dim3 grid((unsigned)((runs * split + SMALL_WAVES - 1) / SMALL_WAVES), (unsigned)tiles);
    if (p.n_in % (4 * BLOCK) == 0) small_kernel<OT, ROWS, HELD, true><<<grid, SMALL_WAVES * 64, 0, s>>>(p, split);
    else small_kernel<OT, ROWS, HELD, false><<<grid, SMALL_WAVES * 64, 0, s>>>(p, split);
    return hipGetLastError();
}

template <typename OT, int T> hipError_t launch_medium(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, T), cols = (p.n_out + T - 1) / T;
    const unsigned tiles = (unsigned)xcd_padded(rows * cols);
    if (p.n_in % (4 * BLOCK) == 0) medium_kernel<OT, T, true><<<tiles, 256, 0, s>>>(p, (int)rows, (int)cols);
    else medium_kernel<OT, T, false><<<tiles, 256, 0, s>>>(p, (int)rows, (int)cols);
    return hipGetLastError();
}

template <typename OT, int RT, int CT> hipError_t launch_gemm(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 64 * RT), cols = (p.n_out + 64 * CT - 1) / (64 * CT);
    const unsigned tiles = (unsigned)xcd_padded(rows * cols);
    if (p.n_in % (4 * BLOCK) == 0) gemm_kernel<OT, RT, CT, true><<<tiles, 256, 0, s>>>(p, (int)rows, (int)cols);
    else gemm_kernel<OT, RT, CT, false><<<tiles, 256, 0, s>>>(p, (int)rows, (int)cols);
    return hipGetLastError();
}

// Row tiles of `high` rows that a product is expected to have: with groups, half a
// tile of each group (or row) is padding.
inline int64_t expected_tiles(const ProductParams& p, int high) {
    if (!p.offsets) return (p.rows + high - 1) / high;
    return p.rows / high + (p.n_groups < p.rows ? p.n_groups : p.rows) / 2 + 1;
}

// Rounds of 128 x 128 tiles, two workgroups a CU; at least one.
inline double rounds128(const ProductParams& p) {
    const double rounds = (double)(expected_tiles(p, 128) * ((p.n_out + 127) / 128)) / 512;
    return rounds > 1 ? rounds : 1;
}

template <typename OT> hipError_t launch_product(const ProductParams& p, hipStream_t s) {
    const int held = held_spans(p.rows, p.n_groups, p.n_in);
    if (p.x) return held == HELD_SPANS ? launch_small<OT, QUANTISED, HELD_SPANS>(p, s) : launch_small<OT, QUANTISED, MORE_HELD_SPANS>(p, s);
    if (held == HELD_SPANS) return launch_small<OT, STAGED, HELD_SPANS>(p, s);
    // Few rows: one row tile of 16, or two while each CU has at most one run of 16
    // outputs of a tile (us, with the quantisation): 16 rows 14336 -> 4096 13.2 in
    // small tiles and 23.8 in 64 x 64 ones, 4096 -> 14336 12.6 and 12.9; 24 rows
    // 14336 -> 4096 15.2 and 24.5, but 4096 -> 14336 17 and 13.2; 8 rows of each of
    // 64 groups 2048 -> 2816 50 and 61.
    const int64_t m = typical_rows(p.rows, p.n_groups);
    if (p.offsets ? m <= 8 : m <= 16 || (m <= 32 && p.n_out <= 16 * CUS)) return launch_small<OT, STREAMED, 0>(p, s);
    // 32 x 32 tiles in one round: 64 rows 14336 -> 4096 (256 of them) 15.0 us against
    // 25.4 in 64 x 64, 256 rows 4096 -> 1024 6.2 against 8.7; two rounds lose (128
    // rows 14336 -> 4096 26.1 against 24.4, 1024 -> 4096 7.3 against 5.1).
    if (expected_tiles(p, 32) * ((p.n_out + 31) / 32) <= CUS) return launch_medium<OT, 32>(p, s);
    // 64 x 64 tiles up to two rounds: 512 rows 4096 -> 4096 15.0 us against 18.5 in
    // 128 x 128, 1024 rows 28.1 against 18.4.
    if (expected_tiles(p, 64) * ((p.n_out + 63) / 64) <= 2 * CUS) return launch_medium<OT, 64>(p, s);
    // 128 x 128 tiles (two workgroups a CU) against 256 x 256 (one).  A round of the
    // former takes 0.7 of the latter's, and with many tiles a CU only whole rounds
    // of the large ones count, as the small ones end one by one.  2048 rows 4096 ->
    // 4096 27.8 against 43.1 us (1 : 1 rounds), 4096 rows 50.5 against 43.3 (2 : 1),
    // 2048 rows 8192 -> 28672 386 against 315 (7 : 4), 2048 rows in 64 groups 2048 ->
    // 2816 46.5 against 67.5 (2.1 : 2), 1024 rows in 8 groups 4096 -> 14336 100
    // against 85 (2.8 : 2).
    const double low = 0.72 * rounds128(p);
    const int64_t row_tiles = expected_tiles(p, 256), tiles = row_tiles * ((p.n_out + 255) / 256), high = (tiles + CUS - 1) / CUS;
    // Whole rounds of large tiles, and small ones for the columns left over: 2048
    // rows 8192 -> 28672 (3 + 0.72 rounds against 4) 261 us against 270, 8192 ->
    // 10240 (1.72 : 2) 101 against 112.
    const int64_t whole = tiles / CUS, cols = row_tiles > 0 ? whole * CUS / row_tiles * 256 : 0;
    if (!p.offsets && cols > 0 && cols < p.n_out) {
        ProductParams left = p, right = p;
        left.n_out = (int)cols;
        right.n_out = (int)(p.n_out - cols);
        right.wc += cols * (p.n_in / 2);
        right.ws += cols * (p.n_in / BLOCK);
        right.y = static_cast<char*>(p.y) + cols * OT::bytes;
        const double both = (double)whole + 0.72 * rounds128(right) + 0.05;
        if (both < low && both < (double)high) {
            const hipError_t e = launch_gemm<OT, 4, 4>(left, s);
            return e == hipSuccess ? launch_gemm<OT, 2, 2>(right, s) : e;
        }
    }
    return low < (double)high ? launch_gemm<OT, 2, 2>(p, s) : launch_gemm<OT, 4, 4>(p, s);
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

// `rows` rows of n values of dtype.
Span values(const void* at, int32_t dtype, int64_t rows, int64_t n, int64_t ld) {
    const int64_t size = dtype_bytes(dtype);
    return Span{at, n * size, rows, (rows > 1 ? ld : n) * size};
}

int64_t codes_bytes(int64_t rows, int32_t n) { return (rows * (n / 2) + 255) & ~int64_t(255); }

// More than one launch of quantise or dequantise takes: 2^24 - 1 workgroups (fewer than 2^32 threads).
bool too_many_units(int64_t rows, int32_t n) {
    return rows > ((int64_t)1 << 40) || rows * (n / 8) > (int64_t)0xFFFFFF * 256 * QUANT_UNROLL;
}

int product_checks(int32_t rows, const int32_t* offsets, int32_t n_groups, const uint8_t* codes, const uint8_t* scales,
                   int32_t n_in, int32_t n_out, const void* y, int32_t dtype) {
    if (bad_dtype(dtype) || bad_row(n_in) || n_out < 1 || rows < 0 || n_groups < 1) return EXL3_EINVAL;
    if (!offsets && n_groups != 1) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!codes || !scales || !y) return EXL3_EINVAL;
    if (misaligned(codes) || misaligned(scales) || misaligned(y) || (reinterpret_cast<uintptr_t>(offsets) & 3)) return EXL3_EINVAL;
    if (n_in > (1 << 20) || n_groups > 4096 || rows > (1 << 23) || n_out > (1 << 24)) return EXL3_EUNSUPPORTED;
    // a launch takes fewer than 2^32 threads: 2^24 workgroups of the smallest tile that many outputs come in
    if ((((int64_t)rows >> 6) + n_groups + 2) * (((int64_t)n_out >> 6) + 1) >= (1 << 24) - XCDS * XCD_UNIT) return EXL3_EUNSUPPORTED;
    return 1;  // proceed
}

}  // namespace mx
}  // namespace exl3

extern "C" {

using exl3::apart;
using namespace exl3::mx;

int exl3_mxfp4_quantize(const void* x, int32_t dtype, int64_t rows, int32_t n, int64_t ldx, uint8_t* codes,
                        uint8_t* scales, void* stream) {
    if (bad_dtype(dtype) || bad_row(n) || rows < 0 || bad_ld(ldx, n, dtype)) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!x || !codes || !scales || misaligned(x) || misaligned(codes) || misaligned(scales)) return EXL3_EINVAL;
    if (too_many_units(rows, n)) return EXL3_EUNSUPPORTED;
    if (!apart({{codes, rows * (n / 2)}, {scales, rows * (n / BLOCK)}}, {values(x, dtype, rows, n, ldx)})) return EXL3_EINVAL;
    return quantize(dtype, x, rows, n, ldx, codes, scales, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int32_t n, void* out,
                          int32_t dtype, void* stream) {
    if (bad_dtype(dtype) || bad_row(n) || rows < 0) return EXL3_EINVAL;
    if (rows == 0) return EXL3_OK;
    if (!out || !codes || !scales || misaligned(out) || misaligned(codes) || misaligned(scales)) return EXL3_EINVAL;
    if (too_many_units(rows, n)) return EXL3_EUNSUPPORTED;
    if (!apart({values(out, dtype, 1, rows * n, rows * n)}, {{codes, rows * (n / 2)}, {scales, rows * (n / BLOCK)}})) return EXL3_EINVAL;
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
    return held_spans(rows, n_groups, n_in) ? 0 : codes_bytes(rows, n_in) + (((int64_t)rows * (n_in / BLOCK) + 255) & ~int64_t(255));
}

int exl3_mxfp4_matmul(const uint8_t* x_codes, const uint8_t* x_scales, int32_t rows, const int32_t* offsets,
                      int32_t n_groups, const uint8_t* codes, const uint8_t* scales, int32_t n_in, int32_t n_out,
                      void* y, int32_t dtype, void* stream) {
    const int rc = product_checks(rows, offsets, n_groups, codes, scales, n_in, n_out, y, dtype);
    if (rc <= 0) return rc;
    if (!x_codes || !x_scales || misaligned(x_codes) || misaligned(x_scales)) return EXL3_EINVAL;
    const int64_t in = rows, w = (int64_t)n_groups * n_out, size = (int64_t)rows * n_out;
    if (!apart({values(y, dtype, 1, size, size)}, {{x_codes, in * (n_in / 2)}, {x_scales, in * (n_in / BLOCK)}, {codes, w * (n_in / 2)},
               {scales, w * (n_in / BLOCK)}, {offsets, 4 * ((int64_t)n_groups + 1)}}))
        return EXL3_EINVAL;
    const ProductParams p = {nullptr, 0, x_codes, x_scales, offsets, n_groups, rows, codes, scales, n_in, n_out, y, n_out};
    return product(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

int exl3_mxfp4_linear(const void* x, int32_t dtype, int32_t rows, int64_t ldx, const int32_t* offsets,
                      int32_t n_groups, const uint8_t* codes, const uint8_t* scales, int32_t n_in, int32_t n_out,
                      void* y, void* workspace, size_t workspace_bytes, void* stream) {
    const int rc = product_checks(rows, offsets, n_groups, codes, scales, n_in, n_out, y, dtype);
    if (rc < 0) return rc;
    if (bad_ld(ldx, n_in, dtype)) return EXL3_EINVAL;
    if (rc == 0) return rc;
    if (!x || misaligned(x) || misaligned(workspace)) return EXL3_EINVAL;
    const int64_t need = exl3_mxfp4_workspace_bytes(rows, n_groups, n_in);
    if (need > 0 && (!workspace || (int64_t)workspace_bytes < need)) return EXL3_EWORKSPACE;
    const int64_t w = (int64_t)n_groups * n_out, size = (int64_t)rows * n_out;
    if (!apart({values(y, dtype, 1, size, size), {workspace, need}}, {values(x, dtype, rows, n_in, ldx), {codes, w * (n_in / 2)},
               {scales, w * (n_in / BLOCK)}, {offsets, 4 * ((int64_t)n_groups + 1)}}))
        return EXL3_EINVAL;
    ProductParams p = {x, ldx, nullptr, nullptr, offsets, n_groups, rows, codes, scales, n_in, n_out, y, n_out};
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
