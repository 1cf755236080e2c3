// int8.hip - products of 8-bit rows with 8-bit weights (gfx950).
//
// y[r][o] = T(fl(fl(sum_k x[r][k] w[o][k]) xs[r]) ws[o]): the sum exact in 32-bit integers, converted to
// fp32 (the first rounding, from 2^24 on), each scale one more rounding of fp32, the type T the last.
// Five kernels for few rows to many; choose_product (int8_plan.hpp) chooses.
#include <hip/hip_runtime.h>

#include "int8_device.hpp"
#include "int8_internal.hpp"
#include "int8_plan.hpp"
#include "tile_device.hpp"

namespace exl3 {
namespace i8 {

struct ProductParams {
    const void* x;  // rows of values (quantised inside), or null
    int64_t ldx;
    const int8_t* xc;  // quantised rows
    const float* xs;
    const int* offsets;  // null: one group of all rows
    int n_groups, rows;
    const int8_t* wc;
    const float* ws;
    int n_in, n_out;
    void* y;
    int ldy;  // outputs from a row of y to the next: n_out, or more where this launch makes some of the columns
};

__device__ inline __amdgpu_buffer_rsrc_t buffer(const int8_t* base, int64_t bytes) {
    return mx::buffer(reinterpret_cast<const uint8_t*>(base), bytes);
}

// v_mfma_i32_16x16x64_i8 takes, per lane, 16 codes (a block) of row lane % 16, of the
// (lane / 16)th of the four blocks of 64 inputs; accumulator i is row 4 (lane / 16) + i of
// the first operand (an output) against row lane % 16 of the second.  With nothing else to do the
// card issues 4.80 P multiplications and additions a second of this one (eight waves a CU; 4.44 with
// four), 4.28 of 32 x 32 x 32 (3.77), which holds the clock lower: 8192^3 took 425 us with this one,
// 446 with that.
__device__ inline i32x4_t mfma(const i32x4_t w, const i32x4_t x, const i32x4_t c) { return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, x, c, 0, 0, 0); }

// Few rows: eight waves, `split` of them on each run of 16 outputs (8 / split runs a
// workgroup), for up to 16 rows; of a run's waves, wave w takes the spans (256 inputs) w,
// w + split, ...  Each wave brings its spans of the weight straight into a ring of its own
// in LDS, four rows of 256 bytes a load, and waits for nobody.  The rows come quantised, the same
// way (STREAMED), or, up to HELD blocks of them, the workgroup brings all of them into LDS
// first, while the weight is on its way: quantised ones (STAGED), or values that it quantises
// (QUANTISED).  A run's sums meet in LDS.
//
// Block b of row r sits in 16-byte slot b ^ r of the row's 256 bytes: the 16 lanes that LDS
// serves together (rows 0-3 and 12-15 of one quarter of the wave, 4-11 of the next) then read
// 16 different slots.
//
// Memory bounds it: 13 rows 14336 -> 4096 take 11.4 us (the weight at 5.1 TB/s, what a large copy
// moves), 3 x 2 tokens of 8 experts 4096 -> 14336 45.7 us.  One row 4096 -> 4096 takes 7.5 us, 2.2 TB/s: launch,
// the row's latency, its quantisation, the weight's latency.
enum Rows { STREAMED, STAGED, QUANTISED };

template <typename OT, Rows ROWS>
__global__ __launch_bounds__(SMALL_WAVES * 64) void small_kernel(const ProductParams p, int split) {
    constexpr bool HELD = ROWS != STREAMED;
    constexpr int SIDES = HELD ? 1 : 2, LOADS = SIDES * 4, BUF = SIDES * 256, RING = SMALL_WAVES * SMALL_RING * BUF;
    __shared__ i32x4_t lds[small_slots(HELD)];  // the rings, and the held rows
    static_assert(!HELD || small_per_cu(HELD) == 2, "two workgroups a CU");
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const RowTile t = find_tile(p.offsets, p.n_groups, p.rows, blockIdx.y, HELD ? held_rows(p.n_in) : SMALL_MAX_ROWS);
    if (t.rows == 0) return;
    const int first = wave % split;  // of the run's spans
    const int n0 = (blockIdx.x * (SMALL_WAVES / split) + wave / split) * 16, cols = min(16, p.n_out - n0);
    const int nb = p.n_in / BLOCK, spans = (nb + SPAN_BLOCKS - 1) / SPAN_BLOCKS;
    i32x4_t* const ring = lds + wave * SMALL_RING * BUF;

    i32x4_t acc = {0, 0, 0, 0};
    float xs = 0.f;
    f32x4_t ws = {0.f, 0.f, 0.f, 0.f};
    if (t.group < p.n_groups) {
        const int mine = cols > 0 ? (spans - first + split - 1) / split : 0;  // spans of this wave
        const int64_t w0 = (int64_t)t.group * p.n_out + (cols > 0 ? n0 : 0);
        const int w_rows = max(cols, 1);
        const __amdgpu_buffer_rsrc_t bw = buffer(p.wc + w0 * p.n_in, (int64_t)w_rows * p.n_in);
        const __amdgpu_buffer_rsrc_t bx = buffer(HELD ? p.wc : p.xc + (int64_t)t.row0 * p.n_in, HELD ? 0 : (int64_t)t.rows * p.n_in);
        uint32_t w_at[4], x_at[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // load i: row 4 i + lane / 16, slot lane % 16; rows behind the tile re-read its last
            const int row = 4 * i + (lane >> 4), block = (lane & 15) ^ row;
            w_at[i] = (uint32_t)min(row, w_rows - 1) * p.n_in + 16 * block;
            x_at[i] = (uint32_t)min(row, t.rows - 1) * p.n_in + 16 * block;
        }
        // The loads of this wave's kth span; behind its last, and behind the end of a row, they give zeros.
        auto ask = [&](int k) {
            const int sp = k < mine ? first + k * split : spans;
            i32x4_t* const buf = ring + k % SMALL_RING * BUF;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int block = (lane & 15) ^ (4 * i + (lane >> 4));
                const bool in = sp * SPAN_BLOCKS + block < nb;
                load16_to_lds(bw, buf + i * 64, in ? w_at[i] : OUTSIDE, (uint32_t)sp * 256);
                if constexpr (!HELD) load16_to_lds(bx, buf + 256 + i * 64, in ? x_at[i] : OUTSIDE, (uint32_t)sp * 256);
            }
        };
        i32x4_t* const xq = lds + RING;  // [row][spans * 16], block b of row r at b ^ r
        uint32_t* const amax = reinterpret_cast<uint32_t*>(xq);  // before the codes: each row's largest magnitude
        if constexpr (ROWS == QUANTISED) {
            if (threadIdx.x < SMALL_MAX_ROWS) amax[threadIdx.x] = 0;
        }
        if (first == 0) {
#pragma unroll
            for (int i = 0; i < 4; ++i) ws[i] = p.ws[w0 + min(4 * q + i, w_rows - 1)];
        }
        if constexpr (ROWS != QUANTISED) xs = p.xs[t.row0 + min(r, t.rows - 1)];
        // The rows are asked for before the weight, as loads come back in order.
        auto ask_ring = [&]() {
#pragma unroll
            for (int k = 0; k < SMALL_RING; ++k) ask(k);
        };
        if constexpr (ROWS == STREAMED) ask_ring();
        if constexpr (ROWS == STAGED) {
            // HELD_BLOCKS / 512 blocks a thread (blocks behind a row's end are anything: the weight's are zeros)
            constexpr int ROUNDS = HELD_BLOCKS / (SMALL_WAVES * 64);
            const int units = t.rows * nb;
            i32x4_t v[ROUNDS];
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int u = threadIdx.x + i * SMALL_WAVES * 64;
                if (u < units) v[i] = *reinterpret_cast<const i32x4_t*>(p.xc + ((int64_t)t.row0 * nb + u) * BLOCK);
            }
            ask_ring();
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int u = threadIdx.x + i * SMALL_WAVES * 64, row = u / nb, block = u - row * nb;
                if (u < units) xq[row * spans * 16 + (block ^ row)] = v[i];
            }
            __syncthreads();
        }
        if constexpr (ROWS == QUANTISED) {
            // all rows' values in registers: their largest magnitudes meet in LDS, then the codes go there
            constexpr int THREADS = SMALL_WAVES * 64, N = 16 / OT::bytes, ROUNDS = HELD_BLOCKS * BLOCK / N / THREADS;
            const int per_row = p.n_in / N, units = t.rows * per_row;
            float u[ROUNDS][N];
            u32x4_t v[ROUNDS];
            int row[ROUNDS];
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int at = threadIdx.x + i * THREADS;
                row[i] = at / per_row;
                v[i] = u32x4_t{0, 0, 0, 0};
                if (at < units) v[i] = load_piece<OT, true>(p.x, (int64_t)(t.row0 + row[i]) * p.ldx + (at - row[i] * per_row) * N, N);
            }
            ask_ring();
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i)
#pragma unroll
                for (int e = 0; e < N; ++e) u[i][e] = piece_value<OT>(v[i], e);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const uint32_t mine = amax_piece<N>(0, u[i]);
                const int one = __builtin_amdgcn_readfirstlane(row[i]);
                if (i * THREADS >= units) break;
                if (__all(row[i] == one)) {
                    const uint32_t most = over_lanes<64>(mine, larger);
                    if (lane == 0 && one < t.rows) atomicMax(&amax[one], most);
                } else if (row[i] < t.rows) {
                    atomicMax(&amax[row[i]], mine);
                }
            }
            __syncthreads();
            uint32_t most[ROUNDS];
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) most[i] = amax[min(row[i], t.rows - 1)];
            xs = row_scale(amax[min(r, t.rows - 1)], 1.0);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < ROUNDS; ++i) {
                const int at = threadIdx.x + i * THREADS;
                if (at >= units) break;
                const uint32_t a = most[i];
                const float largest = __builtin_bit_cast(float, a);
                uint32_t c[N / 4] = {};
                if (a < NOT_FINITE) code_piece<N>(u[i], largest, 127.f / largest, c);
                const int col = (at - row[i] * per_row) * N, block = col / BLOCK;
                uint32_t* const dst = reinterpret_cast<uint32_t*>(xq + row[i] * spans * 16 + (block ^ row[i])) + col % BLOCK / 4;
                if constexpr (N == 8) *reinterpret_cast<uint2*>(dst) = uint2{c[0], c[1]};
                else *dst = c[0];
            }
            __syncthreads();
        }
        for (int k = 0; k < mine; ++k) {
            __builtin_amdgcn_sched_barrier(0);
            wait_loads<(SMALL_RING - 1) * LOADS, false>();
            __builtin_amdgcn_sched_barrier(0);
            const int sp = first + k * split;
            const i32x4_t* const buf = ring + k % SMALL_RING * BUF;
            i32x4_t wv[4], xv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                wv[j] = buf[r * 16 + ((4 * j + q) ^ r)];
                const int row = HELD ? min(r, t.rows - 1) : r;  // rows behind the tile re-read its last
                xv[j] = HELD ? xq[(row * spans + sp) * 16 + ((4 * j + q) ^ row)] : buf[256 + r * 16 + ((4 * j + q) ^ r)];
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read
            __builtin_amdgcn_sched_barrier(0);
            ask(k + SMALL_RING);
#pragma unroll
            for (int j = 0; j < 4; ++j) acc = mfma(wv[j], xv[j], acc);
        }
        wait_loads<0, false>();  // nothing is on its way into LDS any more
    }
    // each wave's sums over its own ring
    ring[lane] = acc;
    __syncthreads();
    if (first == 0) {
        for (int w = 1; w < split; ++w) acc += ring[w * SMALL_RING * BUF + lane];
        const int o = n0 + 4 * q;
        if (r < t.rows && o < p.n_out) {
            f32x4_t v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = rounded((float)acc[i] * xs * ws[i]);
            store4<OT>(p.y, (int64_t)(t.row0 + r) * p.ldy + o, p.n_out - o, (p.ldy & 3) == 0, v);
        }
    }
}

// v, computed where this stands: what follows from it takes no registers over a loop before.
__device__ inline int here(int v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A wave's results: RT times 16 rows, STEP from one 16 to the next, the first at `row0`, and 16 CT
// outputs from `col0`, of which those less than `rows` behind row0 are written.  The sums take
// both scales: xs of this lane's rows, ws of output lane % (16 CT).  A lane holds 4 consecutive
// outputs of a row; for 16-bit results lanes 16 apart exchange halves of two tiles, so that
// each has 8.  A store then writes 64 bytes of each of 16 rows (32 where CT is 1).
template <typename OT, int STEP, int RT, int CT>
__device__ inline void store_tile(const i32x4_t (&acc)[RT][CT], const float (&xs)[RT], float ws, const ProductParams& p, int row0, int rows, int col0) {
    typedef typename OT::raw raw;
    const int lane = here(threadIdx.x & 63), r = lane & 15, q = lane >> 4;
    raw* y = static_cast<raw*>(p.y);
    auto store = [&](int row, int o, auto v) {  // 16 bytes (or 8), or what is left of the row
        constexpr int N = sizeof(v) / OT::bytes;
        raw* const dst = y + (int64_t)(row0 + row) * p.ldy + o;
        if (row >= rows) return;
        if (o + N <= p.n_out) {
            __builtin_memcpy(dst, &v, sizeof(v));  // rows start at any value: an unaligned store
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (o + i < p.n_out) dst[i] = (raw)(OT::bytes == 2 ? v[i / 2] >> (16 * (i & 1)) : v[i]);
        }
    };
    float w[CT][4];
#pragma unroll
    for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) w[c][i] = __shfl(ws, 16 * c + 4 * q + i);
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        auto value = [&](int c, int i) { return rounded((float)acc[m][c][i] * xs[m] * w[c][i]); };
        if constexpr (OT::bytes == 4) {
#pragma unroll
            for (int c = 0; c < CT; ++c) {
                u32x4_t v;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = from_f32(OT{}, value(c, i));
                store(m * STEP + r, col0 + 16 * c + 4 * q, v);
            }
        } else if constexpr (CT == 1) {
            typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
            u32x2_t v;
#pragma unroll
            for (int i = 0; i < 2; ++i) v[i] = (uint32_t)from_f32(OT{}, value(0, 2 * i)) | ((uint32_t)from_f32(OT{}, value(0, 2 * i + 1)) << 16);
            store(m * STEP + r, col0 + 4 * q, v);
        } else {
            static_assert(CT % 2 == 0, "sets of outputs exchange in pairs");
#pragma unroll
            for (int c = 0; c < CT; c += 2) {
                u32x4_t v;
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const uint32_t lo = (uint32_t)from_f32(OT{}, value(c, 2 * i)) | ((uint32_t)from_f32(OT{}, value(c, 2 * i + 1)) << 16);
                    const uint32_t hi = (uint32_t)from_f32(OT{}, value(c + 1, 2 * i)) | ((uint32_t)from_f32(OT{}, value(c + 1, 2 * i + 1)) << 16);
                    // odd rows of 16 lanes of the one for even rows of the other
                    const auto both = __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
                    v[i] = both[0];
                    v[2 + i] = both[1];
                }
                store(m * STEP + r, col0 + 16 * (c + (q & 1)) + 8 * (q >> 1), v);
            }
        }
    }
}

constexpr int STAGE_BLOCKS = 8;  // of a row, in what follows: 128 inputs

// Some rows, or few tiles: a workgroup owns TM rows and TN outputs, each of its waves every WAVESth
// stage (128 inputs), in a ring of its own in LDS as above: they wait for nobody, so that one wave's loads, another's
// reads and a third's matrix instructions overlap.  The waves' sums meet in LDS.  Block b of row r sits in slot
// b ^ (r / 2 & 7) of the row's 128 bytes.
//
// The weight's way to a CU bounds it, 23 to 25 bytes a ns where it comes from memory, and behind that the rows', which
// each workgroup reads again: 32 rows 14336 -> 4096 take 16.7 us (the weight at 3.5 TB/s), 64 rows 4096 -> 4096 6.7.
// Waves on their own against four that share a stage and meet at a barrier, in 32 x 32 tiles: the same where the weight
// comes from memory, 15.1 us against 17.5 for 64 rows 14336 -> 4096 from the caches.
// Rings of 2, 3 and 4 stages, us: 32 x 32 tiles, one a CU, 64 rows 4096 -> 4096 6.7, 7.1 and 7.3, 14336 -> 4096 20.5, 21.1 and 21.4
// (the longer start costs more than what is further ahead brings), and where there are more tiles, two of which a ring of 2 lets a
// CU hold, 64 rows 4096 -> 6144 9.5, 12.5 and 12.9.  32 x 64 tiles, one a CU: 2 and 3 8.5 and 9.0 at that size, 128 rows 14336 -> 4096 26.9 and
// 27.1.  32 x 16 tiles: 2, 3 and 4 17 rows 14336 -> 4096 16.7, 14.2 and 14.4, 24 rows 4096 -> 4096 6.1, 6.2 and 6.5: 3.
template <typename OT, int TM, int TN, int RING>
__global__ __launch_bounds__(256) void strip_kernel(const ProductParams p, int row_tiles, int col_tiles) {
    constexpr int WAVES = 4, PER = STAGE_BLOCKS, RT = TM / 16, CT = TN / 16, BUF = (TM + TN) * PER, EACH = 64 / PER, LOADS = (TM + TN) / EACH;  // rows of a load, loads of a stage
    auto swizzle = [](int row) { return row >> 1 & 7; };
    __shared__ i32x4_t lds[WAVES * RING * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), r = lane & 15, q = lane >> 4;
    const ProductTile t = product_tile(p.offsets, p.n_groups, p.rows, xcd_tile(blockIdx.x), TM, row_tiles, col_tiles);
    if (t.rows == 0) return;
    const int n0 = t.col * TN, cols = min(TN, p.n_out - n0);
    const int nb = p.n_in / BLOCK, stages = (nb + PER - 1) / PER;
    i32x4_t* const ring = lds + wave * RING * BUF;
    // the wave's rows at the end: sets of 16, FINAL waves take turns
    constexpr int FINAL = RT < WAVES ? RT : WAVES, SETS = RT / FINAL;

    i32x4_t acc[RT][CT];
    float xs[SETS], ws = 0.f;
#pragma unroll
    for (int m = 0; m < SETS; ++m) xs[m] = 0.f;
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[m][c] = i32x4_t{0, 0, 0, 0};
    if (t.group < p.n_groups) {
        const int mine = (stages - wave + WAVES - 1) / WAVES;
        const int64_t w0 = (int64_t)t.group * p.n_out + n0;
        const __amdgpu_buffer_rsrc_t bx = buffer(p.xc + (int64_t)t.row0 * p.n_in, (int64_t)t.rows * p.n_in);
        const __amdgpu_buffer_rsrc_t bw = buffer(p.wc + w0 * p.n_in, (int64_t)cols * p.n_in);
        // Rows of both sides together, the weight's from TM on.  Load i: rows EACH i and on, slot lane % PER;
        // rows behind a side's end re-read its last.
        uint32_t at[LOADS];
        int block[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = EACH * i + lane / PER;
            block[i] = (lane % PER) ^ swizzle(row);
            at[i] = (uint32_t)(EACH * i < TM ? min(row, t.rows - 1) : min(row - TM, cols - 1)) * p.n_in + 16 * block[i];
        }
        auto ask = [&](int k) {  // behind the last stage: zeros
            const int st = k < mine ? wave + k * WAVES : stages;
            i32x4_t* const buf = ring + k % RING * BUF;
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                load16_to_lds(EACH * i < TM ? bx : bw, buf + i * 64, st * PER + block[i] < nb ? at[i] : OUTSIDE, (uint32_t)st * PER * 16);
        };
#pragma unroll
        for (int k = 0; k < RING; ++k) ask(k);
#pragma unroll
        for (int m = 0; m < SETS; ++m) xs[m] = p.xs[t.row0 + min(16 * (m * FINAL + wave % FINAL) + r, t.rows - 1)];
        ws = p.ws[w0 + min(lane % TN, cols - 1)];
        for (int k = 0; k < mine; ++k) {
            __builtin_amdgcn_sched_barrier(0);
            wait_loads<(RING - 1) * LOADS, false>();
            __builtin_amdgcn_sched_barrier(0);
            const i32x4_t* const buf = ring + k % RING * BUF;
            i32x4_t xv[PER / 4][RT], wv[PER / 4][CT];
#pragma unroll
            for (int j = 0; j < PER / 4; ++j) {
                const int slot = r * PER + ((4 * j + q) ^ swizzle(r));
#pragma unroll
                for (int m = 0; m < RT; ++m) xv[j][m] = buf[m * 16 * PER + slot];
#pragma unroll
                for (int c = 0; c < CT; ++c) wv[j][c] = buf[(TM + c * 16) * PER + slot];
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0): the buffer is read
            __builtin_amdgcn_sched_barrier(0);
            ask(k + RING);
#pragma unroll
            for (int j = 0; j < PER / 4; ++j)
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[m][c] = mfma(wv[j][c], xv[j][m], acc[m][c]);
        }
        wait_loads<0, false>();  // nothing is on its way into LDS any more
    }
    // each wave's sums over its own ring; then each adds up those of its rows
    static_assert(RT * CT * 64 <= RING * BUF, "the sums fit");
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) ring[(m * CT + c) * 64 + lane] = acc[m][c];
    __syncthreads();
    if (wave >= FINAL) return;
    i32x4_t sum[SETS][CT];
#pragma unroll
    for (int m = 0; m < SETS; ++m)
#pragma unroll
        for (int c = 0; c < CT; ++c) {
            sum[m][c] = i32x4_t{0, 0, 0, 0};
#pragma unroll
            for (int v = 0; v < WAVES; ++v) sum[m][c] += lds[v * RING * BUF + ((m * FINAL + wave) * CT + c) * 64 + lane];
        }
    store_tile<OT, 16 * FINAL, SETS, CT>(sum, xs, ws, p, t.row0 + 16 * wave, t.rows - 16 * wave, n0);
}

// More rows, or outputs: a workgroup of four waves owns 64 rows and 64 outputs, each wave a quarter of
// the tile.  Stages go straight into a ring in LDS, all but one of it ahead.  PER is a stage's blocks a row: 16, block
// b of row r in slot b ^ (r & 15) of the row's 256 bytes, or 8 (slots as in middle_kernel), with which two workgroups
// share a CU and fill each other's waits.
//
// A stage's own way bounds it: a barrier, the loads' issue, the reads, the matrix instructions one after the other (256 rows
// 4096 -> 4096 12.2 us; 512 rows 16.9, 1.0 P operations a second).
template <typename OT, int PER, int RING>
__global__ __launch_bounds__(256) void medium_kernel(const ProductParams p, int row_tiles, int col_tiles) {
    constexpr int T = 64, BUF = 2 * T * PER, LOADS = BUF / 256, EACH = 64 / PER;  // slots: rows, then weight rows; loads of a wave and stage; rows of a load
    auto swizzle = [](int row) { return PER == 16 ? row & 15 : row >> 1 & 7; };
    __shared__ i32x4_t lds[RING * BUF];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4, wy = wave >> 1, wx = wave & 1;
    const ProductTile t = product_tile(p.offsets, p.n_groups, p.rows, xcd_tile(blockIdx.x), T, row_tiles, col_tiles);
    if (t.rows == 0) return;
    const int n0 = t.col * T, cols = min(T, p.n_out - n0);
    const int nb = p.n_in / BLOCK, stages = (nb + PER - 1) / PER;

    i32x4_t acc[2][2];
    float xs[2] = {0.f, 0.f}, ws = 0.f;
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < 2; ++c) acc[m][c] = i32x4_t{0, 0, 0, 0};
    if (t.group < p.n_groups) {
        const int64_t w0 = (int64_t)t.group * p.n_out + n0;
        const __amdgpu_buffer_rsrc_t bx = buffer(p.xc + (int64_t)t.row0 * p.n_in, (int64_t)t.rows * p.n_in);
        const __amdgpu_buffer_rsrc_t bw = buffer(p.wc + w0 * p.n_in, (int64_t)cols * p.n_in);
#pragma unroll
        for (int m = 0; m < 2; ++m) xs[m] = p.xs[t.row0 + min(wy * 32 + 16 * m + r, t.rows - 1)];
        ws = p.ws[w0 + min(wx * 32 + (lane & 31), cols - 1)];
        // Rows of both sides together, the weight's from T on.  Load i of a wave: rows
        // 4 EACH i + EACH wave and on, slot lane % PER; rows behind a side's end re-read its last.
        const int srow = EACH * wave + lane / PER, block = (lane % PER) ^ swizzle(srow);
        uint32_t at[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
            const int row = 4 * EACH * i + srow;
            at[i] = (uint32_t)(4 * EACH * i < T ? min(row, t.rows - 1) : min(row - T, cols - 1)) * p.n_in + 16 * block;
        }
        auto ask = [&](int st) {  // behind the last stage: zeros
            i32x4_t* const buf = lds + st % RING * BUF;
#pragma unroll
            for (int i = 0; i < LOADS; ++i)
                load16_to_lds(4 * EACH * i < T ? bx : bw, buf + i * 256 + wave * 64, st * PER + block < nb ? at[i] : OUTSIDE, (uint32_t)st * PER * 16);
        };
#pragma unroll
        for (int k = 0; k < RING - 1; ++k) ask(k);
        for (int st = 0; st < stages; ++st) {
            // this stage has landed in every wave, and the one before it is read
            __builtin_amdgcn_sched_barrier(0);
            wait_loads<(RING - 2) * LOADS, true>();
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            ask(st + RING - 1);
            const i32x4_t* const buf = lds + st % RING * BUF;
#pragma unroll
            for (int j = 0; j < PER / 4; ++j) {
                const int slot = r * PER + ((4 * j + q) ^ swizzle(r));
                i32x4_t xv[2], wv[2];
#pragma unroll
                for (int m = 0; m < 2; ++m) xv[m] = buf[(wy * 2 + m) * 16 * PER + slot];
#pragma unroll
                for (int c = 0; c < 2; ++c) wv[c] = buf[(T + (wx * 2 + c) * 16) * PER + slot];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                    for (int c = 0; c < 2; ++c) acc[m][c] = mfma(wv[c], xv[m], acc[m][c]);
            }
        }
        wait_loads<0, true>();  // nothing is on its way into LDS any more
    }
    store_tile<OT, 16, 2, 2>(acc, xs, ws, p, t.row0 + wy * 32, t.rows - wy * 32, n0 + wx * 32);
}

// More rows: a workgroup of four waves owns 128 rows and 128 outputs, each wave a quarter of
// them; two workgroups a CU.  A stage is 128 inputs, a unit of 16 KB of each side, that go
// straight from memory into LDS.  LDS holds five units in a ring, weight, rows, weight, rows,
// weight: the rows are asked for one stage ahead, the weight (which more often comes from
// memory) two.  Block b of row r sits in 16-byte slot b ^ (r / 2 & 7) of the row's 128 bytes:
// the 16 lanes that LDS serves together then read 16 different slots of its 256-byte width.
// The loads' way bounds it: 768 rows 4096 -> 4096 take 26.4 us, 1.0 P operations a second.
// Units of the ring of this stage's rows, the next stage's rows and the weight of the one after
// that, from that of this stage's weight; and that of the next stage's weight.
__device__ inline int rows_unit(int u) { return u == 4 ? 0 : u + 1; }
__device__ inline int next_rows_unit(int u) { return u >= 2 ? u - 2 : u + 3; }
__device__ inline int after_next_weight_unit(int u) { return u >= 1 ? u - 1 : u + 4; }
__device__ inline int next_weight_unit(int u) { return u >= 3 ? u - 3 : u + 2; }

template <typename OT>
__global__ __launch_bounds__(256, 2) void middle_kernel(const ProductParams p, int row_tiles, int col_tiles) {
    constexpr int RT = 4, CT = 4, BM = 128, BN = 128, UNIT = 128 * STAGE_BLOCKS;
    __shared__ i32x4_t lds[5 * UNIT];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4, wy = wave >> 1, wx = wave & 1;
    const ProductTile t = product_tile(p.offsets, p.n_groups, p.rows, xcd_tile(blockIdx.x), BM, row_tiles, col_tiles);
    if (t.rows == 0) return;
    const int n0 = t.col * BN, cols = min(BN, p.n_out - n0);
    const int nb = p.n_in / BLOCK, stages = (nb + STAGE_BLOCKS - 1) / STAGE_BLOCKS;

    i32x4_t acc[RT][CT];
    float xs[RT], ws = 0.f;
#pragma unroll
    for (int m = 0; m < RT; ++m) {
        xs[m] = 0.f;
#pragma unroll
        for (int c = 0; c < CT; ++c) acc[m][c] = i32x4_t{0, 0, 0, 0};
    }
    if (t.group < p.n_groups) {
        const int64_t w0 = (int64_t)t.group * p.n_out + n0;
        const __amdgpu_buffer_rsrc_t bx = buffer(p.xc + (int64_t)t.row0 * p.n_in, (int64_t)t.rows * p.n_in);
        const __amdgpu_buffer_rsrc_t bw = buffer(p.wc + w0 * p.n_in, (int64_t)cols * p.n_in);
#pragma unroll
        for (int m = 0; m < RT; ++m) xs[m] = p.xs[t.row0 + min((wy * RT + m) * 16 + r, t.rows - 1)];
        ws = p.ws[w0 + min(wx * 64 + lane, cols - 1)];
        // Rows behind the tile re-read its last (never stored).  Load i of a wave brings
        // rows 32 i + 8 wave .. + 7 of a unit, lane l slot l % 8 of row l / 8.
        const int srow = 8 * wave + (lane >> 3), sblock = (lane & 7) ^ ((srow >> 1) & 7);
        uint32_t xat[4], wat[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            xat[i] = (uint32_t)min(32 * i + srow, t.rows - 1) * p.n_in + 16 * sblock;
            wat[i] = (uint32_t)min(32 * i + srow, cols - 1) * p.n_in + 16 * sblock;
        }
        // The loads of a side of stage st into unit `to` of the ring; behind the end of a row: zeros.
        auto ask = [&](__amdgpu_buffer_rsrc_t b, const uint32_t (&at)[4], int st, int to) {
            const bool in = st * STAGE_BLOCKS + sblock < nb;
            i32x4_t* dst = lds + to * UNIT + wave * 64;
#pragma unroll
            for (int i = 0; i < 4; ++i) load16_to_lds(b, dst + i * 256, in ? at[i] : OUTSIDE, (uint32_t)st * 128);
        };
        ask(bw, wat, 0, 0);
        ask(bx, xat, 0, 1);
        ask(bw, wat, 1, 2);
        int uw = 0;  // the ring's unit of this stage's weight
        for (int st = 0; st < stages; ++st) {
            __builtin_amdgcn_sched_barrier(0);
            wait_loads<4, true>();  // all but the next stage's weight: this stage has landed, the one before it is read
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
            ask(bx, xat, st + 1, next_rows_unit(uw));
            ask(bw, wat, st + 2, after_next_weight_unit(uw));
            const i32x4_t* const xbuf = lds + rows_unit(uw) * UNIT + wy * RT * 128;
            const i32x4_t* const wbuf = lds + uw * UNIT + wx * CT * 128;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int slot = r * 8 + ((4 * j + q) ^ ((r >> 1) & 7));
                i32x4_t xv[RT], wv[CT];
#pragma unroll
                for (int m = 0; m < RT; ++m) xv[m] = xbuf[m * 128 + slot];
#pragma unroll
                for (int c = 0; c < CT; ++c) wv[c] = wbuf[c * 128 + slot];
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[m][c] = mfma(wv[c], xv[m], acc[m][c]);
            }
            uw = next_weight_unit(uw);
        }
        wait_loads<0, true>();  // nothing is on its way into LDS any more
    }
    store_tile<OT, 16, RT, CT>(acc, xs, ws, p, t.row0 + wy * RT * 16, t.rows - wy * RT * 16, n0 + wx * CT * 16);
}

// Many rows: a workgroup of eight waves takes tiles of 256 rows and 256 outputs, one after the
// other; one workgroup a CU.  The waves form two groups, one of each on a SIMD, that take turns:
// while one group reads its operands from LDS and asks for memory, the other has the matrix
// cores; a barrier ends each turn.  A wave has every other 16 of the rows, by its group, and 64 of
// the outputs: where a tile has fewer rows both groups have less to do.
//
// A stage is 128 inputs.  With 256 rows it is a unit of 32 KB of each side, and LDS holds five of
// them in a ring as above; with 128 rows LDS holds three whole stages of 48 KB, and both sides
// are asked for two ahead.  The ring does not run dry between tiles: the last stages of a tile ask
// for the first of the next, and its results leave from registers.
//
// What bounds it: the power that the matrix cores draw at these values (2048 rows 8192 -> 28672: they
// are busy 0.79 of the cycles, at 1.67 GHz; all zeros run at 2.18 GHz and take 30 % less time), and the
// results, which all workgroups store at once between tiles (8192^3: 384 us, without them 354).
// 8192^3 takes 384 to 391 us by itself, 2.8 P operations a second, and 490 in a long run of them; 2048 rows
// 8192 -> 28672 359 to 372, and 16384 rows in 64 groups 2048 -> 2816 144 to 150 with 128 rows a tile.
// Two groups that take turns against all eight waves alike: a stage's reads then wait behind each other.
// One side's loads in each half of a stage, against all in the first: 8192^3 384 us, 415.
template <typename OT, int RT>
__global__ __launch_bounds__(512, 2) void large_kernel(const ProductParams p, int row_tiles, int col_tiles, int tiles) {
    constexpr int CT = 4, ROWS = 32 * RT, UNIT = 256 * STAGE_BLOCKS, STAGE = (ROWS + LARGE_COLS) * STAGE_BLOCKS;
    constexpr bool UNITS = RT == 8;  // a ring of units, not of stages
    constexpr int AHEAD = UNITS ? 4 : 4 + RT / 2;  // loads of a wave in flight over the end of a stage
    __shared__ i32x4_t lds[UNITS ? 5 * UNIT : 3 * STAGE];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r = lane & 15, q = lane >> 4, wy = wave >> 2, wx = wave & 3;
    const int nb = p.n_in / BLOCK, stages = max(2, (nb + STAGE_BLOCKS - 1) / STAGE_BLOCKS);

    struct Tile {
        int row0, rows, n0, cols;
        int64_t w0;
    };
    // The next tile from `index` on, or one without rows behind the last; tiles of rows of no
    // group are filled with zeros on the way.
    int index = blockIdx.x;
    // (with 256 rows there are no registers left for them)
    KeptGroups groups;
    if constexpr (!UNITS) groups = keep_groups(p.offsets, p.n_groups, p.rows);
    auto next_tile = [&]() {
        for (; index < tiles; index += gridDim.x) {
            const ProductTile t = product_tile(p.offsets, p.n_groups, p.rows, xcd_tile(index), ROWS, row_tiles, col_tiles, UNITS ? nullptr : &groups);
            if (t.rows == 0) break;  // the tiles of a workgroup rise: there are no more
            const int n0 = t.col * LARGE_COLS, cols = min(LARGE_COLS, p.n_out - n0);
            if (t.group >= p.n_groups) {
                typedef typename OT::raw raw;
                for (int i = threadIdx.x; i < t.rows * LARGE_COLS; i += 512)
                    if (i % LARGE_COLS < cols) static_cast<raw*>(p.y)[(int64_t)(t.row0 + i / LARGE_COLS) * p.ldy + n0 + i % LARGE_COLS] = 0;
                continue;
            }
            index += gridDim.x;
            return Tile{t.row0, t.rows, n0, cols, (int64_t)t.group * p.n_out + n0};
        }
        return Tile{0, 0, 0, 0, 0};
    };
    // Rows and outputs behind a tile's end are outside its memory: zeros.
    auto rows_of = [&](const Tile& t) { return buffer(p.xc + (int64_t)t.row0 * p.n_in, (int64_t)t.rows * p.n_in); };
    auto weight_of = [&](const Tile& t) { return buffer(p.wc + t.w0 * p.n_in, (int64_t)t.cols * p.n_in); };

    // Load i of a wave brings rows 64 i + 8 wave .. + 7 of a unit, lane l slot l % 8 of row l / 8.
    const int srow = 8 * wave + (lane >> 3), sblock = (lane & 7) ^ ((srow >> 1) & 7);
    uint32_t at[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) at[i] = (uint32_t)(64 * i + srow) * p.n_in + 16 * sblock;
    // The loads of `loads` times 64 rows of a side of stage st to `dst`; behind the end of a row: zeros.
    auto ask = [&](__amdgpu_buffer_rsrc_t b, int loads, int st, i32x4_t* dst) {
        const bool in = st * STAGE_BLOCKS + sblock < nb;
#pragma unroll
        for (int i = 0; i < loads; ++i) load16_to_lds(b, dst + wave * 64 + i * 512, in ? at[i] : OUTSIDE, (uint32_t)st * 128);
    };
    // Where the ring has this stage's weight and rows: u is a unit, or the number of a stage.
    auto weight_at = [&](int u) { return lds + u * (UNITS ? UNIT : STAGE); };
    auto rows_at = [&](int u) { return UNITS ? lds + rows_unit(u) * UNIT : lds + u * STAGE + LARGE_COLS * STAGE_BLOCKS; };
    int frag[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) frag[j] = r * 8 + ((4 * j + q) ^ ((r >> 1) & 7));

    Tile t = {0, 0, 0, 0, 0};
    __amdgpu_buffer_rsrc_t bx, bw;
    int u = 0;  // where the ring has this stage
    bool started = false;
    for (;;) {
        const Tile after = next_tile();
        const __amdgpu_buffer_rsrc_t ax = rows_of(after), aw = weight_of(after);
        if (!started) {
            if (after.rows == 0) return;
            started = true;
            t = after;
            bx = ax;
            bw = aw;
            ask(bw, 4, 0, weight_at(0));
            ask(bx, RT / 2, 0, rows_at(0));
            ask(bw, 4, 1, weight_at(UNITS ? 2 : 1));
            if (!UNITS) ask(bx, RT / 2, 1, rows_at(1));
            __builtin_amdgcn_sched_barrier(0);
            wait_loads<AHEAD, false>();  // the first stage has landed
            __builtin_amdgcn_s_barrier();
            if (wy == 1) __builtin_amdgcn_s_barrier();  // the second group is a turn behind
            __builtin_amdgcn_sched_barrier(0);
            continue;
        }
        i32x4_t acc[RT][CT];
        float xs[RT];
        const int own = here(lane);
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            xs[m] = p.xs[t.row0 + min(32 * m + 16 * wy + (own & 15), t.rows - 1)];
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[m][c] = i32x4_t{0, 0, 0, 0};
        }
        const float ws = p.ws[t.w0 + min(wx * 64 + own, t.cols - 1)];
        for (int st = 0; st < stages; ++st) {
            const i32x4_t* const xbuf = rows_at(u) + wy * 128;
            const i32x4_t* const wbuf = weight_at(u) + wx * CT * 128;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                i32x4_t xv[RT], wv[CT];
#pragma unroll
                for (int c = 0; c < CT; ++c) wv[c] = wbuf[c * 128 + frag[j]];
#pragma unroll
                for (int m = 0; m < RT; ++m) xv[m] = xbuf[m * 256 + frag[j]];
                // Into what held the stage before, which every wave has read; one side in each half of
                // the stage, as the address unit takes 16 cycles a load.
                const int next = st + (UNITS && j == 0 ? 1 : 2);
                const bool in = next < stages;
                const int of = in ? next : next - stages;
                if constexpr (UNITS) {
                    if (j == 0) ask(in ? bx : ax, 4, of, lds + next_rows_unit(u) * UNIT);
                    else ask(in ? bw : aw, 4, of, lds + after_next_weight_unit(u) * UNIT);
                } else {
                    const int to = u == 0 ? 2 : u - 1;
                    if (j == 0) ask(in ? bw : aw, 4, of, weight_at(to));
                    else ask(in ? bx : ax, RT / 2, of, rows_at(to));
                }
                __builtin_amdgcn_sched_barrier(0);
                if (j == 1) wait_loads<AHEAD, true>();  // the next stage has landed
                else __builtin_amdgcn_s_waitcnt(0xC07F);  // lgkmcnt(0)
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_setprio(1);
#pragma unroll
                for (int m = 0; m < RT; ++m)
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[m][c] = mfma(wv[c], xv[m], acc[m][c]);
                __builtin_amdgcn_s_setprio(0);
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_barrier();
                __builtin_amdgcn_sched_barrier(0);
            }
            u = UNITS ? next_weight_unit(u) : u == 2 ? 0 : u + 1;
        }
        store_tile<OT, 32, RT, CT>(acc, xs, ws, p, t.row0 + 16 * wy, t.rows - 16 * wy, t.n0 + wx * 64);
        if (after.rows == 0) break;
        t = after;
        bx = ax;
        bw = aw;
    }
    if (wy == 0) __builtin_amdgcn_s_barrier();
    wait_loads<0, false>();  // nothing is on its way into LDS any more
}

// ---- launches ----

template <typename OT, Rows ROWS> hipError_t launch_small(const ProductParams& p, hipStream_t s) {
    constexpr bool HELD = ROWS != STREAMED;
    const int64_t runs = (p.n_out + 15) / 16, tiles = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, HELD ? held_rows(p.n_in) : SMALL_MAX_ROWS);
    const int split = small_split(p.n_out, tiles, p.n_in, HELD);
    const dim3 grid((unsigned)((runs * split + SMALL_WAVES - 1) / SMALL_WAVES), (unsigned)tiles);
    small_kernel<OT, ROWS><<<grid, SMALL_WAVES * 64, 0, s>>>(p, split);
    return hipGetLastError();
}

template <typename OT, int TM, int TN, int RING> hipError_t launch_strip(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, TM), cols = (p.n_out + TN - 1) / TN;
    strip_kernel<OT, TM, TN, RING><<<(unsigned)xcd_padded(rows * cols), 256, 0, s>>>(p, (int)rows, (int)cols);
    return hipGetLastError();
}

template <typename OT, int PER, int RING> hipError_t launch_medium(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 64), cols = (p.n_out + 63) / 64;
    medium_kernel<OT, PER, RING><<<(unsigned)xcd_padded(rows * cols), 256, 0, s>>>(p, (int)rows, (int)cols);
    return hipGetLastError();
}

template <typename OT> hipError_t launch_middle(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 128), cols = (p.n_out + 127) / 128;
    middle_kernel<OT><<<(unsigned)xcd_padded(rows * cols), 256, 0, s>>>(p, (int)rows, (int)cols);
    return hipGetLastError();
}

template <typename OT, int RT> hipError_t launch_large(const ProductParams& p, hipStream_t s) {
    const int64_t rows = max_row_tiles(p.offsets != nullptr, p.rows, p.n_groups, 32 * RT), cols = (p.n_out + LARGE_COLS - 1) / LARGE_COLS;
    const int64_t tiles = xcd_padded(rows * cols);
    large_kernel<OT, RT><<<(unsigned)(tiles < CUS ? tiles : CUS), 512, 0, s>>>(p, (int)rows, (int)cols, (int)tiles);
    return hipGetLastError();
}

template <typename OT> hipError_t launch_product(const ProductParams& p, hipStream_t s) {
    if (p.x) return launch_small<OT, QUANTISED>(p, s);
    const ProductChoice c = choose_product(ProductShape{p.offsets != nullptr, p.rows, p.n_groups, p.n_in, p.n_out});
    switch (c.kernel) {
        case SMALL_STAGED: return launch_small<OT, STAGED>(p, s);
        case SMALL_STREAMED: return launch_small<OT, STREAMED>(p, s);
        case STRIP_16: return launch_strip<OT, 32, 16, 3>(p, s);
        case STRIP_32: return launch_strip<OT, 32, 32, 2>(p, s);
        case STRIP_64: return launch_strip<OT, 32, 64, 2>(p, s);
        case MEDIUM_LONG: return launch_medium<OT, 16, 4>(p, s);
        case MEDIUM_SHORT: return launch_medium<OT, 8, 5>(p, s);
        case MIDDLE: return launch_middle<OT>(p, s);
        case LARGE_128: return launch_large<OT, 4>(p, s);
        case LARGE_256: return launch_large<OT, 8>(p, s);
        case LARGE_BOTH: {
            ProductParams left = p, right = p;
            left.n_out = c.cols;
            right.n_out = p.n_out - c.cols;
            right.wc += (int64_t)c.cols * p.n_in;
            right.ws += c.cols;
            right.y = static_cast<char*>(p.y) + (int64_t)c.cols * OT::bytes;
            const hipError_t e = launch_large<OT, 8>(left, s);
            return e == hipSuccess ? launch_large<OT, 4>(right, s) : e;
        }
    }
    return hipErrorInvalidValue;  // not reached
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
    return quantised_inside(rows, n_groups, n_in) ? 0 : codes_bytes(rows, n_in) + (((int64_t)rows * 4 + 255) & ~int64_t(255));
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
    const ProductParams p = {nullptr, 0, x_codes, x_scales, offsets, n_groups, rows, codes, scales, n_in, n_out, y, n_out};
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
    ProductParams p = {x, ldx, nullptr, nullptr, offsets, n_groups, rows, codes, scales, n_in, n_out, y, n_out};
    if (need > 0) {
        int8_t* const xc = static_cast<int8_t*>(workspace);
        float* const xs = reinterpret_cast<float*>(xc + codes_bytes(rows, n_in));
        const RowsParams q = {x, ldx, nullptr, 0, nullptr, 0, 0.0, rows, n_in, xc, xs, nullptr};
        if (launch_quantize(dtype, q, (hipStream_t)stream) != hipSuccess) return EXL3_EHIP;
        p.x = nullptr;
        p.xc = xc;
        p.xs = xs;
    }
    return product(dtype, p, (hipStream_t)stream) == hipSuccess ? EXL3_OK : EXL3_EHIP;
}

}  // extern "C"
