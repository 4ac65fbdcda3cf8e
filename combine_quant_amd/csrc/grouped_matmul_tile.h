// grouped_matmul_tile.h -- the experts' products in tiles of up to 256 rows x 256 weight rows.
//
// out = x w^T per expert; every row of x and of the weights is walked in steps of 128 bytes,
// whatever the type (64 16-bit elements, 128 codes), 128 bytes being 2048 matrix clocks of a full
// tile for each of them.  Few rows per expert are bound by the weights' bytes: 512 rows on 32
// experts x 7168 x 4096 bf16 take 306 us, 6.2 TB/s, a read's rate on this chip.  Many rows are
// bound by the matrix units at the clock they leave: 16384 rows on 8 experts x 7168 x 4096 run in
// 737 us in bf16 (1310 Tflop/s), 775 in fp16, 392 in E4M3 (2450), 404 in int8, 461 in MX E4M3, 470
// to 490 in block-scaled E4M3 (whose scaled additions take as many vector cycles as the products
// matrix cycles; three of four left out give 8 %), with the matrix units busy 72 % of a workgroup's
// time at 1.76 GHz (bf16).  Without its loads the loop takes 0.60 ms of the 0.74, without its products
// 0.56; without the barrier 3 % less, without the waits for loads no less.
//
// Also tried at that size: both operands in two stages with one barrier a step (0.99 ms against
// 0.86), the weights straight to registers (1.03), two waves sharing 64 weight rows, which halves
// their LDS reads of x (0.82 against 0.79), an L2 prefetch some steps ahead (no change), a
// persistent grid with shares of equal cost (0.95 against 0.89).
#pragma once

#include "experts_tiles.h"

namespace moe_dc {
namespace {

constexpr int kTileRing = 3;                    // steps of x in LDS

// WAVES: 8, or 4 for thin tiles (kThinRows rows x 128 weight rows), two of which share a CU.
template <int TYPE, int WAVES>
constexpr int kTileM = WAVES == kTileWaves ? tile_rows(TYPE) : kThinRows;

template <int TYPE, int WAVES>
struct TileStages {
    static constexpr int kRows = kTileM<TYPE, WAVES>, kScaleRows = (kRows + 63) / 64 * 64;
    char x[kTileRing][kRows * 128];             // [row][128 bytes], swizzled
    char w[WAVES][2][32 * 128];                 // each wave's own 32 weight rows, swizzled
    // MX: the E8M0 bytes of four steps, 16 of each row of x, then of each weight row (with the
    // four bytes of one step at a time the requests for them outnumbered the rows': 3.45 ms
    // instead of 2.63 at 65536 skewed rows on 256 experts x 7168 x 4096)
    // Block: the floats of four steps, likewise 16 bytes of each row of x, then of the tile's two
    // rows of weight blocks
    char scales[2][Mm<TYPE>::kMx ? (kScaleRows + kTileN) * 16 : Mm<TYPE>::kBlk ? (kScaleRows + 64) * 16 : 0];
};

// The table is done with before the first stage is filled, and the stages before the largest
// values of a coded output meet: of each row, per wave (Mm<TYPE>::kBlk).
template <int TYPE, int WAVES>
union TileLds {
    TileStages<TYPE, WAVES> st;
    TileTable table;
    uint32_t amax[Mm<TYPE>::kBlk ? kTileM<TYPE, WAVES> * WAVES : 1];
};

// Four values as codes, the first in the lowest byte.  None is NaN.
__device__ __forceinline__ uint32_t code4(const float (&v)[4], int code)
{
    const float top = code == kCodeE4m3 ? 448.0f : 57344.0f;
    float c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) c[q] = __builtin_amdgcn_fmed3f(v[q], -top, top);
    int w;
    if (code == kCodeE4m3) {
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], w, true);
    } else {
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c[0], c[1], 0, false);
        w = __builtin_amdgcn_cvt_pk_bf8_f32(c[2], c[3], w, true);
    }
    return (uint32_t)w;
}

// A tile's sums as codes with one scale per row and 128 columns, as dispatch codes a token in mode
// 3.  A tile holds one group of columns with SwiGLU or thin, else two, so the largest values of 8 or 4
// waves meet in LDS and nothing but the codes leaves the workgroup.  In a group with an infinity or a
// NaN (whose bits are the largest) the scale is NaN and the codes are 0.
template <int TYPE, int WAVES, int MT, bool SWIGLU>
__device__ __forceinline__ void code_tile(const MatmulShape& s, const MatmulArgs& a, const Tile& tile,
                                          int half, int left, v4f_t (&acc)[MT][2], uint32_t* amax)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    constexpr int kT = SWIGLU ? 1 : 2;
    constexpr int kMeet = kBlock / (kT * 16);                        // waves of a group
    static_assert(WAVES % kMeet == 0, "a group of columns lies within one tile");
    const int c0 = wave * (kT * 16) + g * 4;
    __syncthreads();                            // the last step's rows have been read
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        uint32_t most = 0;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            if (SWIGLU) {
                float y[4], u[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    y[q] = acc[m][0][q];
                    u[q] = acc[m][1][q];
                }
                silu_mul4(y, u, y);
#pragma unroll
                for (int q = 0; q < 4; ++q) acc[m][0][q] = y[q];
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t bits = __float_as_uint(acc[m][t][q]) & 0x7FFFFFFFu;
                if (c0 + t * 16 + q < left && bits > most) most = bits;
            }
        }
        most = dpp_max(most, __shfl_xor(most, 16, kWave));
        most = dpp_max(most, __shfl_xor(most, 32, kWave));
        if (g == 0) amax[(m * 16 + l16) * WAVES + wave] = most;
    }
    __syncthreads();
    const int first = wave / kMeet * kMeet;
    const int groups = (half + kBlock - 1) / kBlock;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + l16;
        if (row >= tile.rows) continue;
        uint32_t most = 0;
#pragma unroll
        for (int w = 0; w < kMeet; ++w) most = dpp_max(most, amax[row * WAVES + first + w]);
        const bool finite = most < 0x7F800000u;
        float dyn = (s.out_code == kCodeE4m3 ? 448.0f : 57344.0f) / __uint_as_float(most);
        const float scale = finite ? 1.0f / dyn : NAN;
        uint8_t* o = static_cast<uint8_t*>(a.out) + (size_t)(tile.row0 + row) * half + tile.n0;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            const int c = c0 + t * 16;
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float p = acc[m][t][q] * dyn;
                v[q] = finite && p == p ? p : 0.0f;
            }
            const uint32_t p = code4(v, s.out_code);
            if (c + 3 < left && (reinterpret_cast<uintptr_t>(o + c) & 3) == 0) {
                *reinterpret_cast<uint32_t*>(o + c) = p;
            } else {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (c + q < left) o[c + q] = (uint8_t)(p >> (8 * q));
            }
        }
        // the group's first columns' lanes write its scale
        if (wave == first && g == 0 && first * kT * 16 < left)
            a.out_scales[(size_t)(tile.row0 + row) * groups + (tile.n0 + first * kT * 16) / kBlock] = scale;
    }
}

// One tile: 16 * MT rows of x from row0 (of which `rows` exist), 256 weight rows from column n0.
// Wave w owns weight rows 32 * w + 0..31 of the tile (with SwiGLU 16 gate rows and the 16 up rows
// of the same columns) and multiplies them with every row of x.  All operands come through LDS,
// moved there by the loads themselves: the matrix layout wants neighbouring lanes in different
// rows, which as a load from global memory runs at 16 bytes a clock per CU (9.4 TB/s over the
// chip, against 24 TB/s for whole 128-byte rows).
//
// Step k (128 bytes of every row) waits for its own operands only.  x lies in a ring of three
// stages: the barrier of step k makes x(k) visible and frees the stage that step k - 1 read,
// which takes x(k + 2).  A wave's weights are its own, so they need no barrier: the operands of
// step k + 1 move from LDS to registers at the start of step k, and their place takes the weights
// of step k + 3.  Loads past the end of a row return 0 without a memory access, so every step
// issues the same number.
//
// CODED (block): the results leave as codes.  What the fp8 instructions cut (1.5e-5 of a sum) then
// shows as another code, a step of 6 to 25 %, in 8 to 16 of 10 000 results, so tiles of up to 64 rows, which
// the matrix units do not bound, form whole products (333 rows on 12 experts x 1136 x 1424, SwiGLU: 14.5 us
// instead of 11.0).  Taller tiles do not: 16384 rows on 32 experts x 7168 x 4096, SwiGLU, would take 955 us
// instead of 566, for values that are off by 0.00008 of their norm instead of 0.0012 where the codes
// themselves are off by 0.023 (E4M3).  So a row's codes depend on its tile's height, as the header says.
template <int TYPE, int WAVES, int MT, bool SWIGLU, bool CODED = false>
__device__ __forceinline__ void tile_product(const MatmulShape& s, const MatmulArgs& a,
                                             const Tile& tile, TileLds<TYPE, WAVES>& shared)
{
    TileStages<TYPE, WAVES>& lds = shared.st;
    constexpr int kRows = kTileM<TYPE, WAVES>, kWeightRows = 32 * WAVES;
    constexpr int kScaleRows = TileStages<TYPE, WAVES>::kScaleRows;
    constexpr bool kWhole = CODED && MT <= 4;
    const int e = tile.e, n0 = tile.n0, row0 = tile.row0, rows = tile.rows;
    typedef Mm<TYPE> M;
    typedef typename M::Acc Acc;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = (uint32_t)s.in * M::kBytes;
    const int steps = (int)((row_bytes + 127) / 128);
    const int half = SWIGLU ? s.out / 2 : s.out;
    constexpr int kCols = SWIGLU ? kWeightRows / 2 : kWeightRows;    // columns of the output
    const int left = half - n0 < kCols ? half - n0 : kCols;
    const char* wbase = static_cast<const char*>(a.w) + ((size_t)e * s.out + n0) * row_bytes;
    const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(wbase, (uint32_t)left * row_bytes);
    const __amdgpu_buffer_rsrc_t wr1 =
        make_rsrc(wbase + (size_t)half * row_bytes, (uint32_t)left * row_bytes);
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(static_cast<const char*>(a.x) + (size_t)row0 * row_bytes, (uint32_t)rows * row_bytes);
    // bytes of scales of a row of x, and of a weight row (MX) or of 128 of them (block)
    const uint32_t ns = M::kBlk ? (uint32_t)steps * 4 : (uint32_t)s.in / 32;
    const int blocks = (half + kBlock - 1) / kBlock;         // rows of weight blocks, of gate or up
    const char* wsb = static_cast<const char*>(a.w_scales) +
        (M::kBlk ? ((size_t)e * blocks * (SWIGLU ? 2 : 1) + n0 / kBlock) * ns : ((size_t)e * s.out + n0) * ns);

    // One load moves 8 rows of 128 bytes; lane i brings row i / 8 the 16 bytes that belong at
    // position i % 8, which holds chunk (i % 8) ^ (row & 7).
    const int lr = lane >> 3;
    const uint32_t lk = (uint32_t)((lane & 7) ^ lr) * 16;
    constexpr int kBlocks = 2 * MT;                          // of 8 rows
    constexpr int kXLoads = (kBlocks + WAVES - 1) / WAVES;
    // (where the blocks do not go round, some waves load again what another one does, so that
    // every wave issues the same number without a branch)
    uint32_t xoff[kXLoads], woff[4];
    int xblk[kXLoads];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
        xblk[i] = wave + i * WAVES;
        if (xblk[i] >= kBlocks) xblk[i] %= kBlocks;
        xoff[i] = (uint32_t)(xblk[i] * 8 + lr) * row_bytes + lk;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = SWIGLU ? wave * 16 + (i & 1) * 8 : wave * 32 + i * 8;
        woff[i] = (uint32_t)(r + lr) * row_bytes + lk;
    }
    // MX: every fourth step a wave brings 16 bytes of scales of 64 rows: waves 0-2 rows of x,
    // waves 3-6 weight rows (wave 7 the same as wave 6).  Rows are ns bytes, ns a multiple of 4.
    // Block: the first waves rows of x (0-3 of 224 rows, 0 of a thin tile's 64), all others the same two
    // rows of weight blocks, of columns n0 and n0 + 128 or of gate and up.
    constexpr bool kLdsScales = M::kMx || M::kBlk;
    const bool sx = wave * 64 < kRows;
    const int sblk = sx ? wave : M::kBlk ? 0 : (wave < 6 ? wave : 6) - kScaleRows / 64;
    const int srow = sblk * 64 + lane;
    const int scol = SWIGLU ? srow / 32 * 16 + (srow & 15) : srow;      // of the weight row
    const bool sok = sx ? srow < rows : M::kBlk ? srow < 2 && (SWIGLU || srow * kBlock < left) : scol < left;
    const uint32_t soff = (uint32_t)(sx ? srow : M::kBlk ? (SWIGLU ? srow * blocks : srow)
                                                 : SWIGLU && (srow & 16) ? half + scol : scol) * ns;
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(
        sx ? static_cast<const char*>(a.x_scales) + (size_t)row0 * ns : wsb,
        !kLdsScales ? 0 : (uint32_t)(sx ? rows : M::kBlk ? (SWIGLU ? blocks + 1 : left > kBlock ? 2 : 1)
                                                  : SWIGLU ? half + left : left) * ns);
    const int sto = (sx ? 0 : kScaleRows * 16) + sblk * 1024;
    // The 16 bytes of a row's last window end where the row does (from the window's own start they
    // would run into the next row and, of the last row, past the tensor), so that its steps lie
    // scale_shift bytes further; a row of fewer than 16 bytes comes a step's dword at a time, as
    // [64 rows' block][step][row][4 bytes].
    const auto scale_shift = [&](int window) {
        const uint32_t k = (uint32_t)window * 16;
        return k < ns && k + 16 > ns ? (int)(k + 16 - ns) : 0;
    };
    const auto fetch_scales = [&](int window) {
        const uint32_t k = (uint32_t)(window * 16 - scale_shift(window));
        char* to = lds.scales[window & 1] + sto;
        if (ns >= 16) {
            load_lds16(sr, to, sok && k < ns ? soff + k : kRsrcPastEnd);
        } else if (window == 0) {
#pragma unroll
            for (uint32_t d = 0; d < 12; d += 4)
                load_lds4(sr, to + d * 64, sok && d < ns ? soff + d : kRsrcPastEnd);
        }
    };
    // The scale of a step for row r + i (r a multiple of 16 or 64).  Steps of windows known to be
    // full need no shift; only those after the unrolled loop may be of rows below 16 bytes.
    enum Where { kFull, kPerhapsLast, kAfterLoop };
    const auto scale_at = [&](Where where, int step, int r, int i) {
        const char* to = lds.scales[step >> 2 & 1];
        const int k = step & 3;
        // (the address as a pointer moved step by step: summed as a number first, and chosen between the two
        // cases, it cost MX tiles 10 registers, spills and 2.5 %, and block tiles 209 to 225 spilled registers)
        const auto read = [&](const char* at) {
            return M::kBlk ? *reinterpret_cast<const int*>(at) : (int)*reinterpret_cast<const uint8_t*>(at + g);
        };
        if (where == kAfterLoop && ns < 16) return read(to + (r >> 6) * 1024 + k * 256 + ((r & 63) + i) * 4);
        if (where != kFull) to += scale_shift(step >> 2);
        return read(to + (r + i) * 16 + k * 4);
    };
    const auto scale_of = [&](Where where, int step, int r) { return scale_at(where, step, r, l16); };
    // Load i of a step's x, and of its weights.
    const auto fetch_x = [&](int step, int i) {
        const uint32_t k = (uint32_t)step * 128;
        const bool past = k + lk >= row_bytes;
        char* to = lds.x[step % kTileRing];
        load_lds16(xr, to + xblk[i] * 1024, past ? kRsrcPastEnd : xoff[i] + k);
    };
    const auto fetch_w = [&](int step, int i) {
        const uint32_t k = (uint32_t)step * 128;
        const bool past = k + lk >= row_bytes;
        char* to = lds.w[wave][step & 1];
        load_lds16(SWIGLU && i >= 2 ? wr1 : wr0, to + i * 1024, past ? kRsrcPastEnd : woff[i] + k);
    };

    const int f0 = l16 * 128 + ((g ^ (l16 & 7)) << 4);
    const int f1 = l16 * 128 + (((4 + g) ^ (l16 & 7)) << 4);
    v8i_t w[2][2];
    int wsc[2][2] = {{0, 0}, {0, 0}};
    const auto read_w = [&](int par, int step, Where where) {
        const char* wl = lds.w[wave][par];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            w[par][t] = join(*reinterpret_cast<const v4i_t*>(wl + t * 2048 + f0),
                             *reinterpret_cast<const v4i_t*>(wl + t * 2048 + f1));
            if (M::kMx) wsc[par][t] = scale_of(where, step, kScaleRows + wave * 32 + t * 16);
            if (M::kBlk) wsc[par][t] = scale_at(where, step, kScaleRows, SWIGLU ? t : wave >> 2);
        }
    };
    Acc acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = Acc{0, 0, 0, 0};

    // loads issued after those a step waits for: x(k + 1), weights(k + 2)
    constexpr int kAhead = kXLoads + 4;
    const auto all_x = [&](int step) {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) fetch_x(step, i);
    };
    const auto all_w = [&](int step) {
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch_w(step, i);
    };
    if (kLdsScales) fetch_scales(0);
    all_x(0);
    all_w(0);
    all_w(1);
    all_x(1);
    wait_loads<kAhead>();
    if (kLdsScales) meet();                     // the scales come from other waves
    read_w(0, 0, kAfterLoop);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    all_w(2);
    // A step's products go in groups of 32 rows (the last one perhaps 16): a group reads the next
    // group's rows from LDS and issues its share of the step's loads before its own products.
    // (Issued together at the step's start, the loads fill the address queue and hold up the
    // products: 1.09 ms instead of 0.86 at 16384 rows on 32 experts x 7168 x 4096 bf16.)  The
    // first half of the groups loads x(k + 2), the second the weights of k + 3, whose place is
    // free once read_w has returned: two groups after it, since LDS reads return in order and the
    // products between have waited for rows read after it; with fewer groups by a wait.
    constexpr int kGroups = (MT + 1) / 2;
    constexpr int kXGroups = kGroups > 1 ? kGroups / 2 : 1;
    constexpr int kWFirst = kGroups > 1 ? kGroups / 2 : 0, kWGroups = kGroups - kWFirst;
    constexpr int kReadW = kWFirst >= 2 ? kWFirst - 2 : 0;
    // Block: the sums of a group's tiles wait here with their scales until the next group's products
    // (perhaps the next step's) take their place, so that no product is waited for.
    v4f_t late[2][2] = {{{0, 0, 0, 0}, {0, 0, 0, 0}}, {{0, 0, 0, 0}, {0, 0, 0, 0}}};
    float late_scale[2][2] = {{0.0f, 0.0f}, {0.0f, 0.0f}};
    const auto settle = [&](int group, int i, int t) {
        if constexpr (M::kBlk)
            if (group * 2 + i < MT) add_scaled(acc[group * 2 + i][t], late[i][t], late_scale[i][t]);
    };
    const auto settle_all = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) settle(kGroups - 1, i >> 1, i & 1);
    };
    // phase: step modulo the unrolling
    const auto one = [&](int phase, int step, Where where) {
        const int par = phase & 1;
        wait_loads<kAhead>();
        meet();
        const char* xl = lds.x[step % kTileRing];
        if (kLdsScales && phase == 0) fetch_scales((step >> 2) + 1);
        v8i_t x[2][2];
        int xsv[2][2] = {{0, 0}, {0, 0}};
        const auto read_x = [&](int set, int group) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int m = group * 2 + i;
                if (m >= MT) break;
                x[set][i] = join(*reinterpret_cast<const v4i_t*>(xl + m * 2048 + f0),
                                 *reinterpret_cast<const v4i_t*>(xl + m * 2048 + f1));
                if (kLdsScales) xsv[set][i] = scale_of(where, step, m * 16);
            }
        };
        read_x(0, 0);
#pragma unroll
        for (int q = 0; q < kGroups; ++q) {
            if (q == kReadW) {
                read_w(par ^ 1, step + 1, where == kFull && phase == 3 ? kPerhapsLast : where);
                __builtin_amdgcn_sched_barrier(0x7F);        // LDS reads stay before read_x(q + 1)
            }
            if (q + 1 < kGroups) read_x((q + 1) & 1, q + 1);
            if (q == kWFirst && kWFirst < kReadW + 2)
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
#pragma unroll
            for (int i = 0; i < kXLoads; ++i)
                if (i * kXGroups / kXLoads == q) fetch_x(step + 2, i);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (kWFirst + i * kWGroups / 4 == q) fetch_w(step + 3, i);
            __builtin_amdgcn_sched_barrier(0);
            if constexpr (M::kBlk) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if (q > 0 || where == kFull) settle(q > 0 ? q - 1 : kGroups - 1, i, t);
                        if (q * 2 + i >= MT) continue;
                        if constexpr (kWhole) late[i][t] = M::mma_whole(w[par][t], x[q & 1][i]);
                        else late[i][t] = M::mma(w[par][t], x[q & 1][i], Acc{0, 0, 0, 0}, 0, 0);
                        late_scale[i][t] = __int_as_float(wsc[par][t]) * __int_as_float(xsv[q & 1][i]);
                    }
                // in turn: the additions that free a tile's place, its product
#pragma unroll
                for (int i = 0; !kWhole && i < 4 && q * 2 + i / 2 < MT; ++i) {
                    __builtin_amdgcn_sched_group_barrier(0x002, 5, 0);
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < 2 && q * 2 + i < MT; ++i)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        acc[q * 2 + i][t] = M::mma(w[par][t], x[q & 1][i], acc[q * 2 + i][t], wsc[par][t],
                                                   xsv[q & 1][i]);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (where == kAfterLoop) settle_all();
    };
    constexpr int kUnroll = kLdsScales ? 4 : 2;
    int step = 0;
    for (; step + kUnroll <= steps; step += kUnroll) {
#pragma unroll
        for (int r = 0; r < kUnroll; ++r) one(r, step + r, kFull);
    }
    if (step > 0) settle_all();
#pragma unroll
    for (int r = 0; r < kUnroll - 1; ++r)
        if (step + r < steps) one(r, step + r, kAfterLoop);
    wait_loads<0>();                            // nothing may land in LDS after the tile

    constexpr int kT = SWIGLU ? 1 : 2;
    const int c0 = wave * (kT * 16) + g * 4;    // the lane's first column
    if constexpr (CODED) {
        code_tile<TYPE, WAVES, MT, SWIGLU>(s, a, tile, half, left, acc, shared.amax);
        return;
    }
    float ws_[2][4];
    if (M::kRowScaled) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int c = c0 + (SWIGLU ? 0 : t * 16) + q;
                ws_[t][q] = c < left ? static_cast<const float*>(
                    a.w_scales)[(size_t)e * s.out + n0 + c + (SWIGLU ? t * half : 0)] : 0.0f;
            }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int row = m * 16 + l16;
        if (row >= rows) continue;
        float rs = 1.0f;
        if (M::kRowScaled && a.x_scales) rs = static_cast<const float*>(a.x_scales)[row0 + row];
        uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)(row0 + row) * half + n0;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            const int c = c0 + t * 16;
            float y[4], u[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                y[q] = (float)acc[m][t][q];
                if (M::kRowScaled) y[q] = y[q] * ws_[t][q] * rs;
                if (SWIGLU) {
                    u[q] = (float)acc[m][1][q];
                    if (M::kRowScaled) u[q] = u[q] * ws_[1][q] * rs;
                }
            }
            if (SWIGLU) silu_mul4(y, u, y);
            const uint2 p = make_uint2(pack_out2(y[0], y[1], s.tok_f16), pack_out2(y[2], y[3], s.tok_f16));
            store_columns(o, c, left, p);
        }
    }
}

template <int TYPE, bool SWIGLU, bool CODED>
__global__ __launch_bounds__(kTileThreads, 2) void tile_kernel(MatmulShape s, MatmulArgs a)
{
    constexpr int WAVES = kTileWaves;
    __shared__ TileLds<TYPE, WAVES> lds;
    constexpr int kRows = kTileM<TYPE, WAVES>;
    Tile t;
    if (!find_tile<kRows, SWIGLU ? kTileN / 2 : kTileN>(s, a, SWIGLU ? s.out / 2 : s.out, lds.table, &t))
        return;
    switch ((t.rows + 15) / 16) {
    case 1: tile_product<TYPE, WAVES, 1, SWIGLU, CODED>(s, a, t, lds); break;
    case 2: tile_product<TYPE, WAVES, 2, SWIGLU, CODED>(s, a, t, lds); break;
    case 3: tile_product<TYPE, WAVES, 3, SWIGLU, CODED>(s, a, t, lds); break;
    case 4: tile_product<TYPE, WAVES, 4, SWIGLU, CODED>(s, a, t, lds); break;
    case 5: tile_product<TYPE, WAVES, 5, SWIGLU, CODED>(s, a, t, lds); break;
    case 6: tile_product<TYPE, WAVES, 6, SWIGLU, CODED>(s, a, t, lds); break;
    case 7: tile_product<TYPE, WAVES, 7, SWIGLU, CODED>(s, a, t, lds); break;
    case 8: tile_product<TYPE, WAVES, 8, SWIGLU, CODED>(s, a, t, lds); break;
    case 9: tile_product<TYPE, WAVES, 9, SWIGLU, CODED>(s, a, t, lds); break;
    case 10: tile_product<TYPE, WAVES, 10, SWIGLU, CODED>(s, a, t, lds); break;
    case 11: tile_product<TYPE, WAVES, 11, SWIGLU, CODED>(s, a, t, lds); break;
    case 12: tile_product<TYPE, WAVES, 12, SWIGLU, CODED>(s, a, t, lds); break;
    default:
        if constexpr (kRows > 192) switch ((t.rows + 15) / 16) {
            case 13: tile_product<TYPE, WAVES, 13, SWIGLU, CODED>(s, a, t, lds); break;
            case 14: tile_product<TYPE, WAVES, 14, SWIGLU, CODED>(s, a, t, lds); break;
            default:
                if constexpr (kRows > 224) {
                    if ((t.rows + 15) / 16 == 15) tile_product<TYPE, WAVES, 15, SWIGLU, CODED>(s, a, t, lds);
                    else tile_product<TYPE, WAVES, 16, SWIGLU, CODED>(s, a, t, lds);
                }
                break;
            }
        break;
    }
}

// Few rows per expert: tiles of at most kThinRows rows.
template <int TYPE, bool SWIGLU, bool CODED>
__global__ __launch_bounds__(4 * kWave, 2) void thin_tile_kernel(MatmulShape s, MatmulArgs a)
{
    constexpr int WAVES = 4;
    __shared__ TileLds<TYPE, WAVES> lds;
    Tile t;
    if (!find_tile<kThinRows, SWIGLU ? kThinN / 2 : kThinN, WAVES>(s, a, SWIGLU ? s.out / 2 : s.out, lds.table, &t)) return;
    switch ((t.rows + 15) / 16) {
    case 1: tile_product<TYPE, WAVES, 1, SWIGLU, CODED>(s, a, t, lds); break;
    case 2: tile_product<TYPE, WAVES, 2, SWIGLU, CODED>(s, a, t, lds); break;
    case 3: tile_product<TYPE, WAVES, 3, SWIGLU, CODED>(s, a, t, lds); break;
    default: tile_product<TYPE, WAVES, 4, SWIGLU, CODED>(s, a, t, lds); break;
    }
}

template <int TYPE, bool CODED = false>
hipError_t launch_thin_tiles(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    const dim3 grid(tile_grid(s, kThinRows, s.swiglu ? kThinN / 2 : kThinN));
    if constexpr (!CODED) {                      // (thin tiles do not hold whole groups of gate and up)
        if (s.swiglu) {
            thin_tile_kernel<TYPE, true, false><<<grid, 4 * kWave, 0, stream>>>(s, a);
            return hipGetLastError();
        }
    }
    thin_tile_kernel<TYPE, false, CODED><<<grid, 4 * kWave, 0, stream>>>(s, a);
    return hipGetLastError();
}

template <int TYPE, bool CODED = false>
hipError_t launch_tiles(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    const dim3 grid(tile_grid(s, tile_rows(TYPE), s.swiglu ? kTileN / 2 : kTileN));
    if (s.swiglu)
        tile_kernel<TYPE, true, CODED><<<grid, kTileThreads, 0, stream>>>(s, a);
    else
        tile_kernel<TYPE, false, CODED><<<grid, kTileThreads, 0, stream>>>(s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace moe_dc
