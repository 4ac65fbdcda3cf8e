// grouped_matmul_w4_tile.h -- 4-bit products in tiles.
//
// A workgroup of eight waves multiplies up to 128 rows of x with 256 weight rows, or one of four
// waves up to 32 rows with 128, in steps of 128 elements; wave w owns weight rows 32 * w + 0..31
// (with SwiGLU 16 gate rows and the 16 up rows of the same columns) and takes every row of x.  x
// (256 bytes a row and step), a wave's codes (64 bytes a row and step) and its scales lie in LDS
// rings, moved there by the loads themselves; the rings are three steps deep for 96 and 128 rows,
// four below, where a step is short against the memory's latency.  (No load goes to a register:
// the wait for it would be one for every load before it too; with the scales in registers, loaded
// one by one, 512 rows on 32 experts x 7168 x 4096 E2M1 took 285 us instead of 150.)  Each step
// decodes the codes of the next one to 16-bit floats in registers, a part with each part of its
// own products, so that the conversions run beside the matrix instructions.
//
// Few rows are bound by the instructions that turn codes into operands (155 a wave and step),
// above the bytes: 16 rows on 16 of 64 experts x 7168 x 4096 int4 (227 MB) take 53 us with the same
// weights again, 62 with others between, 32 experts with 16 rows each (493 MB) 131 us, 3.8 TB/s.
// With many rows the matrix units are the bound, but with 128 rows a weight's decoding serves few
// products, and a tile's start and end take 10 us: 4096 rows on 32 experts x 2048 x 7168 E2M1 take
// 186-192 us, 640 Tflop/s (16 steps a tile); at inner size 8192 it is 760, int4 at 4096 670.
//
// x is the A operand (rows of the result) and the weights B (columns): lane l holds column l % 16
// and rows (l / 16) * 4 + 0..3, hence one scale per lane and column tile.
#pragma once

#include "grouped_matmul_w4.h"

namespace moe_dc {
namespace {

constexpr int kW4SmallWaves = 4;
constexpr int kW4LdsBytes = 163840;

// Steps held in LDS by tiles of MT * 16 rows.
constexpr int w4_ring(int mt) { return mt <= 4 ? 4 : 3; }

template <int MT, int WAVES>
struct W4Stages {
    char x[w4_ring(MT)][2][MT * 16 * 128];      // [64 elements][row][128 bytes], swizzled
    char w[WAVES][w4_ring(MT)][32 * 64];        // each wave's own weight rows, swizzled
    // dwords of scales: of each of the wave's rows the one a step's scales begin in, then the
    // next; then (8 bytes of scales a step) the one after
    uint32_t s[WAVES][w4_ring(MT)][128];
};

union W4Lds {
    W4Stages<2, kTileWaves> s2;
    W4Stages<4, kTileWaves> s4;
    W4Stages<6, kTileWaves> s6;
    W4Stages<8, kTileWaves> s8;
    TileTable table;
};
union W4SmallLds {
    W4Stages<1, kW4SmallWaves> s1;
    W4Stages<2, kW4SmallWaves> s2;
    TileTable table;
};
static_assert(sizeof(W4Lds) <= kW4LdsBytes && 2 * sizeof(W4SmallLds) <= kW4LdsBytes, "LDS of a CU");

// Eight codes of a dword as decode gives them, int4 for fp16 in their order too (a tile's x is
// used by every column, so the weights are put in order instead).
template <bool F16, bool E2M1>
__device__ __forceinline__ v4i_t decode_tile(uint32_t w, float scale)
{
    v4i_t r = decode<F16, E2M1>(w, scale);
    if constexpr (F16 && !E2M1) {
        const v4i_t p = r;                                   // 0 4, 1 5, 2 6, 3 7
        r.x = (int)__builtin_amdgcn_perm((uint32_t)p.y, (uint32_t)p.x, 0x05040100u);
        r.y = (int)__builtin_amdgcn_perm((uint32_t)p.w, (uint32_t)p.z, 0x05040100u);
        r.z = (int)__builtin_amdgcn_perm((uint32_t)p.y, (uint32_t)p.x, 0x07060302u);
        r.w = (int)__builtin_amdgcn_perm((uint32_t)p.w, (uint32_t)p.z, 0x07060302u);
    }
    return r;
}

template <bool F16, bool E2M1, int STEPS, int MT, bool SWIGLU, int WAVES>
__device__ __forceinline__ void w4_tile_product(const MatmulShape& s, const MatmulArgs& a,
                                                const Tile& tile, W4Stages<MT, WAVES>& lds)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t xrow = (uint32_t)s.in * 2, wrow = (uint32_t)s.in / 2;
    const int steps = (s.in + 127) / 128;
    const int half = SWIGLU ? s.out / 2 : s.out;
    constexpr int kCols = SWIGLU ? WAVES * 16 : WAVES * 32;
    const int left = half - tile.n0 < kCols ? half - tile.n0 : kCols;
    const size_t first = (size_t)tile.e * s.out + tile.n0;
    const char* wbase = static_cast<const char*>(a.w) + first * wrow;
    const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(wbase, (uint32_t)left * wrow);
    const __amdgpu_buffer_rsrc_t wr1 = make_rsrc(wbase + (size_t)half * wrow, (uint32_t)left * wrow);
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(
        static_cast<const char*>(a.x) + (size_t)tile.row0 * xrow, (uint32_t)tile.rows * xrow);
    // Scales are read as whole dwords (the tensor begins at one, rows begin anywhere).
    constexpr int kSize = E2M1 ? 1 : 2;                      // bytes of a scale
    constexpr int kParts = 4 / STEPS;                        // scales of a row and step
    constexpr int kStepBytes = kParts * kSize;               // 2, 4 or 8
    constexpr int kSLoads = kStepBytes == 8 ? 2 : 1;
    const uint32_t srow = (uint32_t)(s.in / (STEPS * 32)) * kSize;      // bytes of a row
    const size_t sfirst = first * srow;
    const __amdgpu_buffer_rsrc_t sr =
        make_rsrc(static_cast<const char*>(a.w_scales) + (sfirst & ~(size_t)3),
                  ((uint32_t)(sfirst & 3) + (uint32_t)(SWIGLU ? half + left : left) * srow + 3) & ~3u);
    // bf16 holds every E2M1 code times a power of two, so its scale enters with the conversion.
    constexpr bool kFolded = E2M1 && !F16;

    const int lr = lane >> 3;
    const uint32_t lk = (uint32_t)((lane & 7) ^ lr) * 16;
    constexpr int kXLoads = 4 * MT / WAVES;                  // 2 halves of 2 * MT blocks of 8 rows
    uint32_t xoff[kXLoads];
    int xto[kXLoads];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i) {
        const int b = wave + i * WAVES;                 // block of 8 rows: half b / (2 MT)
        const int hb = b / (2 * MT), rb = b % (2 * MT);
        xto[i] = hb * MT * 2048 + rb * 1024;
        xoff[i] = (uint32_t)(rb * 8 + lr) * xrow + hb * 128 + lk;
    }
    // Codes: a load moves 16 rows of 64 bytes; lane i brings row i / 4 the 16 bytes of position
    // i % 4, which holds chunk (i % 4) ^ (row / 4 & 3).
    const int wr = lane >> 2;
    const uint32_t wk = (uint32_t)((lane & 3) ^ ((wr >> 2) & 3)) * 16;
    const uint32_t woff0 = (uint32_t)(wave * (SWIGLU ? 16 : 32) + wr) * wrow + wk;
    const uint32_t woff1 = SWIGLU ? woff0 : woff0 + 16 * wrow;
    // Byte of the resource where the scales of the wave's row r (0..31) begin.
    const auto scale_at = [&](int r) {
        const uint32_t row = SWIGLU ? (uint32_t)(wave * 16 + (r & 15)) + (r & 16 ? (uint32_t)half : 0u)
                                    : (uint32_t)(wave * 32 + r);
        return (uint32_t)(sfirst & 3) + row * srow;
    };
    const uint32_t sfetch = scale_at(lane & 31);
    const uint32_t suse[2] = {scale_at(l16), scale_at(16 + l16)};

    constexpr int kRing = w4_ring(MT);
    const auto fetch_x = [&](int step, int i) {
        const uint32_t k = (uint32_t)step * 256;
        // the offset within the row is below xrow (rows end inside a step)
        const int b = wave + i * WAVES;
        const bool past = k + (b / (2 * MT)) * 128 + lk >= xrow;
        load_lds16(xr, lds.x[step % kRing][0] + xto[i], past ? kRsrcPastEnd : xoff[i] + k);
    };
    const auto fetch_w = [&](int step) {
        const uint32_t k = (uint32_t)step * 64;
        const bool past = k + wk >= wrow;
        char* to = lds.w[wave][step % kRing];
        load_lds16(wr0, to, past ? kRsrcPastEnd : woff0 + k);
        load_lds16(SWIGLU ? wr1 : wr0, to + 1024, past ? kRsrcPastEnd : woff1 + k);
        const uint32_t d = (sfetch + (uint32_t)step * kStepBytes) & ~3u;
        char* st = reinterpret_cast<char*>(lds.s[wave][step % kRing]);
        load_lds4(sr, st, d + (lane >> 5) * 4);
        if constexpr (kSLoads == 2) load_lds4(sr, st + 256, d + 8);
    };

    // The codes and scales of a step, from LDS: of row l16 (t = 0) and row 16 + l16, the dword g
    // of chunk j for 32-element step j.
    uint32_t raw[2][4], sraw[2][3];
    const auto read_raw = [&](int step) {
        const char* wl = lds.w[wave][step % kRing] + l16 * 64 + g * 4;
        const uint32_t* st = lds.s[wave][step % kRing] + l16;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                raw[t][j] = *reinterpret_cast<const uint32_t*>(wl + t * 1024 + ((j ^ (l16 >> 2)) << 4));
            sraw[t][0] = st[t * 16];
            if (kStepBytes >= 4) sraw[t][1] = st[32 + t * 16];
            if (kStepBytes == 8) sraw[t][2] = st[64 + t * 16];
        }
    };
    float scale[2][2][kParts];
    const auto take_scale = [&](int par, int step) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint32_t at = suse[t] + (uint32_t)step * kStepBytes;
            uint32_t v[2];
            if constexpr (kStepBytes == 2) {
                v[0] = sraw[t][0] >> ((at & 2) * 8);
            } else {
                v[0] = __builtin_amdgcn_alignbyte(sraw[t][1], sraw[t][0], at & 3);
                if constexpr (kStepBytes == 8) v[1] = __builtin_amdgcn_alignbyte(sraw[t][2], sraw[t][1], at & 3);
            }
#pragma unroll
            for (int j = 0; j < kParts; ++j) {
                if constexpr (E2M1) {
                    const uint32_t b = (v[0] >> (8 * j)) & 255u;
                    scale[par][t][j] = __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
                } else {
                    const uint32_t b = (v[j / 2] >> (16 * (j & 1))) & 0xFFFFu;
                    scale[par][t][j] = F16 ? f16_lo(b) : bf16_lo(b);
                }
                // past the row's end its codes and rows of x are 0, and the scale must be finite
                if (step * kParts + j >= s.in / (STEPS * 32)) scale[par][t][j] = 0.0f;
            }
        }
    };
    v4i_t w[2][2][4];
    const auto decode_part = [&](int par, int j) {
#pragma unroll
        for (int t = 0; t < 2; ++t)
            w[par][t][j] = decode_tile<F16, E2M1>(raw[t][j], kFolded ? scale[par][t][j / STEPS] : 1.0f);
    };

    v4f_t acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = v4f_t{0, 0, 0, 0};
    const int f0 = l16 * 128 + ((g ^ (l16 & 7)) << 4);
    const int f1 = l16 * 128 + (((4 + g) ^ (l16 & 7)) << 4);

    // Before step 0: its codes decoded, the codes of step 1 in registers, every stage but one of
    // x and all places of codes filled or on their way.  In step k the place of x(k - 1) takes
    // x(k + ring - 1), and that of the codes of k + 1 (in registers) those of k + 1 + ring.
    constexpr int kStep = kXLoads + 2 + kSLoads;             // loads of a step
    const auto all_x = [&](int step) {
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) fetch_x(step, i);
    };
    fetch_w(0);
    fetch_w(1);
    all_x(0);
#pragma unroll
    for (int i = 2; i < kRing; ++i) {
        fetch_w(i);
        all_x(i - 1);
    }
    wait_loads<kXLoads + (kRing - 2) * kStep>();
    read_raw(0);
    take_scale(0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) decode_part(0, j);
    read_raw(1);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    fetch_w(kRing);

    const auto one = [&](int par, int step) {
        // x(step): issued after it are the rest of its step's loads, and ring - 2 whole steps
        wait_loads<2 + kSLoads + (kRing - 2) * kStep>();
        meet();
        const char* xl = lds.x[step % kRing][0];
        v4i_t x[2][4];
        const auto read_x = [&](int set, int m) {
            const char* p = xl + m * 2048;
            x[set][0] = *reinterpret_cast<const v4i_t*>(p + f0);
            x[set][1] = *reinterpret_cast<const v4i_t*>(p + f1);
            x[set][2] = *reinterpret_cast<const v4i_t*>(p + MT * 2048 + f0);
            x[set][3] = *reinterpret_cast<const v4i_t*>(p + MT * 2048 + f1);
        };
        read_x(0, 0);
        take_scale(par ^ 1, step + 1);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            if (m + 1 < MT) read_x((m + 1) & 1, m + 1);
#pragma unroll
            for (int i = 0; i < kXLoads; ++i)
                if (i * MT / kXLoads == m) fetch_x(step + kRing - 1, i);
            // (the place of step + 1's codes, which were read before this step's first rows, and
            // those have arrived by the time of the second rows)
            if (m == MT - 1) {
                if (MT == 1) asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                fetch_w(step + 1 + kRing);
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (j * MT / 4 == m) decode_part(par ^ 1, j);
            if constexpr (kFolded) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
#pragma unroll
                    for (int t = 0; t < 2; ++t) acc[m][t] = mma16<F16>(x[m & 1][j], w[par][t][j], acc[m][t]);
            } else {
                v4f_t sum[kParts][2];
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    sum[p][0] = sum[p][1] = v4f_t{0, 0, 0, 0};
#pragma unroll
                    for (int j = 0; j < STEPS; ++j)
#pragma unroll
                        for (int t = 0; t < 2; ++t)
                            sum[p][t] = mma16<F16>(x[m & 1][p * STEPS + j], w[par][t][p * STEPS + j], sum[p][t]);
                }
#pragma unroll
                for (int p = 0; p < kParts; ++p)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            acc[m][t][r] = __builtin_fmaf(sum[p][t][r], scale[par][t][p], acc[m][t][r]);
                // (keeps the additions here: postponed, the sums of all rows stay in registers)
                asm volatile("" : "+v"(acc[m][0]), "+v"(acc[m][1]));
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        // the codes of step + 2: issued after them are ring - 1 whole steps
        wait_loads<(kRing - 1) * kStep>();
        read_raw(step + 2);
    };
    int step = 0;
    for (; step + 2 <= steps; step += 2) {
        one(0, step);
        one(1, step + 1);
    }
    if (step < steps) one(0, step);
    wait_loads<0>();                            // nothing may land in LDS after the tile

    constexpr int kT = SWIGLU ? 1 : 2;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            const int c = wave * (kT * 16) + t * 16 + l16;
            constexpr float unit = kCodeUnit<F16, E2M1>;
            float y[4], u[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                y[r] = acc[m][t][r] * unit;
                u[r] = acc[m][1][r] * unit;
            }
            if (SWIGLU) silu_mul4(y, u, y);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = m * 16 + g * 4 + r;
                if (row < tile.rows && c < left)
                    static_cast<uint16_t*>(a.out)[(size_t)(tile.row0 + row) * half + tile.n0 + c] =
                        (uint16_t)pack_out2(y[r], 0.0f, F16);
            }
        }
}

template <bool F16, bool E2M1, int STEPS, bool SWIGLU>
__global__ __launch_bounds__(kTileThreads, 2) void w4_tile_kernel(MatmulShape s, MatmulArgs a)
{
    __shared__ W4Lds lds;
    Tile t;
    if (!find_tile<kW4TileM, SWIGLU ? kW4TileN / 2 : kW4TileN>(s, a, SWIGLU ? s.out / 2 : s.out,
                                                               lds.table, &t))
        return;
    switch ((t.rows + 31) / 32) {
    case 1: w4_tile_product<F16, E2M1, STEPS, 2, SWIGLU, kTileWaves>(s, a, t, lds.s2); break;
    case 2: w4_tile_product<F16, E2M1, STEPS, 4, SWIGLU, kTileWaves>(s, a, t, lds.s4); break;
    case 3: w4_tile_product<F16, E2M1, STEPS, 6, SWIGLU, kTileWaves>(s, a, t, lds.s6); break;
    default: w4_tile_product<F16, E2M1, STEPS, 8, SWIGLU, kTileWaves>(s, a, t, lds.s8); break;
    }
}

template <bool F16, bool E2M1, int STEPS, bool SWIGLU>
__global__ __launch_bounds__(kW4SmallWaves * kWave, 2) void w4_small_kernel(MatmulShape s, MatmulArgs a)
{
    __shared__ W4SmallLds lds;
    Tile t;
    if (!find_tile<kW4SmallM, SWIGLU ? kW4SmallN / 2 : kW4SmallN, kW4SmallWaves>(
            s, a, SWIGLU ? s.out / 2 : s.out, lds.table, &t))
        return;
    if (t.rows <= 16)
        w4_tile_product<F16, E2M1, STEPS, 1, SWIGLU, kW4SmallWaves>(s, a, t, lds.s1);
    else
        w4_tile_product<F16, E2M1, STEPS, 2, SWIGLU, kW4SmallWaves>(s, a, t, lds.s2);
}

template <bool F16, bool E2M1, int STEPS>
hipError_t launch_w4_tile(const MatmulShape& s, const MatmulArgs& a, bool small, hipStream_t stream)
{
    const int rows = small ? kW4SmallM : kW4TileM, n = small ? kW4SmallN : kW4TileN;
    const dim3 grid(tile_grid(s, rows, s.swiglu ? n / 2 : n));
    if (small) {
        if (s.swiglu)
            w4_small_kernel<F16, E2M1, STEPS, true><<<grid, kW4SmallWaves * kWave, 0, stream>>>(s, a);
        else
            w4_small_kernel<F16, E2M1, STEPS, false><<<grid, kW4SmallWaves * kWave, 0, stream>>>(s, a);
    } else if (s.swiglu) {
        w4_tile_kernel<F16, E2M1, STEPS, true><<<grid, kTileThreads, 0, stream>>>(s, a);
    } else {
        w4_tile_kernel<F16, E2M1, STEPS, false><<<grid, kTileThreads, 0, stream>>>(s, a);
    }
    return hipGetLastError();
}

template <bool F16>
hipError_t launch_w4_tiles(const MatmulShape& s, const MatmulArgs& a, bool small, hipStream_t stream)
{
    if (s.w4 == MOE_W4_E2M1) return launch_w4_tile<F16, true, 1>(s, a, small, stream);
    if (s.group == 32) return launch_w4_tile<F16, false, 1>(s, a, small, stream);
    if (s.group == 64) return launch_w4_tile<F16, false, 2>(s, a, small, stream);
    return launch_w4_tile<F16, false, 4>(s, a, small, stream);
}

}  // namespace
}  // namespace moe_dc
