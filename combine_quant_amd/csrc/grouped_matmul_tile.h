// grouped_matmul_tile.h -- the experts' products for many rows per expert.
#pragma once

#include "experts_device.h"

namespace moe_dc {
namespace {

constexpr int kTileWaves = 8;
constexpr int kTileThreads = kTileWaves * kWave;
constexpr int kTileN = 256;                     // weight rows of a workgroup
constexpr int kTileM = 256;                     // most rows of x of a workgroup
constexpr int kTileScales = (kTileN + kTileM) * 4;
constexpr int kMaxExperts = 1024;
constexpr int kGroupM = 8;                      // row tiles that share a sweep over the weights

struct TileLds {
    char x[2][kTileM * 128];                    // [row][128 bytes], swizzled
    char w[2][kTileN * 128];
    char scales[2][kTileScales];                // MX: four E8M0 bytes a row of x, then weights
    int cum[kMaxExperts + 1];                   // tiles before each expert
    int wave_sum[kTileWaves];
};

__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)lds, 16, (int)off, 0, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t r, char* lds, uint32_t off)
{
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)lds, 4, (int)off, 0, 0, 0);
}

// One tile: 32 * MS rows of x from row0 (of which `rows` exist), 256 weight rows from column n0.
// Wave w: row half w / 4 (16 * MS rows), weight rows 64 * (w % 4) + 0..63 of the tile.
template <int TYPE, int MS, bool SWIGLU>
__device__ __forceinline__ void tile_product(const MatmulShape& s, const MatmulArgs& a, int e,
                                             int n0, int row0, int rows, TileLds& lds)
{
    typedef Mm<TYPE> M;
    typedef typename M::Acc Acc;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    const int wn = wave & 3, wm = wave >> 2;
    const uint32_t row_bytes = (uint32_t)s.in * M::kBytes;
    const int steps = (int)((row_bytes + 127) / 128);
    const int half = SWIGLU ? s.out / 2 : s.out;
    constexpr int kCols = SWIGLU ? kTileN / 2 : kTileN;      // columns of the output
    const int left = half - n0 < kCols ? half - n0 : kCols;
    const char* wbase = static_cast<const char*>(a.w) + ((size_t)e * s.out + n0) * row_bytes;
    const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(wbase, (uint32_t)left * row_bytes);
    const __amdgpu_buffer_rsrc_t wr1 =
        make_rsrc(wbase + (size_t)half * row_bytes, (uint32_t)left * row_bytes);
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(static_cast<const char*>(a.x) + (size_t)row0 * row_bytes, (uint32_t)rows * row_bytes);
    const uint32_t ns = (uint32_t)s.in / 32;
    const char* wsb = static_cast<const char*>(a.w_scales) + ((size_t)e * s.out + n0) * ns;
    const __amdgpu_buffer_rsrc_t ws0 = make_rsrc(wsb, M::kMx ? (uint32_t)left * ns : 0);
    const __amdgpu_buffer_rsrc_t ws1 =
        make_rsrc(wsb + (size_t)half * ns, M::kMx ? (uint32_t)left * ns : 0);
    const __amdgpu_buffer_rsrc_t xs =
        make_rsrc(static_cast<const char*>(a.x_scales) + (size_t)row0 * ns,
                  M::kMx ? (uint32_t)rows * ns : 0);

    // Staging: one instruction moves 8 rows of 128 bytes; lane i brings row i / 8 the 16 bytes
    // that belong at position i % 8, which holds chunk (i % 8) ^ (row & 7).
    const int lr = lane >> 3;
    const uint32_t lk = (uint32_t)((lane & 7) ^ lr) * 16;
    constexpr int kXLoads = (4 * MS + kTileWaves - 1) / kTileWaves;
    uint32_t xoff[kXLoads], woff[4];
#pragma unroll
    for (int i = 0; i < kXLoads; ++i)
        xoff[i] = (uint32_t)((wave + i * kTileWaves) * 8 + lr) * row_bytes + lk;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // weight row block wave + 8 * i of 32; with SwiGLU each 64 rows hold 32 gate, 32 up
        const int blk = wave + i * kTileWaves;
        const int r = SWIGLU ? (blk >> 3) * 32 + (blk & 3) * 8 : blk * 8;
        woff[i] = (uint32_t)(r + lr) * row_bytes + lk;
    }
    const auto stage_x = [&](int step) {
        const uint32_t k = (uint32_t)step * 128;
        char* xl = lds.x[step & 1];
        const bool past = k + lk >= row_bytes;
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            const int blk = wave + i * kTileWaves;
            if ((4 * MS) % kTileWaves == 0 || blk < 4 * MS)
                load_lds16(xr, xl + blk * 1024, past ? kRsrcPastEnd : xoff[i] + k);
        }
        if (M::kMx) {
            // 64 rows of four bytes per instruction: waves 0-3 the weights, 4-7 the rows of x
            char* sl = lds.scales[step & 1];
            if (wave < 4) {
                const int up = SWIGLU && lane >= 32;
                const int r = SWIGLU ? wave * 32 + (lane & 31) : wave * 64 + lane;
                if (!up) load_lds4(ws0, sl + 1024 + wave * 256, (uint32_t)r * ns + step * 4);
                if (up) load_lds4(ws1, sl + 1024 + wave * 256, (uint32_t)r * ns + step * 4);
            } else if ((wave - 4) * 2 < MS) {
                load_lds4(xs, sl + (wave - 4) * 256,
                          (uint32_t)((wave - 4) * 64 + lane) * ns + step * 4);
            }
        }
    };
    const auto stage_w = [&](int step) {
        const uint32_t k = (uint32_t)step * 128;
        char* wl = lds.w[step & 1];
        const bool past = k + lk >= row_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int blk = wave + i * kTileWaves;
            load_lds16(SWIGLU && (blk & 4) ? wr1 : wr0, wl + blk * 1024,
                       past ? kRsrcPastEnd : woff[i] + k);
        }
    };

    Acc acc[MS][4];
#pragma unroll
    for (int m = 0; m < MS; ++m)
#pragma unroll
        for (int t = 0; t < 4; ++t) acc[m][t] = Acc{0, 0, 0, 0};
    const int f0 = l16 * 128 + ((g ^ (l16 & 7)) << 4);
    const int f1 = l16 * 128 + (((4 + g) ^ (l16 & 7)) << 4);

    stage_x(0);
    stage_w(0);
    for (int step = 0; step < steps; ++step) {
        const int b = step & 1;
        __syncthreads();                        // this step's operands are in LDS
        if (step + 1 < steps) {
            stage_x(step + 1);
            stage_w(step + 1);
        }
        const char* xl = lds.x[b] + wm * MS * 2048;
        const char* wl = lds.w[b] + wn * 8192;
        v4i_t w0[4], w1[4];
        int sa[4] = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            w0[t] = *reinterpret_cast<const v4i_t*>(wl + t * 2048 + f0);
            w1[t] = *reinterpret_cast<const v4i_t*>(wl + t * 2048 + f1);
            if (M::kMx)
                sa[t] = *reinterpret_cast<const uint8_t*>(lds.scales[b] + 1024 +
                                                          (wn * 64 + t * 16 + l16) * 4 + g);
        }
#pragma unroll
        for (int m = 0; m < MS; ++m) {
            const v4i_t x0 = *reinterpret_cast<const v4i_t*>(xl + m * 2048 + f0);
            const v4i_t x1 = *reinterpret_cast<const v4i_t*>(xl + m * 2048 + f1);
            int sb = 0;
            if (M::kMx)
                sb = *reinterpret_cast<const uint8_t*>(lds.scales[b] +
                                                       ((wm * MS + m) * 16 + l16) * 4 + g);
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[m][t] = M::mma(w0[t], w1[t], x0, x1, acc[m][t], sa[t], sb);
        }
    }

    constexpr int kT = SWIGLU ? 2 : 4;
    const int c0 = wn * (kT * 16) + g * 4;      // the lane's first column of sub-tile 0
#pragma unroll
    for (int m = 0; m < MS; ++m) {
        const int row = (wm * MS + m) * 16 + l16;
        if (row >= rows) continue;
        float rs = 1.0f;
        if (M::kRowScaled && a.x_scales) rs = static_cast<const float*>(a.x_scales)[row0 + row];
        uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)(row0 + row) * half + n0;
#pragma unroll
        for (int t = 0; t < kT; ++t) {
            const int c = c0 + t * 16;
            float y[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                float r = (float)acc[m][t][q], u = 0.0f;
                if (SWIGLU) u = (float)acc[m][(t + kT) & 3][q];
                if (M::kRowScaled && c + q < left) {
                    const float* sc = static_cast<const float*>(a.w_scales) + (size_t)e * s.out + n0 + c + q;
                    r = r * sc[0] * rs;
                    if (SWIGLU) u = u * sc[half] * rs;
                }
                y[q] = SWIGLU ? silu(r) * u : r;
            }
            const uint2 p = make_uint2(pack_out2(y[0], y[1], s.tok_f16), pack_out2(y[2], y[3], s.tok_f16));
            if (c + 3 < left && half % 4 == 0) {
                *reinterpret_cast<uint2*>(o + c) = p;
            } else {
                if (c < left) o[c] = (uint16_t)p.x;
                if (c + 1 < left) o[c + 1] = (uint16_t)(p.x >> 16);
                if (c + 2 < left) o[c + 2] = (uint16_t)p.y;
                if (c + 3 < left) o[c + 3] = (uint16_t)(p.y >> 16);
            }
        }
    }
}

// Every workgroup counts the tiles of all experts (ragged counts live on the device), then
// finds its own.  An expert's rows are cut into as few tiles of at most 256 rows as possible,
// all of nearly the same height.  Consecutive tiles go to one XCD (workgroups are dealt to the
// XCDs in turn), so that the tiles of an expert share its weights in that XCD's L2.
template <int TYPE, bool SWIGLU>
__global__ __launch_bounds__(kTileThreads, 2) void tile_kernel(MatmulShape s, MatmulArgs a)
{
    __shared__ TileLds lds;
    const int half = SWIGLU ? s.out / 2 : s.out;
    constexpr int kCols = SWIGLU ? kTileN / 2 : kTileN;
    const int nt = (half + kCols - 1) / kCols;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;

    // experts 2 * thread and 2 * thread + 1
    const int e0 = threadIdx.x * 2;
    int t0 = 0, t1 = 0;
    if (e0 < s.E) {
        const int b = expert_end(s, a.ep_recv_count, a.recv_offsets, e0 - 1);
        const int m = expert_end(s, a.ep_recv_count, a.recv_offsets, e0);
        t0 = m > b ? (m - b + kTileM - 1) / kTileM * nt : 0;
        if (e0 + 1 < s.E) {
            const int f = expert_end(s, a.ep_recv_count, a.recv_offsets, e0 + 1);
            t1 = f > m ? (f - m + kTileM - 1) / kTileM * nt : 0;
        }
    }
    int sum = t0 + t1;
#pragma unroll
    for (int off = 1; off < kWave; off <<= 1) {
        const int o = __shfl_up(sum, off, kWave);
        if (lane >= off) sum += o;
    }
    if (lane == kWave - 1) lds.wave_sum[wave] = sum;
    __syncthreads();
    for (int w = 0; w < wave; ++w) sum += lds.wave_sum[w];
    if (e0 < s.E) lds.cum[e0 + 1] = sum - t1;
    if (e0 + 1 < s.E) lds.cum[e0 + 2] = sum;
    if (threadIdx.x == 0) lds.cum[0] = 0;
    __syncthreads();

    const int total = lds.cum[s.E];
    const int chunk = (total + 7) / 8;
    const int slot = blockIdx.x >> 3;
    const int tile = (int)(blockIdx.x & 7) * chunk + slot;
    if (slot >= chunk || tile >= total) return;
    int lo = 0, hi = s.E;                       // cum[lo] <= tile < cum[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (lds.cum[mid] <= tile) lo = mid; else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    const int idx = __builtin_amdgcn_readfirstlane(tile - lds.cum[lo]);
    const int begin = expert_end(s, a.ep_recv_count, a.recv_offsets, e - 1);
    const int count = expert_end(s, a.ep_recv_count, a.recv_offsets, e) - begin;
    const int mt = (count + kTileM - 1) / kTileM;
    const int height = ((count + mt - 1) / mt + 31) / 32 * 32;
    const int band = idx / (kGroupM * nt), in_band = idx - band * kGroupM * nt;
    const int bm = mt - band * kGroupM < kGroupM ? mt - band * kGroupM : kGroupM;
    const int n0 = in_band / bm * kCols;
    const int r0 = (band * kGroupM + in_band % bm) * height;
    const int rows = count - r0 < height ? count - r0 : height;
    if (rows <= 0) return;
    switch ((rows + 31) / 32) {
    case 1: tile_product<TYPE, 1, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    case 2: tile_product<TYPE, 2, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    case 3: tile_product<TYPE, 3, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    case 4: tile_product<TYPE, 4, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    case 5: tile_product<TYPE, 5, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    case 6: tile_product<TYPE, 6, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    case 7: tile_product<TYPE, 7, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    default: tile_product<TYPE, 8, SWIGLU>(s, a, e, n0, begin + r0, rows, lds); break;
    }
}

template <int TYPE>
hipError_t launch_tiles(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    const int64_t half = s.swiglu ? s.out / 2 : s.out;
    const int64_t cols = s.swiglu ? kTileN / 2 : kTileN;
    const int64_t active = s.rows < s.E ? s.rows : s.E;
    const int64_t tiles = (s.rows / kTileM + active) * ((half + cols - 1) / cols);
    const dim3 grid((unsigned)((tiles + 7) / 8 * 8));
    if (s.swiglu)
        tile_kernel<TYPE, true><<<grid, kTileThreads, 0, stream>>>(s, a);
    else
        tile_kernel<TYPE, false><<<grid, kTileThreads, 0, stream>>>(s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace moe_dc
