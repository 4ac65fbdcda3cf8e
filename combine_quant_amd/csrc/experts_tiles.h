// experts_tiles.h -- tiles of the experts' products: how ragged rows are cut and dealt out, and
// loads that move their data to LDS by themselves.
#pragma once

#include "experts_device.h"
#include "experts_path.h"

namespace moe_dc {
namespace {

constexpr int kTileWaves = 8;
constexpr int kTileThreads = kTileWaves * kWave;
constexpr int kMaxExperts = 1024;
constexpr int kWaveExperts = 128;               // most experts a wave counts by itself
constexpr int kGroupM = 8;                      // row tiles that share a sweep over the weights

struct TileTable {
    int cum[kMaxExperts + 1];                   // tiles before each expert
    int wave_sum[kTileWaves];
};

struct Tile {
    int e;                                      // expert
    int n0;                                     // first output column
    int row0, rows;                             // rows of x
};

// Workgroups that suffice for any counts of s.rows rows (tiles of `height` rows, `cols` columns).
inline unsigned tile_grid(const MatmulShape& s, int height, int cols)
{
    const int64_t half = s.swiglu ? s.out / 2 : s.out;
    const int64_t active = s.rows < s.E ? s.rows : s.E;
    const int64_t tiles = (s.rows / height + active) * ((half + cols - 1) / cols);
    return (unsigned)((tiles + 7) / 8 * 8);
}

// The place of this workgroup among `total` tiles, or -1.  Workgroup b runs on XCD b % 8.  Each
// XCD takes 32 consecutive tiles (one per CU) at a time, so that the tiles of an expert share its
// weights and its rows in that XCD's L2 while experts with many and with few rows are spread over
// the XCDs; the last tiles are shared out evenly.
__device__ __forceinline__ int tile_of_workgroup(int total)
{
    const int xcd = blockIdx.x & 7, slot = blockIdx.x >> 3;
    const int full = total / 256, rest = total % 256;
    if (slot < full * 32) return (slot / 32) * 256 + xcd * 32 + slot % 32;
    const int share = (rest + 7) / 8, r = slot - full * 32;
    return r < share && xcd * share + r < rest ? full * 256 + xcd * share + r : -1;
}

// The workgroup's tile.  The ragged counts live on the device, so every workgroup counts the
// tiles of all experts, then finds its own: for up to 128 experts each wave by itself (lane l
// counts experts l * per + 0..per - 1; 71 -> 65 us at 32 experts, 512 rows x 2048 x 7168 int4),
// for more the workgroup's threads together through LDS (228 -> 201 us at 1024 experts, 4096 rows
// x 2048 x 512 E4M3).  An expert's rows are cut into as few tiles of at most ROWS rows as
// possible, all of nearly the same height (a multiple of 16).
template <int ROWS, int COLS, int WAVES = kTileWaves>
__device__ __forceinline__ bool find_tile(const MatmulShape& s, const MatmulArgs& a, int columns,
                                          TileTable& table, Tile* out)
{
    const int nt = (columns + COLS - 1) / COLS;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    int e, idx, begin, count;
    if (s.E <= kWaveExperts) {
        constexpr int kMaxPer = kWaveExperts / kWave;
        const int per = (s.E + kWave - 1) / kWave;
        const int e0 = lane * per;
        int end[kMaxPer];
#pragma unroll
        for (int i = 0; i < kMaxPer; ++i)
            if (i < per) end[i] = expert_end(s, a.ep_recv_count, a.recv_offsets, e0 + i < s.E ? e0 + i : s.E - 1);
        const int start = expert_end(s, a.ep_recv_count, a.recv_offsets, (e0 < s.E ? e0 : s.E) - 1);
        int sum = 0, from = start;
#pragma unroll
        for (int i = 0; i < kMaxPer; ++i)
            if (i < per) {
                if (end[i] > from) sum += (end[i] - from + ROWS - 1) / ROWS * nt;
                from = end[i];
            }
        int upto = sum;
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int o = __shfl_up(upto, off, kWave);
            if (lane >= off) upto += o;
        }
        const int total = lane_value(upto, kWave - 1);
        const int tile = tile_of_workgroup(total);
        if (tile < 0) return false;
        const uint64_t holds = __ballot(upto > tile && upto - sum <= tile);
        const int src = __ffsll((unsigned long long)holds) - 1;
        int rest = tile - (upto - sum), found = -1, first = 0, rows = 0;
        from = start;
#pragma unroll
        for (int i = 0; i < kMaxPer; ++i)
            if (i < per) {
                const int c = end[i] > from ? (end[i] - from + ROWS - 1) / ROWS * nt : 0;
                if (found < 0 && rest < c) {
                    found = e0 + i;
                    first = from;
                    rows = end[i] - from;
                } else if (found < 0) {
                    rest -= c;
                }
                from = end[i];
            }
        e = __builtin_amdgcn_readlane(found, src);
        idx = __builtin_amdgcn_readlane(rest, src);
        begin = __builtin_amdgcn_readlane(first, src);
        count = __builtin_amdgcn_readlane(rows, src);
    } else {
        // kPer experts per thread
        constexpr int kPer = kMaxExperts / (WAVES * kWave);
        const int e0 = threadIdx.x * kPer;
        int tiles[kPer];
        int sum = 0;
        int from = e0 < s.E ? expert_end(s, a.ep_recv_count, a.recv_offsets, e0 - 1) : 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int end = e0 + i < s.E ? expert_end(s, a.ep_recv_count, a.recv_offsets, e0 + i) : from;
            tiles[i] = end > from ? (end - from + ROWS - 1) / ROWS * nt : 0;
            sum += tiles[i];
            from = end;
        }
#pragma unroll
        for (int off = 1; off < kWave; off <<= 1) {
            const int o = __shfl_up(sum, off, kWave);
            if (lane >= off) sum += o;
        }
        if (lane == kWave - 1) table.wave_sum[wave] = sum;
        __syncthreads();
        for (int w = 0; w < wave; ++w) sum += table.wave_sum[w];
#pragma unroll
        for (int i = kPer - 1; i >= 0; --i) {
            if (e0 + i < s.E) table.cum[e0 + i + 1] = sum;
            sum -= tiles[i];
        }
        if (threadIdx.x == 0) table.cum[0] = 0;
        __syncthreads();

        const int total = table.cum[s.E];
        const int tile = tile_of_workgroup(total);
        if (tile < 0) return false;
        int lo = 0, hi = s.E;                       // cum[lo] <= tile < cum[hi]
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (table.cum[mid] <= tile) lo = mid; else hi = mid;
        }
        e = __builtin_amdgcn_readfirstlane(lo);
        idx = __builtin_amdgcn_readfirstlane(tile - table.cum[lo]);
        __syncthreads();                            // the table's LDS is free again
        begin = expert_end(s, a.ep_recv_count, a.recv_offsets, e - 1);
        count = expert_end(s, a.ep_recv_count, a.recv_offsets, e) - begin;
    }
    const int mt = (count + ROWS - 1) / ROWS;
    const int height = ((count + mt - 1) / mt + 15) / 16 * 16;
    const int band = idx / (kGroupM * nt), in_band = idx - band * kGroupM * nt;
    const int bm = mt - band * kGroupM < kGroupM ? mt - band * kGroupM : kGroupM;
    const int r0 = (band * kGroupM + in_band % bm) * height;
    out->e = e;
    out->n0 = in_band / bm * COLS;
    out->row0 = begin + r0;
    out->rows = count - r0 < height ? count - r0 : height;
    return out->rows > 0;
}

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

// Four tokens to columns c..c+3 of a row, of which `left` are the tile's (rows begin at any
// token).
__device__ __forceinline__ void store_columns(uint16_t* row, int c, int left, uint2 p)
{
    if (c + 3 < left && (reinterpret_cast<uintptr_t>(row + c) & 7) == 0) {
        *reinterpret_cast<uint2*>(row + c) = p;
    } else {
        if (c < left) row[c] = (uint16_t)p.x;
        if (c + 1 < left) row[c + 1] = (uint16_t)(p.x >> 16);
        if (c + 2 < left) row[c + 2] = (uint16_t)p.y;
        if (c + 3 < left) row[c + 3] = (uint16_t)(p.y >> 16);
    }
}

// A workgroup barrier that leaves loads on their way: what other waves' loads put into LDS is
// there for those that each wave has waited for (wait_loads) before it.
__device__ __forceinline__ void meet()
{
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");              // no LDS access moves above it
}

// Waits until at most N of the wave's global loads are outstanding (they return in order).
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(N) : "memory");
}

}  // namespace
}  // namespace moe_dc
