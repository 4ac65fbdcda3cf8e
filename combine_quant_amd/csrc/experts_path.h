// experts_path.h -- which kernel takes a product: a rule on its sizes and types alone, known on
// the host before the launch.
#pragma once

#include "experts_internal.h"

namespace moe_dc {

enum ProductPath : int32_t {
    kPathStream = 0,            // 32 weight rows a workgroup, memory to registers
    kPathTiles = 1,             // 256 weight rows a workgroup, through LDS
    kPathSmallTiles = 2         // 128 weight rows, 4-bit weights only
};

constexpr int kTileN = 256;                     // weight rows of a workgroup
// Most rows of x of a workgroup: as many as the 160 KB of LDS take (MX keeps scales there too).
constexpr int tile_rows(int type) { return type == kMmMxE4m3 || type == kMmMxE5m2 ? 192 : 256; }

constexpr int kW4TileM = 128;                   // rows of x and weight rows of a workgroup
constexpr int kW4TileN = 256;
constexpr int kW4SmallM = 32;                   // and of the smaller one, two to a CU
constexpr int kW4SmallN = 128;

// Fewer tiles leave CUs idle, more the streaming kernel's narrow column blocks use.  Tiles against
// streaming in us, 8 experts, inner size 2048 (7168):
//   64 rows an expert, 32 tiles: bf16 20.1 and 15.2 (55.9 and 41.6), E4M3 12.8 and 11.2 (31.3 and
//     24.3), MX 13.9 and 12.3 (35.8 and 32.2); 48 tiles: bf16 20.4 and 26.8 (56.4 and 78.9), E4M3
//     12.9 and 17.9 (31.8 and 43.7), MX 14.2 and 21.5 (36.6 and 60.4)
//   8 rows, 56 tiles: bf16 16.5 and 15.0 (48 and 37), E4M3 9.6 and 9.4 (27 and 22), MX 10.1 and 11.1
//     (31 and 30); 80 tiles: bf16 16.9 and 21.2 (82 and 59), E4M3 11.1 and 17.1 (28 and 34), MX
//     11.4 and 15.1 (32 and 43)
// int8 is as E4M3.  The one number serves all but long bf16 rows on few rows an expert, which
// streaming would serve better up to about 100 tiles.
constexpr int kTileLeast = 56;

// The same for 4-bit weights, 8 experts, inner size 2048 (7168).
//   8 rows an expert, 128 small tiles: int4 11.5 and 8.8 us (30 and 20), E2M1 11.5 and 13.6 (31 and
//     47); 160: int4 11.5 and 12.4 (30 and 32), E2M1 11.5 and 21.8 (31 and 89)
//   64 rows, 64 tiles: int4 22.4 and 22.0 (63 and 62), E2M1 21.6 and 27.3 (61 and 86); 80: int4 22.6
//     and 30.7 (63 and 90), E2M1 21.7 and 41.8 (61 and 133)
constexpr int kSmallLeast = 144;
constexpr int kW4TileLeast = 80;

// Whether there are at least `least` tiles of `height` rows and `cols` columns, in the mean over
// the experts that can have rows.
inline bool tiles_suffice(const MatmulShape& s, int height, int cols, int least)
{
    const int64_t half = s.swiglu ? s.out / 2 : s.out;
    const int64_t active = s.rows < s.E ? s.rows : s.E;
    if (active == 0) return false;
    return active * ((s.rows / active + height - 1) / height) * ((half + cols - 1) / cols) >= least;
}

inline ProductPath product_path(const MatmulShape& s)
{
    const int part = s.swiglu ? 2 : 1;
    if (!s.w4)
        return tiles_suffice(s, tile_rows(s.type), kTileN / part, kTileLeast) ? kPathTiles : kPathStream;
    // few rows per expert: the smaller tiles, where they are enough
    const int64_t active = s.rows < s.E ? s.rows : s.E;
    if (s.rows <= kW4SmallM * active && tiles_suffice(s, kW4SmallM, kW4SmallN / part, kSmallLeast))
        return kPathSmallTiles;
    return tiles_suffice(s, kW4TileM, kW4TileN / part, kW4TileLeast) ? kPathTiles : kPathStream;
}

}  // namespace moe_dc
