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

// Fewer tiles leave CUs idle, more the streaming kernel's narrow column blocks use.  bf16, inner
// size 4096, 8 experts: 32 tiles 29.7 us against 21.8 by streaming (8 rows an expert), 44.5
// against 38.7 (64 rows); 64 tiles 29.7 against 34.9, 45.7 against 73.1.
constexpr int kTileLeast = 56;

// The same for 4-bit weights.  int4, inner size 4096, 8 experts: with 8 rows an expert 128 small
// tiles take 18.0 us against 16.3 by streaming, 256 19.6 against 28.0; with 64 rows 64 tiles 58.7
// against 51.4, 128 60.0 against 93.1.
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
