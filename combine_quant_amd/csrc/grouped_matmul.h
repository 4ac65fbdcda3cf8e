// grouped_matmul.h -- which kernel takes a product, for one row type.
#pragma once

#include "grouped_matmul_stream.h"
#include "grouped_matmul_tile.h"

namespace moe_dc {
namespace {

constexpr int kTileMinRows = 24;                // mean rows per expert from which tiles are used
constexpr int kTileMinTiles = 192;              // and tiles enough for most of the 256 CUs

template <int TYPE>
hipError_t launch_type(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    const int64_t nt = ((int64_t)s.out + kTileN - 1) / kTileN;
    const int64_t mt = (s.rows / s.E + kTileM<TYPE> - 1) / kTileM<TYPE>;
    if (s.rows >= kTileMinRows * (int64_t)s.E && s.E * mt * nt >= kTileMinTiles)
        return launch_tiles<TYPE>(s, a, stream);
    return launch_stream<TYPE>(s, a, stream);
}

}  // namespace
}  // namespace moe_dc
