// grouped_matmul.h -- which kernel takes a product, for one row type.
#pragma once

#include "grouped_matmul_stream.h"
#include "grouped_matmul_tile.h"

namespace moe_dc {
namespace {

// Fewer tiles leave CUs idle, more the streaming kernel's narrow column blocks use.  bf16, inner
// size 4096, 8 experts: 32 tiles 29.7 us against 21.8 by streaming (8 rows an expert), 44.5
// against 38.7 (64 rows); 64 tiles 29.7 against 34.9, 45.7 against 73.1.
constexpr int kTileLeast = 56;

template <int TYPE>
hipError_t launch_type(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    if (tiles_suffice(s, kTileM<TYPE>, s.swiglu ? kTileN / 2 : kTileN, kTileLeast))
        return launch_tiles<TYPE>(s, a, stream);
    return launch_stream<TYPE>(s, a, stream);
}

}  // namespace
}  // namespace moe_dc
