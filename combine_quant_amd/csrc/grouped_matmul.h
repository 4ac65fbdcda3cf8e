// grouped_matmul.h -- which kernel takes a product, for one row type.
#pragma once

#include "grouped_matmul_stream.h"
#include "grouped_matmul_tile.h"

namespace moe_dc {
namespace {

template <int TYPE>
hipError_t launch_type(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return product_path(s) == kPathTiles ? launch_tiles<TYPE>(s, a, stream) : launch_stream<TYPE>(s, a, stream);
}

}  // namespace
}  // namespace moe_dc
