// grouped_matmul_coded.hip -- the experts' products on block-scaled fp8 rows, their results coded again.
#include "grouped_matmul_tile.h"

namespace moe_dc {
namespace {

template <int TYPE>
hipError_t launch_coded(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return product_path(s) == kPathThinTiles ? launch_thin_tiles<TYPE, true>(s, a, stream)
                                             : launch_tiles<TYPE, true>(s, a, stream);
}

}  // namespace

hipError_t launch_grouped_coded_e4m3(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_coded<kMmBlockE4m3>(s, a, stream);
}

hipError_t launch_grouped_coded_e5m2(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_coded<kMmBlockE5m2>(s, a, stream);
}

}  // namespace moe_dc
