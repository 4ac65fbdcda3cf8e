// grouped_matmul_block.hip -- the experts' products on fp8 rows with a scale per 128 elements and
// weights with a scale per 128 x 128 block.
#include "grouped_matmul.h"

namespace moe_dc {

hipError_t launch_grouped_block_e4m3(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmBlockE4m3>(s, a, stream);
}

hipError_t launch_grouped_block_e5m2(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmBlockE5m2>(s, a, stream);
}

}  // namespace moe_dc
