// grouped_matmul_fp8.hip -- the experts' products on row-scaled fp8 rows.
#include "grouped_matmul.h"

namespace moe_dc {

hipError_t launch_grouped_e4m3(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmE4m3>(s, a, stream);
}

hipError_t launch_grouped_e5m2(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmE5m2>(s, a, stream);
}

}  // namespace moe_dc
