// grouped_matmul_mx.hip -- the experts' products on MX fp8 rows.
#include "grouped_matmul.h"

namespace moe_dc {

hipError_t launch_grouped_mxe4m3(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmMxE4m3>(s, a, stream);
}

hipError_t launch_grouped_mxe5m2(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmMxE5m2>(s, a, stream);
}

}  // namespace moe_dc
