// grouped_matmul_int8.hip -- the experts' products on int8 rows.
#include "grouped_matmul.h"

namespace moe_dc {

hipError_t launch_grouped_int8(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmInt8>(s, a, stream);
}

}  // namespace moe_dc
