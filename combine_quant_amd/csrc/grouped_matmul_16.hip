// grouped_matmul_16.hip -- the experts' products on bf16 and fp16 rows.
#include "grouped_matmul.h"

namespace moe_dc {

hipError_t launch_grouped_bf16(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmBf16>(s, a, stream);
}

hipError_t launch_grouped_f16(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return launch_type<kMmF16>(s, a, stream);
}

}  // namespace moe_dc
