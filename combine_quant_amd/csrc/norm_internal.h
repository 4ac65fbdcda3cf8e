// norm_internal.h -- launch interface of the RMS norm.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "dc_internal.h"

namespace moe_dc {

// One validated norm (see moe_norm in include/moe_dc.h).
struct NormShape {
    int32_t tokens, H;
    int32_t tok_f16;
    int32_t quant_mode, code_type, scale_format, scales_per_row;     // as in Shape
    float epsilon;
};

struct NormArgs {
    const void* x;
    const void* residual;        // null: none
    const void* gamma;
    void* residual_out;          // null: not wanted
    void* y;                     // null: not wanted
    void* codes;                 // null in mode 0
    void* scales;
};

// vectorized: H is a multiple of 8 and every pointer 16-byte aligned.
hipError_t launch_rms_norm(const NormShape& s, const NormArgs& a, bool vectorized, hipStream_t stream);

}  // namespace moe_dc
