// experts_internal.h -- launch interface of the router and the experts' products.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "dc_internal.h"

namespace moe_dc {

// Row and weight types of the products.  Row kinds (Int8, E4m3, E5m2) carry one fp32 scale per
// row and one per weight row; the MX kinds one E8M0 byte per 32 elements of each.
enum MmType : int32_t {
    kMmBf16 = 0, kMmF16 = 1, kMmInt8 = 2, kMmE4m3 = 3, kMmE5m2 = 4, kMmMxE4m3 = 5, kMmMxE5m2 = 6
};

// One validated product (see moe_matmul in include/moe_dc.h).
struct MatmulShape {
    int32_t W, E, L;
    int32_t in;              // inner size (elements of a row)
    int32_t out;             // weight rows per expert
    int32_t type;            // MmType
    int32_t swiglu;          // 1: out holds gate rows, then up rows; out/2 columns are written
    int32_t w4;              // 0, or moe_w4_dtype
    int32_t group;           // w4: elements per scale
    int32_t tok_f16;
    int64_t rows;            // W*BS*K, the most rows there can be
    int64_t cap;
};

struct MatmulArgs {
    const void* x;
    const void* x_scales;
    const void* w;
    const void* w_scales;
    const int32_t* ep_recv_count;
    const int64_t* recv_offsets;
    void* out;
};

// One per MmType.
hipError_t launch_grouped_bf16(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_f16(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_int8(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_e4m3(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_e5m2(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_mxe4m3(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_mxe5m2(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream);
hipError_t launch_grouped_matmul_w4(const MatmulShape& s, const MatmulArgs& a,
                                    hipStream_t stream);

// One validated router call (see moe_gate in include/moe_dc.h).
struct GateShape {
    int32_t tokens, n, K;
    int32_t sigmoid;
    int32_t groups, keep, top;
    int32_t renormalize;
    float factor;
    uint32_t group_magic;    // 2^21 / (n / groups) + 1

    // id / (n / groups) for id < n <= 2048: exact, since id * (n / groups) <= 2^21 with a group
    // limit
    __host__ __device__ int group_of(int id) const { return (int)(((uint32_t)id * group_magic) >> 21); }
};

hipError_t launch_gate_topk(const GateShape& s, const float* logits, const float* bias,
                            int32_t* expert_ids, float* expert_scales, hipStream_t stream);

}  // namespace moe_dc
