// grouped_matmul_w4.h -- 4-bit codes as operands of the 16-bit matrix instructions.
#pragma once

#include "experts_tiles.h"

namespace moe_dc {
namespace {

typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
typedef uint32_t u2_t __attribute__((ext_vector_type(2)));

// 4 x 4 transpose of dwords over the lane groups l / 16.
__device__ __forceinline__ v4i_t exchange(v4i_t v)
{
    const u2_t p = __builtin_amdgcn_permlane32_swap((uint32_t)v.x, (uint32_t)v.z, false, false);
    const u2_t q = __builtin_amdgcn_permlane32_swap((uint32_t)v.y, (uint32_t)v.w, false, false);
    const u2_t r = __builtin_amdgcn_permlane16_swap(p.x, q.x, false, false);
    const u2_t t = __builtin_amdgcn_permlane16_swap(p.y, q.y, false, false);
    return v4i_t{(int)r.x, (int)r.y, (int)t.x, (int)t.y};
}

// Eight codes of a dword as 16-bit floats.  int4: in the order 0 4 1 5 2 6 3 7 (see pair_order);
// for bf16 each is 136 + code.
template <bool F16, bool E2M1>
__device__ __forceinline__ v4i_t decode(uint32_t w)
{
    v4i_t r;
    if constexpr (E2M1) {
        if constexpr (F16) {
            r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
            r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
            r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
            r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
        } else {
            r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 0));
            r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 1));
            r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 2));
            r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f, 3));
        }
    } else {
        constexpr uint32_t magic = F16 ? 0x64086408u : 0x43084308u;   // the XOR makes code + 8
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) ^ magic;
            if constexpr (F16) {
                const h2_t off = {(_Float16)-1032.0f, (_Float16)-1032.0f};
                u = __builtin_bit_cast(uint32_t, __builtin_bit_cast(h2_t, u) + off);
            }
            r[i] = (int)u;
        }
    }
    return r;
}

// Eight 16-bit elements 0..7 in the order 0 4 1 5 2 6 3 7.
__device__ __forceinline__ v4i_t pair_order(v4i_t x)
{
    v4i_t r;
    r.x = (int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x05040100u);
    r.y = (int)__builtin_amdgcn_perm((uint32_t)x.z, (uint32_t)x.x, 0x07060302u);
    r.z = (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x05040100u);
    r.w = (int)__builtin_amdgcn_perm((uint32_t)x.w, (uint32_t)x.y, 0x07060302u);
    return r;
}

template <bool F16>
__device__ __forceinline__ v4f_t mma16(v4i_t a, v4i_t b, v4f_t c)
{
    if constexpr (F16)
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h_t, a),
                                                      __builtin_bit_cast(v8h_t, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_t, a),
                                                       __builtin_bit_cast(v8bf_t, b), c, 0, 0, 0);
}

}  // namespace
}  // namespace moe_dc
