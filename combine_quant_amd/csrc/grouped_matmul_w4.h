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

// int4 codes reach bf16 as sixteenths, so their sums are formed in sixteenths too.
template <bool F16, bool E2M1>
constexpr float kCodeUnit = !F16 && !E2M1 ? 16.0f : 1.0f;

// code / 16 of the low four bits of byte B.  (From the builtin the compiler makes a shift for every
// second byte: 56.2 us instead of 53.5 for 16 rows on 16 of 64 experts x 7168 x 4096.)
template <int B>
__device__ __forceinline__ float sixteenth(uint32_t w)
{
    float f;
    if constexpr (B == 0) asm("v_cvt_off_f32_i4 %0, %1" : "=v"(f) : "v"(w));
#define MOE_DC_CVT_I4(byte)                                                                    \
    asm("v_cvt_off_f32_i4_sdwa %0, %1 dst_sel:DWORD dst_unused:UNUSED_PAD src0_sel:" byte     \
        : "=v"(f) : "v"(w))
    if constexpr (B == 1) MOE_DC_CVT_I4("BYTE_1");
    if constexpr (B == 2) MOE_DC_CVT_I4("BYTE_2");
    if constexpr (B == 3) MOE_DC_CVT_I4("BYTE_3");
#undef MOE_DC_CVT_I4
    return f;
}
__device__ __forceinline__ int pack_bf16(float lo, float hi)
{
    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
    const b2_t p = {(__bf16)lo, (__bf16)hi};
    return __builtin_bit_cast(int, p);
}

// Eight codes of a dword as 16-bit floats, each exactly code / kCodeUnit, in their order; int4 for
// fp16 in the order 0 4 1 5 2 6 3 7 (see pair_order).  scale (E2M1 for bf16 only): a power of two
// that multiplies them.
//
// int4 for bf16 takes 13 instructions: eight v_cvt_off_f32_i4, and a packed conversion for every
// two of their results.  (As 136 + code, four bits under an exponent of 2^7, it takes 8, but the
// surplus then has to leave the fp32 sums again, which keeps neither a code of 0 at 0 nor rows
// near the type's largest value finite; that took 52 us at the size above.  Through E4M3 bytes it
// takes 21.)
template <bool F16, bool E2M1>
__device__ __forceinline__ v4i_t decode(uint32_t w, float scale = 1.0f)
{
    v4i_t r;
    if constexpr (E2M1 && F16) {
        r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
        r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
        r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
        r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
    } else if constexpr (E2M1) {
        r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
        r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
        r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
        r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
    } else if constexpr (F16) {
        const h2_t off = {(_Float16)-1032.0f, (_Float16)-1032.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {                        // the XOR makes code + 8, below 2^10
            const uint32_t u = ((w >> (4 * i)) & 0x000F000Fu) ^ 0x64086408u;
            r[i] = (int)__builtin_bit_cast(uint32_t, __builtin_bit_cast(h2_t, u) + off);
        }
    } else {
        const uint32_t v = w >> 4;
        r.x = pack_bf16(sixteenth<0>(w), sixteenth<0>(v));
        r.y = pack_bf16(sixteenth<1>(w), sixteenth<1>(v));
        r.z = pack_bf16(sixteenth<2>(w), sixteenth<2>(v));
        r.w = pack_bf16(sixteenth<3>(w), sixteenth<3>(v));
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
