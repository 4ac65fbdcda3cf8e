// dc_quantize.h -- how values become codes and scales (modes 1 to 5), shared by the kernels that
// write 8-bit rows.
#pragma once
#include "dc_convert.h"

namespace moe_dc {
namespace {

constexpr int kGroup = 128;          // mode 3 group length

template <int CT>
__device__ __forceinline__ uint32_t fp8_code(float v)
{
    return CT == kCodeE4m3 ? e4m3_code(v) : CT == kCodeE5m2 ? e5m2_code(v) : e2m1_code(v);
}

// Largest finite value of a code type (dst_type_max / fp8_max of the formulas).
template <int CT>
constexpr float type_max()
{
    return CT == kCodeInt8 ? 127.0f : CT == kCodeE4m3 ? 448.0f : CT == kCodeE5m2 ? 57344.0f
                                                                                 : 6.0f;
}

// A per-128-group dynamic scale pair (mode 3): dyn = type_max / amax and scale = 1 / dyn, both
// correctly rounded, as the per-element division gives them.
template <int CT>
__device__ __forceinline__ void group_dyn(uint32_t amax_bits, float& dyn, float& scale)
{
    const float amax = __uint_as_float(amax_bits);
    if (CT == kCodeE4m3) dyn = div_rn<8>(448.0f, amax);
    else if (CT == kCodeE5m2) dyn = div_rn<15>(57344.0f, amax);
    else dyn = type_max<CT>() / amax;
    scale = div_rn<1>(1.0f, dyn);
}

// Shared exponent of an MX block from the bit pattern of its absolute maximum.
template <int MODE, int CT>
__device__ __forceinline__ int mx_shared_exp(uint32_t amax_bits)
{
    constexpr int emax = CT == kCodeE4m3 ? 8 : CT == kCodeE5m2 ? 15 : 2;
    if (MODE == 4) {
        if (amax_bits == 0) return -127;
        const int ex = (int)(amax_bits >> 23);
        const int fl = ex != 0 ? ex - 127 : (31 - __clz(amax_bits)) - 149;   // floor(log2)
        return fl - emax > -127 ? fl - emax : -127;
    } else {
        const float c = fmaxf(__uint_as_float(amax_bits), 1e-4f);
        const uint32_t vb = __float_as_uint(c / type_max<CT>());           // normal, > 0
        return (int)(vb >> 23) - 127 + ((vb & 0x7FFFFFu) != 0u ? 1 : 0);     // ceil(log2)
    }
}

// 2^e for e in [-127, 126] as a binary32 (2^-127 is the subnormal 0x00400000).
__device__ __forceinline__ float pow2f(int e)
{
    return e >= -126 ? __uint_as_float((uint32_t)(127 + e) << 23) : __uint_as_float(0x00400000u);
}

// Eight token elements of one 16-byte vector, widened to binary32 (exact): bf16, or
// binary16 when f16 is set (a wave-uniform flag).
__device__ __forceinline__ void unpack8(uint4 w, float (&f)[8], bool f16)
{
    if (f16) {
        f[0] = f16_lo(w.x); f[1] = f16_hi(w.x); f[2] = f16_lo(w.y); f[3] = f16_hi(w.y);
        f[4] = f16_lo(w.z); f[5] = f16_hi(w.z); f[6] = f16_lo(w.w); f[7] = f16_hi(w.w);
    } else {
        f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
        f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
    }
}

__device__ __forceinline__ void mul8(float (&f)[8], float4 a, float4 b)
{
    f[0] = f[0] * a.x; f[1] = f[1] * a.y; f[2] = f[2] * a.z; f[3] = f[3] * a.w;
    f[4] = f[4] * b.x; f[5] = f[5] * b.y; f[6] = f[6] * b.z; f[7] = f[7] * b.w;
}

__device__ __forceinline__ uint32_t absmax8(const float (&f)[8], uint32_t amax)
{
#pragma unroll
    for (int c = 0; c < 8; ++c) {
        const uint32_t bits = __float_as_uint(f[c]) & 0x7FFFFFFFu;
        amax = amax > bits ? amax : bits;
    }
    return amax;
}

// absmax8 for values that are products of a multiplication (canonical floats, never NaN for
// finite inputs): a float maximum of absolute values, which the compiler forms from max3
// instructions with absolute-value operand modifiers; for non-negative non-NaN floats the
// float order is the order of the bit patterns, so the result is absmax8's.
__device__ __forceinline__ uint32_t absmax8_products(const float (&f)[8], uint32_t amax)
{
    float m = __uint_as_float(amax);
#pragma unroll
    for (int c = 0; c < 8; ++c) m = __builtin_fmaxf(m, __builtin_fabsf(f[c]));
    return __float_as_uint(m);
}

__device__ __forceinline__ uint2 pack_codes8(const uint32_t (&c)[8])
{
    return make_uint2((c[0] & 0xFF) | ((c[1] & 0xFF) << 8) | ((c[2] & 0xFF) << 16) | (c[3] << 24),
                      (c[4] & 0xFF) | ((c[5] & 0xFF) << 8) | ((c[6] & 0xFF) << 16) | (c[7] << 24));
}

// Eight int8 codes of f * dyn for a finite dyn (dyn = 127 / amax with amax > 0 and not tiny):
// then |f * dyn| <= 127 * (1 + 2^-23), so no clamp is needed and no NaN can arise.  Adding
// 1.5 * 2^23 to the binary32 product puts the sum in [2^23, 2^24), where binary32 spacing is 1:
// the addition rounds the product to an integer, ties to even, and the low byte of the sum's
// bit pattern is that integer in two's complement.  Byte permutes gather the four low bytes.
__device__ __forceinline__ uint2 int8_codes8_finite(const float (&f)[8], float dyn)
{
    uint32_t b[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float v = f[q] * dyn;
        b[q] = __float_as_uint(v + 12582912.0f);
    }
    const uint32_t lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[3], b[2], 0x0c0c0400u),
                                              __builtin_amdgcn_perm(b[1], b[0], 0x0c0c0400u),
                                              0x05040100u);
    const uint32_t hi = __builtin_amdgcn_perm(__builtin_amdgcn_perm(b[7], b[6], 0x0c0c0400u),
                                              __builtin_amdgcn_perm(b[5], b[4], 0x0c0c0400u),
                                              0x05040100u);
    return make_uint2(lo, hi);
}

// Eight codes of the dynamic modes: type(f * dyn), NaN products -> 0.
template <int CT>
__device__ __forceinline__ uint2 dynamic_codes8(const float (&f)[8], float dyn)
{
    if (CT == kCodeInt8 && __float_as_uint(dyn) < 0x7F800000u)    // dyn > 0 here
        return int8_codes8_finite(f, dyn);
    if (CT == kCodeE4m3 || CT == kCodeE5m2) {
        float v[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            const float p = f[q] * dyn;
            v[q] = p != p ? 0.0f : p;                  // a NaN product's code is 0
        }
        return fp8_codes8_hw<CT>(v);
    }
    uint32_t c[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) {
        const float v = f[q] * dyn;
        if (CT == kCodeInt8) c[q] = int8_code(v);
        else c[q] = v != v ? 0u : fp8_code<CT>(v);
    }
    return pack_codes8(c);
}

// Eight static int8 codes (mode 1): the scales are already applied.
__device__ __forceinline__ uint2 static_codes8(const float (&f)[8])
{
    return static_int8_codes8(f);
}

}  // namespace
}  // namespace moe_dc
