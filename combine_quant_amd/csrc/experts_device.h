// experts_device.h -- device helpers of the experts' products: the rows of an expert, buffer
// loads of operand chunks, and the matrix instructions of every row type.
#pragma once

#include <type_traits>

#include "dc_device.h"
#include "experts_internal.h"

namespace moe_dc {

typedef int v4i_t __attribute__((ext_vector_type(4)));
typedef int v8i_t __attribute__((ext_vector_type(8)));
typedef float v4f_t __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf_t __attribute__((ext_vector_type(8)));
typedef _Float16 v8h_t __attribute__((ext_vector_type(8)));

// First row past expert e (experts are packed one after another, so it is also the first row of
// expert e + 1).  Held within [0, cap] whatever the tensors hold.
__device__ __forceinline__ int expert_end(const MatmulShape& s, const int32_t* recv_count,
                                          const int64_t* recv_offsets, int e)
{
    if (e < 0) return 0;
    const int r = e / s.L, j = e - r * s.L;
    const int64_t end = recv_offsets[r] + recv_count[(size_t)r * s.L * s.W + (size_t)(j + 1) * s.W - 1];
    return (int)(end < 0 ? 0 : end > s.cap ? s.cap : end);
}

__device__ __forceinline__ v4i_t load_chunk(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
    return __builtin_bit_cast(v4i_t, v);
}

// Row types.  All products walk rows in chunks of 128 bytes; lane l of a wave holds, of row l %
// 16, the 16 bytes at (l / 16) * 16 and the 16 bytes at 64 + (l / 16) * 16 of the chunk, which is
// the operand layout of every instruction used here (two of K = 32 for 16-bit types, two of K =
// 64 for int8, one of K = 128 for fp8).  The result of A (16 weight rows) times B (16 rows of x)
// has, in lane l, row l % 16 of x and weight rows (l / 16) * 4 + 0..3.
template <int TYPE>
struct Mm {
    static constexpr bool kMx = TYPE == kMmMxE4m3 || TYPE == kMmMxE5m2;
    static constexpr bool kRowScaled = TYPE == kMmInt8 || TYPE == kMmE4m3 || TYPE == kMmE5m2;
    static constexpr bool kInt = TYPE == kMmInt8;
    static constexpr bool kF16Out = TYPE == kMmF16;
    static constexpr int kBytes = TYPE == kMmBf16 || TYPE == kMmF16 ? 2 : 1;
    typedef typename std::conditional<kInt, v4i_t, v4f_t>::type Acc;

    // acc += A chunk * B chunk; sa, sb: the chunk's E8M0 bytes of the lane's 32-element block
    // l / 16 (MX only).
    static __device__ __forceinline__ Acc mma(v8i_t a, v8i_t b, Acc acc, int sa, int sb)
    {
        const v4i_t a0 = __builtin_shufflevector(a, a, 0, 1, 2, 3);
        const v4i_t a1 = __builtin_shufflevector(a, a, 4, 5, 6, 7);
        const v4i_t b0 = __builtin_shufflevector(b, b, 0, 1, 2, 3);
        const v4i_t b1 = __builtin_shufflevector(b, b, 4, 5, 6, 7);
        if constexpr (TYPE == kMmBf16) {
            acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_t, a0),
                                                          __builtin_bit_cast(v8bf_t, b0), acc, 0, 0, 0);
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_t, a1),
                                                           __builtin_bit_cast(v8bf_t, b1), acc, 0, 0, 0);
        } else if constexpr (TYPE == kMmF16) {
            acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h_t, a0),
                                                         __builtin_bit_cast(v8h_t, b0), acc, 0, 0, 0);
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h_t, a1),
                                                          __builtin_bit_cast(v8h_t, b1), acc, 0, 0, 0);
        } else if constexpr (TYPE == kMmInt8) {
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a0, b0, acc, 0, 0, 0);
            return __builtin_amdgcn_mfma_i32_16x16x64_i8(a1, b1, acc, 0, 0, 0);
        } else {
            // weights are E4M3 (format 0); x is E4M3 or E5M2 (format 1).  Row-scaled codes run
            // with block scales of 2^0, for the rate of 128 elements an instruction; it cuts each
            // product at 2^-13 of the power of two of the largest of eight before its fp32 sum,
            // 5 bits below the half step of a bf16 result.
            constexpr int fx = TYPE == kMmE5m2 || TYPE == kMmMxE5m2 ? 1 : 0;
            if constexpr (!kMx) sa = sb = 127;
            return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 0, fx, 0, sa, 0, sb);
        }
    }
};

// The two halves of a lane's chunk as one operand.
__device__ __forceinline__ v8i_t join(v4i_t lo, v4i_t hi)
{
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
}

// Two fp32 values as a pair of tokens, rounded to nearest even by the conversion instructions.
__device__ __forceinline__ uint32_t pack_out2(float lo, float hi, bool f16)
{
    typedef __bf16 b2_t __attribute__((ext_vector_type(2)));
    typedef _Float16 h2_t __attribute__((ext_vector_type(2)));
    const b2_t b = {(__bf16)lo, (__bf16)hi};
    const h2_t h = {(_Float16)lo, (_Float16)hi};
    return f16 ? __builtin_bit_cast(uint32_t, h) : __builtin_bit_cast(uint32_t, b);
}

// silu(t) * u = t * u / (1 + exp(-t)).  Below t = -87 exp(-t) leaves the range of binary32, and the
// quotient, that of its normal numbers, while times u it need not: numerator and denominator are
// then both multiplied by 2^-126, and u by the numerator, which reaches to t = -176.
__device__ __forceinline__ float silu_mul(float t, float u, bool low)
{
    const float e = __builtin_amdgcn_exp2f(__builtin_fmaf(t, -1.44269504f, low ? -126.0f : 0.0f));
    const float num = low ? t * 0x1p-126f * u : t;
    const float q = num / (low ? e : 1.0f + e);
    return low ? q : q * u;
}

// y = silu(t) * u of four values.  The scaled form only where a lane of the wave needs it (its
// selects cost a 192 x 256 tile of 56 steps 1 %); a value is the same either way.
__device__ __forceinline__ void silu_mul4(const float (&t)[4], const float (&u)[4], float (&y)[4])
{
    constexpr float edge = -87.0f;
    const float least = fminf(fminf(t[0], t[1]), fminf(t[2], t[3]));
    if (__ballot(least < edge) == 0) {
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = silu_mul(t[q], u[q], false);
    } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) y[q] = silu_mul(t[q], u[q], t[q] < edge);
    }
}

}  // namespace moe_dc
