// gate_math.h -- the router's exponentials, for the device and (for a check of their error) the
// host.
#pragma once

#include <hip/hip_runtime.h>

namespace moe_dc {

// 2^t for t <= 0, relative error below 2^-24.8: Taylor series of (2^f - 1) / f to the sixth power
// for |f| <= 1/2 (remainder 5.2e-9 of the result) in binary32, the rest in binary64.  (The product
// with f and f itself rounded to binary32 would double the error: 2^-24.0.)
__host__ __device__ __forceinline__ double exp2_fine(double t)
{
    const double r = __builtin_rint(t);
    const double f = t - r;
    const float g = (float)f;
    float p = 1.525273380e-5f;                            // ln2^7 / 7!
    p = __builtin_fmaf(p, g, 1.540353039e-4f);
    p = __builtin_fmaf(p, g, 1.333355815e-3f);
    p = __builtin_fmaf(p, g, 9.618129108e-3f);
    p = __builtin_fmaf(p, g, 5.550410866e-2f);
    p = __builtin_fmaf(p, g, 2.402265070e-1f);
    p = __builtin_fmaf(p, g, 6.931471806e-1f);
    return t < -1100.0 ? 0.0 : __builtin_ldexp(__builtin_fma((double)p, f, 1.0), (int)r);
}

// e^x for x <= 0 (or NaN) to about an ulp: x = k ln 2 + f, Taylor series of e^f to the 13th power
// for |f| <= ln(2) / 2 (remainder 4.2e-18).
__host__ __device__ __forceinline__ double exp_below(double x)
{
    const double k = __builtin_rint(x * 1.4426950408889634);
    double f = __builtin_fma(-k, 0.6931471805599453, x);
    f = __builtin_fma(-k, 2.3190468138462996e-17, f);     // ln 2 less its binary64 value
    double p = 1.0 / 6227020800.0;
    p = __builtin_fma(p, f, 1.0 / 479001600.0);
    p = __builtin_fma(p, f, 1.0 / 39916800.0);
    p = __builtin_fma(p, f, 1.0 / 3628800.0);
    p = __builtin_fma(p, f, 1.0 / 362880.0);
    p = __builtin_fma(p, f, 1.0 / 40320.0);
    p = __builtin_fma(p, f, 1.0 / 5040.0);
    p = __builtin_fma(p, f, 1.0 / 720.0);
    p = __builtin_fma(p, f, 1.0 / 120.0);
    p = __builtin_fma(p, f, 1.0 / 24.0);
    p = __builtin_fma(p, f, 1.0 / 6.0);
    p = __builtin_fma(p, f, 0.5);
    p = __builtin_fma(p, f, 1.0);
    p = __builtin_fma(p, f, 1.0);
    return x < -760.0 ? 0.0 : __builtin_ldexp(p, (int)k);
}

}  // namespace moe_dc
