// norm.hip -- RMS norm of the tokens, with the residual's addition before and codes behind.
//
//   s = x + residual (fp32), y = s / sqrt(mean(s^2) + epsilon) * gamma, codes of y
//
// The kernel reads every token once and holds it in registers: one workgroup per token, SLOTS
// vectors of eight elements a thread, so that a group of 128 is 16 adjacent lanes and an MX block 4.
// The sum of squares (and in mode 2 the largest value) meets in LDS.  Codes are formed from y before
// its rounding to the token type, by the functions dispatch uses.
//
// Bound by memory: 8192 tokens x 7168 with residual and a scale per 128 (530 MB) take 92 us, 5.8 TB/s (a
// large copy 4.9, a large read 6.2); by latency: 2 tokens 4.1 us (4.8 with sums by
// lane shuffles and a loop over the waves).
#include "dc_quantize.h"
#include "norm_internal.h"

#include <type_traits>

namespace moe_dc {
namespace {

__device__ __forceinline__ uint4 load16(__amdgpu_buffer_rsrc_t r, uint32_t off)
{
    const u32x4_t v = __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 0);
    return make_uint4(v.x, v.y, v.z, v.w);
}

// STREAM: past the caches.
template <bool STREAM>
__device__ __forceinline__ void store16(__amdgpu_buffer_rsrc_t r, uint32_t off, uint4 o)
{
    const u32x4_t v = {o.x, o.y, o.z, o.w};
    __builtin_amdgcn_raw_buffer_store_b128(v, r, (int)off, 0, STREAM ? kRsrcNonTemporal : 0);
}

template <bool STREAM>
__device__ __forceinline__ void store8(__amdgpu_buffer_rsrc_t r, uint32_t off, uint2 o)
{
    const u32x2_t v = {o.x, o.y};
    __builtin_amdgcn_raw_buffer_store_b64(v, r, (int)off, 0, STREAM ? kRsrcNonTemporal : 0);
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8], bool f16)
{
    return f16 ? make_uint4(pack_f16x2(f[0], f[1]), pack_f16x2(f[2], f[3]), pack_f16x2(f[4], f[5]),
                            pack_f16x2(f[6], f[7]))
               : make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                            pack_bf16x2(f[6], f[7]));
}

// The sum of a row of 16 lanes, in every lane of the row.
__device__ __forceinline__ float row_sum(float v)
{
    const auto moved = [&](auto pattern) {
        return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(pattern)::value, 0xF, 0xF, false));
    };
    v += moved(std::integral_constant<int, kDppQuadXor1>());
    v += moved(std::integral_constant<int, kDppQuadXor2>());
    v += moved(std::integral_constant<int, kDppRowHalfMirror>());
    v += moved(std::integral_constant<int, kDppRowMirror>());
    return v;
}

// The workgroup's sum, or largest value, in every thread: up to 64 rows of 16 lanes meet in
// `scratch` (64 words, those of rows that are not there cleared by the first wave).
__device__ __forceinline__ float block_sum(float v, float* scratch)
{
    const int lane = threadIdx.x & (kWave - 1);
    v = row_sum(v);
    if ((lane & 15) == 0) scratch[threadIdx.x / 16] = v;
    if (threadIdx.x < kWave && threadIdx.x >= blockDim.x / 16) scratch[threadIdx.x] = 0.0f;
    __syncthreads();
    v = row_sum(scratch[lane]);
    v += __shfl_xor(v, 16, kWave);
    return v + __shfl_xor(v, 32, kWave);
}
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* scratch)
{
    const int lane = threadIdx.x & (kWave - 1);
    v = group_max_u32<16>(v);
    if ((lane & 15) == 0) scratch[threadIdx.x / 16] = v;
    if (threadIdx.x < kWave && threadIdx.x >= blockDim.x / 16) scratch[threadIdx.x] = 0;
    __syncthreads();
    return group_max_u32<64>(scratch[lane]);
}

__device__ __forceinline__ float reciprocal_rms(const NormShape& s, float squares)
{
    return 1.0f / __builtin_sqrtf(squares / (float)s.H + s.epsilon);
}

// A dynamic scale pair from the largest value's bits, as dispatch forms it; the scale of values with an
// infinity or NaN among them is NaN (dyn is 0 or NaN then, and with it every code).
template <int CT>
__device__ __forceinline__ void dynamic_scale(uint32_t peak, float& dyn, float& scale)
{
    group_dyn<CT>(peak, dyn, scale);
    if (peak >= 0x7F800000u) scale = NAN;
}

// Shared exponent of an MX block, 0 where it holds an infinity or NaN.
template <int MODE, int CT>
__device__ __forceinline__ int shared_exp(uint32_t peak)
{
    return peak < 0x7F800000u ? mx_shared_exp<MODE, CT>(peak) : 0;
}

__device__ __forceinline__ float inverse_power(int e) { return __uint_as_float((uint32_t)(127 - e) << 23); }

// The scale of an MX block as the config stores it; `bad`: the block holds an infinity or NaN.
__device__ __forceinline__ void store_mx_scale(const NormShape& s, void* scales, size_t at, int e, bool bad)
{
    if (s.scale_format == MOE_SCALE_E8M0)
        static_cast<uint8_t*>(scales)[at] = bad ? 0xFFu : (uint8_t)(e + 127);
    else
        static_cast<float*>(scales)[at] = bad ? NAN : s.scale_format == MOE_SCALE_FP32 ? pow2f(e)
                                                                                             : inverse_power(e);
}

template <int MODE, int CT, int SLOTS, bool STREAM>
__global__ __launch_bounds__(1024) void norm_kernel(NormShape s, NormArgs a)
{
    __shared__ float sums[kWave];
    __shared__ uint32_t peaks[kWave];
    const size_t token = blockIdx.x;
    const uint32_t row = (uint32_t)s.H * 2;
    const bool f16 = s.tok_f16;
    const auto rsrc = [&](const void* p, uint32_t bytes) {
        return make_rsrc(static_cast<const char*>(p) + token * bytes, bytes);
    };
    const __amdgpu_buffer_rsrc_t xr = rsrc(a.x, row), gr = make_rsrc(a.gamma, row);
    // (an absent residual is a resource of no bytes: zeros)
    const __amdgpu_buffer_rsrc_t rr = a.residual ? rsrc(a.residual, row) : make_rsrc(a.x, 0);
    uint4 xv[SLOTS], rv[SLOTS], gv[SLOTS];
    uint32_t at[SLOTS];
#pragma unroll
    for (int n = 0; n < SLOTS; ++n) {
        at[n] = (threadIdx.x + n * blockDim.x) * 16;
        xv[n] = load16(xr, at[n]);
        rv[n] = load16(rr, at[n]);
        gv[n] = load16(gr, at[n]);
    }
    float f[SLOTS][8];
    float squares = 0.0f;
#pragma unroll
    for (int n = 0; n < SLOTS; ++n) {
        float r[8];
        unpack8(xv[n], f[n], f16);
        unpack8(rv[n], r, f16);
        float part = 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            if (a.residual) f[n][q] = f[n][q] + r[q];
            part += f[n][q] * f[n][q];
        }
        squares += part;
    }
    squares = block_sum(squares, sums);
    if (a.residual_out) {
        const __amdgpu_buffer_rsrc_t so = rsrc(a.residual_out, row);
#pragma unroll
        for (int n = 0; n < SLOTS; ++n) store16<STREAM>(so, at[n], pack8(f[n], f16));
    }
    const float rms = reciprocal_rms(s, squares);
#pragma unroll
    for (int n = 0; n < SLOTS; ++n) {
        float g[8];
        unpack8(gv[n], g, f16);
#pragma unroll
        for (int q = 0; q < 8; ++q) f[n][q] = f[n][q] * rms * g[q];
    }
    if (a.y) {
        const __amdgpu_buffer_rsrc_t yo = rsrc(a.y, row);
#pragma unroll
        for (int n = 0; n < SLOTS; ++n) store16<STREAM>(yo, at[n], pack8(f[n], f16));
    }
    if (MODE == 0) return;

    // vectors past the row's end hold zeros (gamma is read as 0 there), or NaN where the row's
    // reciprocal is infinite or NaN; they are left out of the largest values
    const __amdgpu_buffer_rsrc_t co = rsrc(a.codes, (uint32_t)s.H);
    uint32_t most[SLOTS];
#pragma unroll
    for (int n = 0; n < SLOTS; ++n) most[n] = at[n] < row ? absmax8(f[n], 0u) : 0u;
    if (MODE == 2) {
        uint32_t peak = most[0];
#pragma unroll
        for (int n = 1; n < SLOTS; ++n) peak = dpp_max(peak, most[n]);
        peak = block_max(peak, peaks);
        float dyn, scale;
        dynamic_scale<CT>(peak, dyn, scale);
#pragma unroll
        for (int n = 0; n < SLOTS; ++n) store8<STREAM>(co, at[n] / 2, dynamic_codes8<CT>(f[n], dyn));
        if (threadIdx.x == 0) static_cast<float*>(a.scales)[token] = scale;
    } else if (MODE == 3) {
#pragma unroll
        for (int n = 0; n < SLOTS; ++n) {
            const uint32_t peak = group_max_u32<kGroup / 8>(most[n]);
            float dyn, scale;
            dynamic_scale<CT>(peak, dyn, scale);
            store8<STREAM>(co, at[n] / 2, dynamic_codes8<CT>(f[n], dyn));
            if ((threadIdx.x & (kGroup / 8 - 1)) == 0 && at[n] < row)
                static_cast<float*>(a.scales)[token * s.scales_per_row + at[n] / (2 * kGroup)] = scale;
        }
    } else if (MODE >= 4) {
#pragma unroll
        for (int n = 0; n < SLOTS; ++n) {
            const uint32_t peak = group_max_u32<kMxBlock / 8>(most[n]);
            const int e = shared_exp<MODE, CT>(peak);
            store8<STREAM>(co, at[n] / 2, dynamic_codes8<CT>(f[n], inverse_power(e)));
            if ((threadIdx.x & (kMxBlock / 8 - 1)) == 0 && at[n] < row)
                store_mx_scale(s, a.scales, token * s.scales_per_row + at[n] / (2 * kMxBlock), e,
                               peak >= 0x7F800000u);
        }
        // the pad entry of an odd number of blocks
        if (threadIdx.x == 0 && (s.H + kMxBlock - 1) / kMxBlock < s.scales_per_row) {
            const size_t pad = token * s.scales_per_row + s.scales_per_row - 1;
            if (s.scale_format == MOE_SCALE_E8M0) static_cast<uint8_t*>(a.scales)[pad] = 0;
            else static_cast<float*>(a.scales)[pad] = 0.0f;
        }
    }
}

// Any H and any alignment: y of the token in LDS, element by element, and a thread per group of codes, which
// walks it alone: what no vector takes, as in dispatch's element-wise kernel, and not made fast.  8192
// tokens x 7161, modes 0, 2, 3 and 4: 334, 356, 649 and 519 us (7168: 68, 78, 78 and 79 on inputs that the
// last cache holds in part); 2 tokens x 1025, mode 3: 29 us.
constexpr int kAnyThreads = 256;

template <int MODE, int CT>
__global__ __launch_bounds__(kAnyThreads) void norm_any_kernel(NormShape s, NormArgs a)
{
    __shared__ float y[8192];
    __shared__ float sums[kWave];
    __shared__ uint32_t peaks[kWave];
    const size_t token = blockIdx.x, base = token * s.H;
    const bool f16 = s.tok_f16;
    const auto value = [&](const void* p, size_t i) { return tok_lo_rt(static_cast<const uint16_t*>(p)[i], f16); };
    float squares = 0.0f;
    for (int i = threadIdx.x; i < s.H; i += kAnyThreads) {
        float v = value(a.x, base + i);
        if (a.residual) v = v + value(a.residual, base + i);
        y[i] = v;
        squares += v * v;
    }
    squares = block_sum(squares, sums);
    const float rms = reciprocal_rms(s, squares);
    uint32_t peak = 0;
    for (int i = threadIdx.x; i < s.H; i += kAnyThreads) {
        if (a.residual_out) static_cast<uint16_t*>(a.residual_out)[base + i] = (uint16_t)f32_to_tok_rt(y[i], f16);
        const float v = y[i] * rms * value(a.gamma, i);
        y[i] = v;
        peak = dpp_max(peak, __float_as_uint(v) & 0x7FFFFFFFu);
        if (a.y) static_cast<uint16_t*>(a.y)[base + i] = (uint16_t)f32_to_tok_rt(v, f16);
    }
    if (MODE == 0) return;
    __syncthreads();
    uint8_t* codes = static_cast<uint8_t*>(a.codes) + base;
    const auto code = [&](int i, float by) {
        const float p = y[i] * by;
        codes[i] = CT == kCodeInt8 ? (uint8_t)int8_code(p) : p != p ? (uint8_t)0 : (uint8_t)fp8_code<CT>(p);
    };
    if (MODE == 2) {
        peak = block_max(peak, peaks);
        float dyn, scale;
        dynamic_scale<CT>(peak, dyn, scale);
        for (int i = threadIdx.x; i < s.H; i += kAnyThreads) code(i, dyn);
        if (threadIdx.x == 0) static_cast<float*>(a.scales)[token] = scale;
        return;
    }
    constexpr int kSpan = MODE == 3 ? kGroup : kMxBlock;
    for (int b = threadIdx.x; b < s.scales_per_row; b += kAnyThreads) {
        const int lo = b * kSpan, hi = lo + kSpan < s.H ? lo + kSpan : s.H;
        const size_t at = token * s.scales_per_row + b;
        uint32_t most = 0;
        for (int i = lo; i < hi; ++i) most = dpp_max(most, __float_as_uint(y[i]) & 0x7FFFFFFFu);
        if (MODE == 3) {
            float dyn, scale;
            dynamic_scale<CT>(most, dyn, scale);
            for (int i = lo; i < hi; ++i) code(i, dyn);
            static_cast<float*>(a.scales)[at] = scale;
        } else if (lo >= s.H) {
            if (s.scale_format == MOE_SCALE_E8M0) static_cast<uint8_t*>(a.scales)[at] = 0;
            else static_cast<float*>(a.scales)[at] = 0.0f;
        } else {
            const int e = shared_exp<MODE, CT>(most);
            for (int i = lo; i < hi; ++i) code(i, inverse_power(e));
            store_mx_scale(s, a.scales, at, e, most >= 0x7F800000u);
        }
    }
}

// Few tokens: as many threads as vectors, many: two vectors a thread.  One and two, us, H = 7168: 2 tokens
// 4.1 and 4.7, 512 8.3 and 8.6, 1024 14.4 and 13.1, 8192 102 and 95.
constexpr int kManyTokens = 1024;
// Elements from which the outputs pass the caches by: they would push out what is read next.  Norm,
// logits and dispatch after each other with and without, us: 8192 tokens x 7168 198 and 202, 8192 x 2048
// 73 and 77, but 1024 x 7168 55.5 and 53.6 (the norm alone: 92 and 95, 24.3 and 31.9, 11.7 and 13.1).
constexpr int64_t kStreamElements = 12 << 20;

template <int MODE, int CT>
hipError_t launch(const NormShape& s, const NormArgs& a, bool vectorized, hipStream_t stream)
{
    const dim3 grid((unsigned)s.tokens);
    if (!vectorized) {
        norm_any_kernel<MODE, CT><<<grid, kAnyThreads, 0, stream>>>(s, a);
        return hipGetLastError();
    }
    const int vectors = s.H / 8;
    const int threads = ((s.tokens < kManyTokens ? vectors : (vectors + 1) / 2) + kWave - 1) / kWave * kWave;
    if (s.tokens < kManyTokens)
        norm_kernel<MODE, CT, 1, false><<<grid, threads, 0, stream>>>(s, a);
    else if ((int64_t)s.tokens * s.H < kStreamElements)
        norm_kernel<MODE, CT, 2, false><<<grid, threads, 0, stream>>>(s, a);
    else
        norm_kernel<MODE, CT, 2, true><<<grid, threads, 0, stream>>>(s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_rms_norm(const NormShape& s, const NormArgs& a, bool vectorized, hipStream_t stream)
{
    switch (s.quant_mode * 8 + (s.quant_mode ? s.code_type : 0)) {
    case 0: return launch<0, kCodeBf16>(s, a, vectorized, stream);
    case 2 * 8 + kCodeInt8: return launch<2, kCodeInt8>(s, a, vectorized, stream);
    case 2 * 8 + kCodeE4m3: return launch<2, kCodeE4m3>(s, a, vectorized, stream);
    case 2 * 8 + kCodeE5m2: return launch<2, kCodeE5m2>(s, a, vectorized, stream);
    case 3 * 8 + kCodeE4m3: return launch<3, kCodeE4m3>(s, a, vectorized, stream);
    case 3 * 8 + kCodeE5m2: return launch<3, kCodeE5m2>(s, a, vectorized, stream);
    case 4 * 8 + kCodeE4m3: return launch<4, kCodeE4m3>(s, a, vectorized, stream);
    case 4 * 8 + kCodeE5m2: return launch<4, kCodeE5m2>(s, a, vectorized, stream);
    case 5 * 8 + kCodeE4m3: return launch<5, kCodeE4m3>(s, a, vectorized, stream);
    default: return launch<5, kCodeE5m2>(s, a, vectorized, stream);
    }
}

}  // namespace moe_dc
