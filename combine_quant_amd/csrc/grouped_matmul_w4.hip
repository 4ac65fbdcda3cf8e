// grouped_matmul_w4.hip -- products of the packed token rows with 4-bit expert weights.
//
// A workgroup takes NT * 16 weight rows of one expert; its four waves take chunks of 128
// elements (64 bytes of codes) in turn, straight from global memory.  Lane l loads, of weight row
// l % 16, the 16 bytes that hold elements (l / 16) * 32 + 0..31 of the chunk; a 4 x 4 exchange
// of dwords between the four lane groups then leaves in dword j the lane's eight elements of
// 32-element step j, the operand layout of the 16x16x32 instructions.
//
// Codes become 16-bit floats exactly (decode).  x is the A operand (rows of the result), the
// weights B (columns), so that one lane holds one weight row's results and one scale: each
// group's sum is formed by itself in fp32, scaled and added in fp32.
#include "grouped_matmul_w4.h"
#include "grouped_matmul_w4_tile.h"

namespace moe_dc {
namespace {

constexpr int kW4Waves = 4;
constexpr int kW4MaxZ = 8;

// STEPS: 32-element steps per scale (1, 2 or 4).
template <bool F16, bool E2M1, int STEPS, int MT, int NT>
__device__ __forceinline__ void w4_tile(const MatmulShape& s, const MatmulArgs& a, int e, int n0,
                                        int row0, int rows, float* lds)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t xrow = (uint32_t)s.in * 2, wrow = (uint32_t)s.in / 2;
    const int chunks = (s.in + 127) / 128;
    const int half = s.swiglu ? s.out / 2 : s.out;
    const int per = s.swiglu ? NT / 2 * 16 : NT * 16;
    const int left = half - n0 < per ? half - n0 : per;
    const int mrows = rows < MT * 16 ? rows : MT * 16;
    const char* wbase = static_cast<const char*>(a.w) + ((size_t)e * s.out + n0) * wrow;
    const __amdgpu_buffer_rsrc_t wr0 = make_rsrc(wbase, (uint32_t)left * wrow);
    const __amdgpu_buffer_rsrc_t wr1 =
        make_rsrc(wbase + (size_t)half * wrow, (uint32_t)left * wrow);
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(static_cast<const char*>(a.x) + (size_t)row0 * xrow, (uint32_t)mrows * xrow);
    const int ns = s.in / (STEPS * 32);                     // scales per weight row
    const size_t srow = (size_t)e * s.out + n0;

    v4f_t acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = v4f_t{0, 0, 0, 0};
    v4i_t wv[NT], xv[MT][4];
    float sc[NT][4 / STEPS];
    const auto fetch = [&](int c) {
        const uint32_t kw = (uint32_t)c * 64 + g * 16;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int part = s.swiglu ? t / (NT / 2) : 0;
            const int rt = s.swiglu ? t % (NT / 2) : t;
            wv[t] = load_chunk(part ? wr1 : wr0,
                               kw < wrow ? (uint32_t)(rt * 16 + l16) * wrow + kw : kRsrcPastEnd);
            const int n = rt * 16 + l16 < left ? rt * 16 + l16 : left - 1;
            const size_t so = (srow + (size_t)part * half + n) * ns;
#pragma unroll
            for (int j = 0; j < 4 / STEPS; ++j) {
                const int gi = c * (4 / STEPS) + j < ns ? c * (4 / STEPS) + j : ns - 1;
                if constexpr (E2M1) {
                    // 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 NaN
                    const uint32_t b = static_cast<const uint8_t*>(a.w_scales)[so + gi];
                    sc[t][j] = __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
                } else {
                    const uint32_t b = static_cast<const uint16_t*>(a.w_scales)[so + gi];
                    sc[t][j] = F16 ? f16_lo(b) : bf16_lo(b);
                }
                // past the row's end the sum is 0, and its scale must be finite
                if (c * (4 / STEPS) + j >= ns) sc[t][j] = 0.0f;
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t kx = (uint32_t)c * 256 + j * 64 + g * 16;
                xv[m][j] = load_chunk(xr, kx < xrow ? (uint32_t)(m * 16 + l16) * xrow + kx : kRsrcPastEnd);
            }
    };
    for (int c = wave; c < chunks; c += kW4Waves) {
        fetch(c);
#pragma unroll
        for (int t = 0; t < NT; ++t) wv[t] = exchange(wv[t]);
#pragma unroll
        for (int j = 0; j < 4 / STEPS; ++j) {
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                v4i_t xo[STEPS];
#pragma unroll
                for (int i = 0; i < STEPS; ++i)
                    xo[i] = F16 && !E2M1 ? pair_order(xv[m][j * STEPS + i]) : xv[m][j * STEPS + i];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    v4f_t p = {0, 0, 0, 0};
#pragma unroll
                    for (int i = 0; i < STEPS; ++i)
                        p = mma16<F16>(xo[i], decode<F16, E2M1>((uint32_t)wv[t][j * STEPS + i]), p);
#pragma unroll
                    for (int q = 0; q < 4; ++q) acc[m][t][q] = __builtin_fmaf(p[q], sc[t][j], acc[m][t][q]);
                }
            }
        }
    }

    v4f_t* part = reinterpret_cast<v4f_t*>(lds);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[((wave * MT + m) * NT + t) * kWave + lane] = acc[m][t];
    __syncthreads();
    const int nt = s.swiglu ? NT / 2 : NT;
    for (int i = wave; i < MT * nt; i += kW4Waves) {
        const int m = i / nt, t = i - m * nt;
        v4f_t r = part[(m * NT + t) * kWave + lane], u = r;
#pragma unroll
        for (int w = 1; w < kW4Waves; ++w) r += part[((w * MT + m) * NT + t) * kWave + lane];
        if (s.swiglu) {
            u = part[(m * NT + t + nt) * kWave + lane];
#pragma unroll
            for (int w = 1; w < kW4Waves; ++w) u += part[((w * MT + m) * NT + t + nt) * kWave + lane];
        }
        constexpr float unit = kCodeUnit<F16, E2M1>;
        const int n = t * 16 + l16;
        r *= unit;
        u *= unit;
        float y[4] = {r[0], r[1], r[2], r[3]};
        const float up[4] = {u[0], u[1], u[2], u[3]};
        if (s.swiglu) silu_mul4(y, up, y);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int row = m * 16 + g * 4 + q;
            if (row < mrows && n < left)
                static_cast<uint16_t*>(a.out)[(size_t)(row0 + row) * half + n0 + n] =
                    (uint16_t)f32_to_tok_rt(y[q], F16);
        }
    }
    __syncthreads();
}

template <bool F16, bool E2M1, int STEPS>
__global__ __launch_bounds__(kW4Waves * kWave) void w4_kernel(MatmulShape s, MatmulArgs a)
{
    constexpr int NT = 2, MT = 4;
    __shared__ float lds[kW4Waves * MT * NT * kWave * 4];
    const int half = s.swiglu ? s.out / 2 : s.out;
    const int per = s.swiglu ? NT / 2 * 16 : NT * 16;
    const int e = blockIdx.y;
    const int begin = expert_end(s, a.ep_recv_count, a.recv_offsets, e - 1);
    const int end = expert_end(s, a.ep_recv_count, a.recv_offsets, e);
    for (int n0 = blockIdx.x * per; n0 < half; n0 += gridDim.x * per) {
        for (int row = begin + blockIdx.z * MT * 16; row < end; row += gridDim.z * MT * 16) {
            const int rows = end - row;
            if (rows <= 16)
                w4_tile<F16, E2M1, STEPS, 1, NT>(s, a, e, n0, row, rows, lds);
            else if (rows <= 32)
                w4_tile<F16, E2M1, STEPS, 2, NT>(s, a, e, n0, row, rows, lds);
            else
                w4_tile<F16, E2M1, STEPS, MT, NT>(s, a, e, n0, row, rows, lds);
        }
    }
}

template <bool F16>
hipError_t launch_token(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    const ProductPath path = product_path(s);
    if (path != kPathStream) return launch_w4_tiles<F16>(s, a, path == kPathSmallTiles, stream);
    const int half = s.swiglu ? s.out / 2 : s.out;
    const int per = s.swiglu ? 16 : 32;
    int64_t z = (s.rows / s.E + 63) / 64;
    z = z < 1 ? 1 : z > kW4MaxZ ? kW4MaxZ : z;
    const dim3 grid((unsigned)((half + per - 1) / per), (unsigned)s.E, (unsigned)z);
    const dim3 block(kW4Waves * kWave);
    if (s.w4 == MOE_W4_E2M1)
        w4_kernel<F16, true, 1><<<grid, block, 0, stream>>>(s, a);
    else if (s.group == 32)
        w4_kernel<F16, false, 1><<<grid, block, 0, stream>>>(s, a);
    else if (s.group == 64)
        w4_kernel<F16, false, 2><<<grid, block, 0, stream>>>(s, a);
    else
        w4_kernel<F16, false, 4><<<grid, block, 0, stream>>>(s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grouped_matmul_w4(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    return s.tok_f16 ? launch_token<true>(s, a, stream) : launch_token<false>(s, a, stream);
}

}  // namespace moe_dc
