// grouped_matmul_stream.h -- the experts' products where tiles are too few for the chip.
//
// A workgroup takes 32 weight rows of one expert (with SwiGLU 16 gate and 16 up rows) and walks
// their inner dimension once, its four waves taking 128-byte chunks in turn, straight from global
// memory into matrix registers; the waves' sums meet in LDS at the end.  Bound by latency: 64
// rows on 8 experts x 1024 x 1024 bf16 (17 MB) take 6 us, 333 rows on 12 experts x 1144 x 777
// fp16 11 us.  (Loads in the matrix layout run at 16 bytes a clock per CU, which is why larger
// products go through LDS.)
#pragma once

#include "experts_device.h"

namespace moe_dc {
namespace {

constexpr int kStreamWaves = 4;
constexpr int kStreamMaxZ = 8;

// One tile: 16 * MT rows of x (row0 + 0..), weight rows of the workgroup.
template <int TYPE, int MT, int NT, int D>
__device__ __forceinline__ void stream_tile(const MatmulShape& s, const MatmulArgs& a, int e,
                                            int n0, int row0, int rows, float* lds)
{
    typedef Mm<TYPE> M;
    typedef typename M::Acc Acc;
    constexpr int kB = M::kBytes;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = (uint32_t)s.in * kB;
    const int chunks = (int)((row_bytes + 127) / 128);
    const int half = s.swiglu ? s.out / 2 : s.out;
    // Weight tiles t of the workgroup: with SwiGLU the first half of them are gate rows and the
    // others the up rows of the same columns.
    constexpr int kParts = 2;
    __amdgpu_buffer_rsrc_t wr[kParts];
    const int per = s.swiglu ? NT / 2 * 16 : NT * 16;          // columns of the workgroup
    const int left = half - n0 < per ? half - n0 : per;
    const char* wbase = static_cast<const char*>(a.w) + ((size_t)e * s.out + n0) * row_bytes;
    wr[0] = make_rsrc(wbase, (uint32_t)left * row_bytes);
    wr[1] = make_rsrc(wbase + (size_t)half * row_bytes, (uint32_t)left * row_bytes);
    const int mrows = rows < MT * 16 ? rows : MT * 16;
    const __amdgpu_buffer_rsrc_t xr =
        make_rsrc(static_cast<const char*>(a.x) + (size_t)row0 * row_bytes, (uint32_t)mrows * row_bytes);
    // MX: bytes of 32 elements.  Block: floats, one a chunk, for the weights in rows of 128 weight
    // rows, those of the gate and of the up rows begun anew (n0 + 0..31 lies within one block).
    const int ns = M::kBlk ? chunks : s.in / 32;
    const uint8_t* wsc = static_cast<const uint8_t*>(a.w_scales) + ((size_t)e * s.out + n0) * ns;
    const uint8_t* xsc = static_cast<const uint8_t*>(a.x_scales) + (size_t)row0 * ns;
    const int blocks = (half + kBlock - 1) / kBlock;
    const float* wblock = static_cast<const float*>(a.w_scales) +
        ((size_t)e * blocks * (s.swiglu ? 2 : 1) + n0 / kBlock) * ns;
    const float* xblock = static_cast<const float*>(a.x_scales) + (size_t)row0 * ns;

    Acc acc[MT][NT];
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) acc[m][t] = Acc{0, 0, 0, 0};

    v4i_t wv[D][NT][2], xv[D][MT][2];
    int wsv[D][NT], xsv[D][MT];
    const auto fetch = [&](int d, int c) {
        const uint32_t k0 = (uint32_t)c * 128 + g * 16, k1 = k0 + 64;
        const uint32_t p0 = k0 < row_bytes ? k0 : kRsrcPastEnd;
        const uint32_t p1 = k1 < row_bytes ? k1 : kRsrcPastEnd;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int part = s.swiglu ? t / (NT / 2) : 0;
            const int rt = s.swiglu ? t % (NT / 2) : t;
            const uint32_t ro = (uint32_t)(rt * 16 + l16) * row_bytes;
            const __amdgpu_buffer_rsrc_t r = part ? wr[1] : wr[0];
            wv[d][t][0] = load_chunk(r, p0 == kRsrcPastEnd ? p0 : ro + p0);
            wv[d][t][1] = load_chunk(r, p1 == kRsrcPastEnd ? p1 : ro + p1);
            if (M::kMx) {
                const int rr = rt * 16 + l16 < left ? rt * 16 + l16 : left - 1;
                const int cc = c < chunks ? c : chunks - 1;
                wsv[d][t] = wsc[((size_t)part * half + rr) * ns + cc * 4 + g];
            } else if (M::kBlk) {
                const int cc = c < chunks ? c : chunks - 1;
                wsv[d][t] = __float_as_int(wblock[(size_t)part * blocks * ns + cc]);
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const uint32_t ro = (uint32_t)(m * 16 + l16) * row_bytes;
            xv[d][m][0] = load_chunk(xr, p0 == kRsrcPastEnd ? p0 : ro + p0);
            xv[d][m][1] = load_chunk(xr, p1 == kRsrcPastEnd ? p1 : ro + p1);
            if (M::kMx) {
                const int rr = m * 16 + l16 < mrows ? m * 16 + l16 : mrows - 1;
                const int cc = c < chunks ? c : chunks - 1;
                xsv[d][m] = xsc[(size_t)rr * ns + cc * 4 + g];
            } else if (M::kBlk) {
                const int rr = m * 16 + l16 < mrows ? m * 16 + l16 : mrows - 1;
                const int cc = c < chunks ? c : chunks - 1;
                xsv[d][m] = __float_as_int(xblock[(size_t)rr * ns + cc]);
            }
        }
    };
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, wave + d * kStreamWaves);
    for (int c = wave; c < chunks; c += D * kStreamWaves) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const v8i_t wc = join(wv[d][t][0], wv[d][t][1]), xc = join(xv[d][m][0], xv[d][m][1]);
                    if constexpr (M::kBlk) {
                        // past the last chunk the operands are 0, and an infinite scale must not be met
                        const Acc sum = M::mma(wc, xc, Acc{0, 0, 0, 0}, 0, 0);
                        if (c + d * kStreamWaves < chunks)
                            add_scaled(acc[m][t], sum, __int_as_float(wsv[d][t]) * __int_as_float(xsv[d][m]));
                    } else {
                        acc[m][t] = M::mma(wc, xc, acc[m][t], wsv[d][t], xsv[d][m]);
                    }
                }
            fetch(d, c + (d + D) * kStreamWaves);
        }
    }

    // The waves' sums: [wave][m][t][lane] of 4 values; then one (m, t) part per wave.
    Acc* part = reinterpret_cast<Acc*>(lds);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < NT; ++t) part[((wave * MT + m) * NT + t) * kWave + lane] = acc[m][t];
    __syncthreads();
    const int nt = s.swiglu ? NT / 2 : NT;
    for (int i = wave; i < MT * nt; i += kStreamWaves) {
        const int m = i / nt, t = i - m * nt;
        const int row = m * 16 + l16;
        float r[4], u[4];
        for (int h = 0; h < (s.swiglu ? 2 : 1); ++h) {
            Acc v = part[(m * NT + t + h * nt) * kWave + lane];
#pragma unroll
            for (int w = 1; w < kStreamWaves; ++w) v += part[((w * MT + m) * NT + t + h * nt) * kWave + lane];
            float* f = h ? u : r;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                f[q] = (float)v[q];
                if (M::kRowScaled) {
                    const int n = t * 16 + g * 4 + q;
                    if (n < left) {
                        f[q] *= static_cast<const float*>(a.w_scales)[(size_t)e * s.out + h * half + n0 + n];
                        if (a.x_scales && row < mrows)
                            f[q] *= static_cast<const float*>(a.x_scales)[row0 + row];
                    }
                }
            }
        }
        if (row < mrows) {
            uint16_t* o = static_cast<uint16_t*>(a.out) + (size_t)(row0 + row) * half + n0;
            if (s.swiglu) silu_mul4(r, u, r);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int n = t * 16 + g * 4 + q;
                if (n < left) o[n] = (uint16_t)f32_to_tok_rt(r[q], s.tok_f16);
            }
        }
    }
    __syncthreads();
}

// Two workgroups a CU: without the bound block kinds take 269 registers a lane, which leaves one (333
// rows on 12 experts x 1136 x 777: 8.6 us, 7.5 with it); the other types take 202 to 256 either way and
// their times differ by less than 1 % (bf16, fp16, int8, E4M3, E5M2, MX; 2 to 60 rows an expert).
template <int TYPE>
__global__ __launch_bounds__(kStreamWaves * kWave, 2) void stream_kernel(MatmulShape s, MatmulArgs a)
{
    constexpr int NT = 2, MT = 4, D = 2;
    __shared__ float lds[kStreamWaves * MT * NT * kWave * 4];
    const int half = s.swiglu ? s.out / 2 : s.out;
    const int per = s.swiglu ? NT / 2 * 16 : NT * 16;
    const int e = blockIdx.y;
    const int begin = expert_end(s, a.ep_recv_count, a.recv_offsets, e - 1);
    const int end = expert_end(s, a.ep_recv_count, a.recv_offsets, e);
    for (int n0 = blockIdx.x * per; n0 < half; n0 += gridDim.x * per) {
        for (int row = begin + blockIdx.z * MT * 16; row < end; row += gridDim.z * MT * 16) {
            const int rows = end - row;
            // Up to two chunks a wave are all in flight with two stages, and four would only ask for
            // zeros past the end (1024 inner, 8 rows to an expert, with four and with two: block 5.7 and
            // 5.2 us, int8 and row-scaled fp8 6.3 and 5.7, MX 6.4 and 5.3).  Not for tokens: 512 of them
            // would gain as much (bf16 5.0 and 4.4), but with a fourth form of the tile in the kernel
            // 1024, the least hidden size, lose 2 % (6.06 and 6.15).
            if (rows <= 16 && Mm<TYPE>::kBytes == 1 && s.in <= 2 * 128 * kStreamWaves)
                stream_tile<TYPE, 1, NT, 2>(s, a, e, n0, row, rows, lds);
            else if (rows <= 16)
                stream_tile<TYPE, 1, NT, 4>(s, a, e, n0, row, rows, lds);
            else if (rows <= 32)
                stream_tile<TYPE, 2, NT, 2>(s, a, e, n0, row, rows, lds);
            else
                stream_tile<TYPE, MT, NT, D>(s, a, e, n0, row, rows, lds);
        }
    }
}

template <int TYPE>
hipError_t launch_stream(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    const int half = s.swiglu ? s.out / 2 : s.out;
    const int per = s.swiglu ? 16 : 32;
    int64_t z = (s.rows / s.E + 63) / 64;
    z = z < 1 ? 1 : z > kStreamMaxZ ? kStreamMaxZ : z;
    const dim3 grid((unsigned)((half + per - 1) / per), (unsigned)s.E, (unsigned)z);
    stream_kernel<TYPE><<<grid, kStreamWaves * kWave, 0, stream>>>(s, a);
    return hipGetLastError();
}

}  // namespace
}  // namespace moe_dc
