// layer.hip -- the experts' layer of a few tokens: y[t] = sum over k of w[t][k] * down(swiglu(up(x[t])))
// of the pick's expert, in two kernels.
//
// With few tokens the layer is the reading of the weights of the experts that have any, once.  Both
// kernels walk weight rows in chunks of 128 bytes from memory to matrix registers, as the streaming
// products do; nothing is packed or sent, a row of the matrix operand is a token where it lies.
//
//   up:   one workgroup per (expert with tokens, 16 columns): four waves take chunks of the inner
//         dimension in turn; gate and up rows, SwiGLU and the pick's weight, h in the token type.
//         Every workgroup finds its expert and its tokens in the ids by itself, one lane a token.
//   down: one workgroup per 16 columns of y: eight waves take the chunks of all experts in turn;
//         an expert's sums are added to its tokens' in LDS, and the waves' in the end, in an order
//         that depends on the ids only.
#include "dc_device.h"
#include "experts_device.h"
#include "layer_internal.h"

namespace moe_dc {
namespace {

constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;
constexpr int kCols = 16;                       // columns of a workgroup (SwiGLU: of gate and of up)
constexpr int kMaxIds = 1024;                   // experts

// Operands.  A chunk is 128 bytes of a weight row: 64 tokens or 128 E4M3 codes.  Lane l holds, of
// weight row l % 16, the 16 bytes at (l / 16) * 16 and at 64 + (l / 16) * 16, and of x (or h) the
// elements that meet them.
template <bool F16, bool BLOCK>
struct Chunk {
    static constexpr int kElements = BLOCK ? 128 : 64;
    static constexpr int kXLoads = BLOCK ? 4 : 2;           // of 16 bytes, per row of x and chunk

    // Two codes of a dword as a pair of 16-bit floats, exactly.
    template <bool HI>
    static __device__ __forceinline__ int pair(int w)
    {
        if constexpr (F16) return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, HI));
        else return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
    }
    static __device__ __forceinline__ v4f_t mma16(v4i_t a, v4i_t b, v4f_t acc)
    {
        if constexpr (F16)
            return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h_t, a),
                                                          __builtin_bit_cast(v8h_t, b), acc, 0, 0, 0);
        else
            return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf_t, a),
                                                           __builtin_bit_cast(v8bf_t, b), acc, 0, 0, 0);
    }
    // acc + weights (two loads) times x (kXLoads loads)
    static __device__ __forceinline__ v4f_t mma(const v4i_t (&w)[2], const v4i_t (&x)[kXLoads], v4f_t acc)
    {
        if constexpr (BLOCK) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const v4i_t lo = {pair<false>(w[p].x), pair<true>(w[p].x), pair<false>(w[p].y), pair<true>(w[p].y)};
                const v4i_t hi = {pair<false>(w[p].z), pair<true>(w[p].z), pair<false>(w[p].w), pair<true>(w[p].w)};
                acc = mma16(lo, x[2 * p], acc);
                acc = mma16(hi, x[2 * p + 1], acc);
            }
            return acc;
        } else {
            return mma16(w[1], x[1], mma16(w[0], x[0], acc));
        }
    }
    // Byte offsets of the lane's pieces of chunk c; past the row's end they are past every resource.
    static __device__ __forceinline__ void offsets(int c, int g, uint32_t row_bytes, uint32_t (&wo)[2],
                                                   uint32_t (&xo)[kXLoads])
    {
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            const uint32_t k = (uint32_t)c * 128 + p * 64 + g * 16;
            wo[p] = k < row_bytes ? k : kRsrcPastEnd;
            if constexpr (BLOCK) {
                xo[2 * p] = k < row_bytes ? 2 * k : kRsrcPastEnd;
                xo[2 * p + 1] = k < row_bytes ? 2 * k + 16 : kRsrcPastEnd;
            } else {
                xo[p] = wo[p];
            }
        }
    }
};

__device__ __forceinline__ uint32_t beyond(uint32_t base, uint32_t off)
{
    return off == kRsrcPastEnd ? off : base + off;
}

__device__ __forceinline__ bool active(const LayerShape& s, const LayerArgs& a, int t, int k)
{
    return s.mask_kind == 0 || a.mask[s.mask_kind == 1 ? t : t * s.K + k] != 0;
}

struct UpLds {
    float part[kUpWaves * 4 * 2 * kWave * 4];   // sums of [wave][row tile][gate, up][lane]
    uint32_t present[kMaxIds / 32];
    int token[kLayerTokens];
    float weight[kLayerTokens];
};

// The expert of slot j (the j-th of those that have tokens, by id), its tokens in ascending order and
// the sum of the weights with which each chose it.  Lane t holds the ids of token t.
__device__ __forceinline__ Slot find_slot(const LayerShape& s, const LayerArgs& a, int j, UpLds& lds)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    int id[kMaxK];
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
        id[k] = -1;
        if (k < s.K && lane < s.T) {
            const int v = a.ids[lane * s.K + k];
            if (v >= 0 && v < s.E && active(s, a, lane, k)) id[k] = v;
        }
    }
    if (threadIdx.x < kMaxIds / 32) lds.present[threadIdx.x] = 0;
    __syncthreads();
    if (wave == 0) {
#pragma unroll
        for (int k = 0; k < kMaxK; ++k)
            if (id[k] >= 0) atomicOr(&lds.present[id[k] >> 5], 1u << (id[k] & 31));
    }
    __syncthreads();
    const uint32_t word = lane < kMaxIds / 32 ? lds.present[lane] : 0;
    int upto = __popc(word);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up(upto, off, kWave);
        if (lane >= off) upto += o;
    }
    const uint64_t holds = __ballot(lane < kMaxIds / 32 && upto > j && upto - __popc(word) <= j);
    Slot slot = {-1, 0, 0, 0};
    if (holds == 0) return slot;
    const int src = __ffsll((unsigned long long)holds) - 1;
    uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, src);
    const int skip = j - (__builtin_amdgcn_readlane(upto, src) - __popc(bits));
    for (int i = 0; i < skip; ++i) bits &= bits - 1;
    slot.expert = src * 32 + __ffs((int)bits) - 1;
    int before = 0;
    bool has = false;
    float weight = 0.0f;
#pragma unroll
    for (int k = 0; k < kMaxK; ++k) {
        if (id[k] >= 0 && id[k] < slot.expert) ++before;
        if (id[k] == slot.expert) {
            has = true;
            weight += a.weights[lane * s.K + k];
        }
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) before += __shfl_xor(before, off, kWave);
    const uint64_t who = __ballot(has);
    slot.first = __builtin_amdgcn_readfirstlane(before);
    slot.rows = __popcll((unsigned long long)who);
    if (has && wave == 0) {
        const int at = __popcll((unsigned long long)(who & ((1ull << lane) - 1)));
        lds.token[at] = lane;
        lds.weight[at] = weight;
    }
    __syncthreads();
    return slot;
}

template <bool F16, bool BLOCK, int MT, int D>
__device__ __forceinline__ void up_tile(const LayerShape& s, const LayerArgs& a, const Slot& slot, int n0,
                                        UpLds& lds)
{
    typedef Chunk<F16, BLOCK> C;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    const uint32_t row_bytes = (uint32_t)s.H * (BLOCK ? 1 : 2);
    const int chunks = (int)((row_bytes + 127) / 128);
    const int left = s.F - n0 < kCols ? s.F - n0 : kCols;
    const char* base = static_cast<const char*>(a.up) + ((size_t)slot.expert * 2 * s.F + n0) * row_bytes;
    const __amdgpu_buffer_rsrc_t wr[2] = {make_rsrc(base, (uint32_t)left * row_bytes),
                                          make_rsrc(base + (size_t)s.F * row_bytes, (uint32_t)left * row_bytes)};
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)s.T * s.H * 2);
    const int blocks = (s.F + 127) / 128;
    const float* scales = a.up_scales + ((size_t)slot.expert * 2 * blocks + n0 / 128) * chunks;
    const uint32_t wrow = (uint32_t)l16 * row_bytes;
    uint32_t xrow[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int r = m * 16 + l16;
        xrow[m] = r < slot.rows ? (uint32_t)lds.token[r] * s.H * 2 : kRsrcPastEnd;
    }
    v4i_t w[D][2][2], x[D][MT][C::kXLoads];
    float sc[D][2];
    const auto fetch = [&](int d, int c) {
        uint32_t wo[2], xo[C::kXLoads];
        C::offsets(c, g, row_bytes, wo, xo);
#pragma unroll
        for (int t = 0; t < 2; ++t) {
#pragma unroll
            for (int p = 0; p < 2; ++p) w[d][t][p] = load_chunk(wr[t], beyond(wrow, wo[p]));
            if (BLOCK) sc[d][t] = scales[(size_t)t * blocks * chunks + (c < chunks ? c : chunks - 1)];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int p = 0; p < C::kXLoads; ++p)
                x[d][m][p] = load_chunk(xr, xrow[m] == kRsrcPastEnd ? kRsrcPastEnd : beyond(xrow[m], xo[p]));
    };
    v4f_t acc[MT][2];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m][0] = acc[m][1] = v4f_t{0, 0, 0, 0};
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d, wave + d * kUpWaves);
    for (int c = wave; c < chunks; c += D * kUpWaves) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int t = 0; t < 2; ++t) {
                    if constexpr (BLOCK) {
                        const v4f_t sum = C::mma(w[d][t], x[d][m], v4f_t{0, 0, 0, 0});
                        if (c + d * kUpWaves < chunks) add_scaled(acc[m][t], sum, sc[d][t]);
                    } else {
                        acc[m][t] = C::mma(w[d][t], x[d][m], acc[m][t]);
                    }
                }
            fetch(d, c + (d + D) * kUpWaves);
        }
    }
    v4f_t* part = reinterpret_cast<v4f_t*>(lds.part);
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int t = 0; t < 2; ++t) part[((wave * MT + m) * 2 + t) * kWave + lane] = acc[m][t];
    __syncthreads();
    // one row tile a wave
    for (int m = wave; m < MT; m += kUpWaves) {
        float r[2][4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            v4f_t v = part[(m * 2 + t) * kWave + lane];
#pragma unroll
            for (int o = 1; o < kUpWaves; ++o) v += part[((o * MT + m) * 2 + t) * kWave + lane];
#pragma unroll
            for (int q = 0; q < 4; ++q) r[t][q] = v[q];
        }
        const int row = m * 16 + l16;
        if (row >= slot.rows) continue;
        silu_mul4(r[0], r[1], r[0]);
        const float weight = lds.weight[row];
        uint16_t* o = static_cast<uint16_t*>(a.h) + (size_t)(slot.first + row) * s.F + n0 + g * 4;
        if (g * 4 < left)                       // F is a multiple of 8
            *reinterpret_cast<uint2*>(o) = make_uint2(pack_out2(r[0][0] * weight, r[0][1] * weight, F16),
                                                      pack_out2(r[0][2] * weight, r[0][3] * weight, F16));
    }
}

template <bool F16, bool BLOCK>
__global__ __launch_bounds__(kUpWaves * kWave) void up_kernel(LayerShape s, LayerArgs a)
{
    __shared__ UpLds lds;
    const int j = blockIdx.y;
    const Slot slot = find_slot(s, a, j, lds);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) a.slots[j] = slot;
        if ((int)threadIdx.x < slot.rows) a.tokens[slot.first + threadIdx.x] = lds.token[threadIdx.x];
    }
    if (slot.expert < 0) return;
    const int n0 = blockIdx.x * kCols;
    if (slot.rows <= 16) up_tile<F16, BLOCK, 1, 4>(s, a, slot, n0, lds);
    else if (slot.rows <= 32) up_tile<F16, BLOCK, 2, 2>(s, a, slot, n0, lds);
    else up_tile<F16, BLOCK, 4, 2>(s, a, slot, n0, lds);
}

// MT: tiles of 16 rows an expert can have.  LDS: sums [wave][token][column], the slots, the rows'
// tokens.
template <bool F16, bool BLOCK, int MT, int D>
__global__ __launch_bounds__(kDownWaves * kWave) void down_kernel(LayerShape s, LayerArgs a)
{
    typedef Chunk<F16, BLOCK> C;
    extern __shared__ float sums[];
    __shared__ int count_lds;
    Slot* slots = reinterpret_cast<Slot*>(sums + kDownWaves * s.T * kCols);
    int* tokens = reinterpret_cast<int*>(slots + s.slots);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    if (threadIdx.x == 0) count_lds = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < s.slots; i += kDownWaves * kWave) {
        slots[i] = a.slots[i];
        if (slots[i].expert >= 0) atomicMax(&count_lds, i + 1);
    }
    for (int i = threadIdx.x; i < s.T * s.K; i += kDownWaves * kWave)
        tokens[i] = a.tokens[i];
    for (int i = threadIdx.x; i < kDownWaves * s.T * kCols; i += kDownWaves * kWave) sums[i] = 0.0f;
    __syncthreads();
    const int count = __builtin_amdgcn_readfirstlane(count_lds);
    const char* h = static_cast<const char*>(a.h);
    const uint32_t row_bytes = (uint32_t)s.F * (BLOCK ? 1 : 2);
    const uint32_t h_bytes = (uint32_t)s.F * 2;
    const int chunks = (int)((row_bytes + 127) / 128);
    const int n0 = blockIdx.x * kCols;
    const int left = s.H - n0 < kCols ? s.H - n0 : kCols;
    const int blocks = (s.H + 127) / 128;
    const uint32_t wrow = (uint32_t)l16 * row_bytes;

    // Units (slot, chunk) go round the waves.
    struct Place { int slot, chunk; };
    const auto step = [&](Place p) {
        p.chunk += kDownWaves;
        while (p.chunk >= chunks) {
            p.chunk -= chunks;
            ++p.slot;
        }
        return p;
    };
    const auto slot_at = [&](int i) {
        Slot r;
        r.expert = __builtin_amdgcn_readfirstlane(slots[i].expert);
        r.first = __builtin_amdgcn_readfirstlane(slots[i].first);
        r.rows = __builtin_amdgcn_readfirstlane(slots[i].rows);
        return r;
    };
    v4i_t w[D][2], x[D][MT][C::kXLoads];
    float sc[D];
    Place ahead = {0, wave - kDownWaves};
    ahead = step(ahead);
    Slot next = {0, 0, 0, 0};
    int held = -1;                              // the slot that `next` describes
    const auto fetch = [&](int d) {
        const bool there = ahead.slot < count;
        if (there && held != ahead.slot) {
            next = slot_at(ahead.slot);
            held = ahead.slot;
        }
        const __amdgpu_buffer_rsrc_t wr = make_rsrc(
            static_cast<const char*>(a.down) + ((size_t)next.expert * s.H + n0) * row_bytes,
            there ? (uint32_t)left * row_bytes : 0);
        const __amdgpu_buffer_rsrc_t hr =
            make_rsrc(h + (size_t)next.first * h_bytes, there ? (uint32_t)next.rows * h_bytes : 0);
        uint32_t wo[2], xo[C::kXLoads];
        C::offsets(ahead.chunk, g, row_bytes, wo, xo);
#pragma unroll
        for (int p = 0; p < 2; ++p) w[d][p] = load_chunk(wr, beyond(wrow, wo[p]));
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int p = 0; p < C::kXLoads; ++p)
                x[d][m][p] = load_chunk(hr, beyond((uint32_t)(m * 16 + l16) * h_bytes, xo[p]));
        if (BLOCK) sc[d] = a.down_scales[((size_t)next.expert * blocks + n0 / 128) * chunks + ahead.chunk];
        ahead = step(ahead);
    };
    v4f_t acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4f_t{0, 0, 0, 0};
    float* mine = sums + wave * s.T * kCols;
    // Adds an expert's sums to those of its tokens.
    const auto flush = [&](int i) {
        const Slot slot = slot_at(i);
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int row = m * 16 + l16;
            if (row < slot.rows) {
                v4f_t* to = reinterpret_cast<v4f_t*>(mine + tokens[slot.first + row] * kCols + g * 4);
                *to = *to + acc[m];
            }
            acc[m] = v4f_t{0, 0, 0, 0};
        }
    };
    Place now = {0, wave - kDownWaves};
    now = step(now);
    int open = now.slot;
#pragma unroll
    for (int d = 0; d < D; ++d) fetch(d);
    while (now.slot < count) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (now.slot < count) {
                if (now.slot != open) {
                    flush(open);
                    open = now.slot;
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    if constexpr (BLOCK) add_scaled(acc[m], C::mma(w[d], x[d][m], v4f_t{0, 0, 0, 0}), sc[d]);
                    else acc[m] = C::mma(w[d], x[d][m], acc[m]);
                }
            }
            now = step(now);
            fetch(d);
        }
    }
    if (open < count) flush(open);
    __syncthreads();
    const bool f16 = F16;
    for (int i = threadIdx.x; i < s.T * kCols; i += kDownWaves * kWave) {
        const int t = i / kCols, n = i % kCols;
        if (n >= left) continue;
        float v = 0.0f;
#pragma unroll
        for (int o = 0; o < kDownWaves; ++o) v += sums[o * s.T * kCols + i];
        const size_t at = (size_t)t * s.H + n0 + n;
        if (s.id_end > s.zero_end)
            for (int k = 0; k < s.K; ++k) {
                const int id = a.ids[t * s.K + k];
                if (id >= s.zero_end && id < s.id_end && active(s, a, t, k))
                    v += a.weights[t * s.K + k] * tok_lo_rt(static_cast<const uint16_t*>(a.x)[at], f16);
            }
        if (a.shared) v += tok_lo_rt(static_cast<const uint16_t*>(a.shared)[at], f16);
        static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_tok_rt(v, f16);
    }
}

template <bool F16, bool BLOCK>
hipError_t launch(const LayerShape& s, const LayerArgs& a, hipStream_t stream)
{
    up_kernel<F16, BLOCK><<<dim3((unsigned)((s.F + kCols - 1) / kCols), (unsigned)s.slots), kUpWaves * kWave, 0,
                            stream>>>(s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((unsigned)((s.H + kCols - 1) / kCols));
    const size_t lds = (size_t)kDownWaves * s.T * kCols * 4 + s.slots * sizeof(Slot) + (size_t)s.T * s.K * 4;
    if (s.T <= 16) down_kernel<F16, BLOCK, 1, 4><<<grid, kDownWaves * kWave, lds, stream>>>(s, a);
    else if (s.T <= 32) down_kernel<F16, BLOCK, 2, 4><<<grid, kDownWaves * kWave, lds, stream>>>(s, a);
    else down_kernel<F16, BLOCK, 4, 2><<<grid, kDownWaves * kWave, lds, stream>>>(s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_layer(const LayerShape& s, const LayerArgs& a, hipStream_t stream)
{
    if (s.tok_f16) return s.block ? launch<true, true>(s, a, stream) : launch<true, false>(s, a, stream);
    return s.block ? launch<false, true>(s, a, stream) : launch<false, false>(s, a, stream);
}

}  // namespace moe_dc
