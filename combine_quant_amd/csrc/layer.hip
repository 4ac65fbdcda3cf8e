// layer.hip -- the experts' layer of a few tokens: y[t] = sum over k of w[t][k] * down(swiglu(up(x[t])))
// of the pick's expert, in two kernels.
//
// With few tokens the layer is the reading of the weights of the experts that have any, once; nothing is
// packed or sent, a row of the matrix operand is a token where it lies.  Both kernels walk weight rows
// in chunks of 128 bytes.  Every wave has a ring of stages in LDS, which its own loads fill directly,
// several chunks ahead (whole 128-byte rows, and no registers for what is on its way), so that no
// barrier holds the stream up.
//
//   up:   one workgroup per (expert with tokens, 16 columns): the waves take chunks of the inner
//         dimension in turn; gate and up rows, SwiGLU, h in the token type.
//         Every wave finds its expert and its tokens in the ids by itself, one lane a token.
//   down: one workgroup per 16 or 32 columns of y: the waves take the chunks of all experts in turn;
//         an expert's sums are added to its tokens' in LDS, times the pick's weight, and the waves' in
//         the end, in an order that depends on the ids only.
//
// h is kept as two numbers of the token type, its rounding and what that leaves (16 bits in bf16, 22 in
// fp16), each a matrix operand as it lies: the down kernel multiplies twice, where HBM leaves it the
// time (an infinite weight meets both parts, and gives NaN).  With one the result would be sqrt(2) further
// from 64 bits (bf16 0.0024 against 0.0017, fp16 0.00029 against 0.00020).  A weight of a pick multiplies
// fp32 sums: in fp16 a small one would push h among the subnormals, a large one past 65504.
//
// Bound by HBM: 32 tokens on 256 experts x 7168 x 2048 E4M3 (7.2 GB) take 1.19 to 1.24 ms, 6.0 TB/s, a
// read's rate; 1 token on 8 experts bf16 (0.70 GB) 122 us, 5.8 TB/s.  By latency: 5 tokens on 8 experts x
// 1024 x 520 fp16 12.0 us, of which the up kernel's ids and list of tokens take 2.0, the down kernel's list of
// experts 1.0, the first bytes 1.2 each and the gap between the kernels 1.3.  (Weights straight to matrix
// registers, rows of x too: 1.79 ms, 139 and 15.4 us.)
#include "dc_device.h"
#include "experts_device.h"
#include "experts_tiles.h"
#include "layer_internal.h"

namespace moe_dc {
namespace {

constexpr int kRing = 2;                        // stages of a wave
// Many small workgroups hide each other's start and end, so the up kernel's have two waves; with few
// columns in all, four waves share the chunks of a workgroup's.  Two waves against four, us: 1 token on 8
// experts of 7168 x 2048 bf16 122 and 127; 32 tokens on 256 experts E4M3 1239 and 1242, on 64 experts 497
// and 508; 64 tokens on 8 experts of 4096 x 4096 E4M3 121 and 149; 5 tokens on 8 experts of 1024 x 520
// fp16 12.8 and 12.7 (13.8 and 12.7 before the weights moved to the down kernel).  A third stage with
// four waves: 2, 4 and 14 % more in the first three.
constexpr int64_t kFewUp = 16 * 512;            // columns (of all experts) up to which it has four
// Columns of y and waves of a workgroup: many columns share the rows of h, but few workgroups leave
// CUs idle.  32 columns and four waves against 16 and eight (four where the rings are large), us: H = 7168,
// 32 tokens on 64 experts x 2048 E4M3 497 and 617, 64 tokens 546 and 642; H = 5120, 64 tokens on 64 x 1536
// E4M3 339 and 409, 8 tokens 119 and 122; H = 4608, 64 tokens on 64 x 1536 bf16 540 and 589, 8 tokens 200
// and 214; H = 4096, 64 tokens on 64 x 1536 E4M3 292 and 270, 32 tokens on 32 x 1024 E4M3 101 and 87, 8
// tokens on 8 x 1024 bf16 48.8 and 43.1; H = 2048, 16 tokens on 32 x 1408 bf16 130 and 103.
constexpr int kWideDown = 32 * 144;             // H from which it takes 32
constexpr int kMaxIds = 1024;                   // experts
constexpr int kMaxChunks = 64;                  // of an up row with scales (H <= 8192)

// A chunk is 128 bytes of a weight row: 64 tokens or 128 E4M3 codes, which meet one or two runs of 64
// elements of a row of x (or h).  A run is 128 bytes, or PARTS times 128 one after another (the two
// parts of h).  NT tiles of 16 weight rows and RP rows of x make a stage; a load fills 1 KB of it.
template <bool F16, bool BLOCK, int NT, int RP, int PARTS>
struct Stage {
    static constexpr int kRuns = BLOCK ? 2 : 1;
    static constexpr int kHalves = kRuns * PARTS;            // 128 bytes each
    static constexpr int kTiles = (RP + 15) / 16;            // of rows of x
    static constexpr int kW = NT * 2048;
    static constexpr int kX = RP * 128 * kHalves < 1024 ? 1024 : RP * 128 * kHalves;
    static constexpr int kBytes = kW + kX;
    static constexpr int kXLoads = kX / 1024;
    static constexpr int kLoads = NT * 2 + kXLoads;

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

    // What a lane reads of a stage: of weight row l % 16 the pieces (16 bytes) l / 16 and 4 + l / 16,
    // and of row l % 16 of x those that meet them.  Piece p of row r lies at place p ^ (r & 7).
    struct Regs {
        v4i_t w[NT][2];
        v4i_t x[kTiles][PARTS][2 * kRuns];
    };
    static __device__ __forceinline__ void read(const char* st, Regs& r)
    {
        const int lane = threadIdx.x & (kWave - 1), l16 = lane & 15, g = lane >> 4;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int p = 0; p < 2; ++p)
                r.w[t][p] = *reinterpret_cast<const v4i_t*>(st + t * 2048 + l16 * 128 +
                                                            (((p * 4 + g) ^ (l16 & 7)) << 4));
#pragma unroll
        for (int m = 0; m < kTiles; ++m) {
            const int row = m * 16 + (RP < 16 ? l16 % RP : l16);
            const char* xs = st + kW + row * 128;
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
                for (int i = 0; i < 2 * kRuns; ++i) {
                    const int half = (BLOCK ? i >> 1 : 0) * PARTS + p, piece = BLOCK ? 2 * g + (i & 1) : i * 4 + g;
                    r.x[m][p][i] = *reinterpret_cast<const v4i_t*>(xs + half * RP * 128 + ((piece ^ (row & 7)) << 4));
                }
        }
    }
    // acc + a weight tile times a tile of rows
    static __device__ __forceinline__ v4f_t mma(const v4i_t (&w)[2], const v4i_t (&x)[PARTS][2 * kRuns], v4f_t acc)
    {
        if constexpr (BLOCK) {
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const v4i_t lo = {pair<false>(w[p].x), pair<true>(w[p].x), pair<false>(w[p].y), pair<true>(w[p].y)};
                const v4i_t hi = {pair<false>(w[p].z), pair<true>(w[p].z), pair<false>(w[p].w), pair<true>(w[p].w)};
#pragma unroll
                for (int q = 0; q < PARTS; ++q) acc = mma16(hi, x[q][2 * p + 1], mma16(lo, x[q][2 * p], acc));
            }
        } else {
#pragma unroll
            for (int q = 0; q < PARTS; ++q) acc = mma16(w[1], x[q][1], mma16(w[0], x[q][0], acc));
        }
        return acc;
    }

    // Byte offsets of the lane's pieces within 128 bytes, for the loads: weights (of a tile's first 8
    // rows) and, of load i, the row of x, its half and piece.
    static __device__ __forceinline__ uint32_t wpiece()
    {
        const int lane = threadIdx.x & (kWave - 1);
        return (uint32_t)((lane & 7) ^ (lane >> 3)) * 16;
    }
    static __device__ __forceinline__ int xrow(int i)
    {
        const int at = (i * kWave + (int)(threadIdx.x & (kWave - 1))) / 8;
        return at / RP < kHalves ? at % RP : RP;             // RP: none
    }
    static __device__ __forceinline__ uint32_t xhalf(int i)
    {
        return (uint32_t)(i * kWave + (int)(threadIdx.x & (kWave - 1))) / 8 / RP;
    }
    static __device__ __forceinline__ uint32_t xpiece(int i)
    {
        const int lane = threadIdx.x & (kWave - 1), at = (i * kWave + lane) / 8;
        return (uint32_t)((lane & 7) ^ (at % RP & 7)) * 16;
    }
    // Loads chunk c into a stage.  wr: NT tiles' resources; row_bytes of a weight row; xoff: offset of
    // the row of x (kRsrcPastEnd: none) for load i.
    static __device__ __forceinline__ void fill(char* st, const __amdgpu_buffer_rsrc_t (&wr)[NT],
                                                __amdgpu_buffer_rsrc_t xr, uint32_t row_bytes,
                                                const uint32_t (&xoff)[kXLoads], int c)
    {
        const uint32_t k = (uint32_t)c * 128 + wpiece();
        const uint32_t w0 = k < row_bytes ? ((threadIdx.x & (kWave - 1)) >> 3) * row_bytes + k : kRsrcPastEnd;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            load_lds16(wr[t], st + t * 2048, w0);
            load_lds16(wr[t], st + t * 2048 + 1024, w0 == kRsrcPastEnd ? w0 : w0 + 8 * row_bytes);
        }
#pragma unroll
        for (int i = 0; i < kXLoads; ++i) {
            // the piece's place among the row's elements, in bytes of tokens, and where it lies
            const uint32_t e = (uint32_t)c * (128 * kRuns) + xhalf(i) / PARTS * 128 + xpiece(i);
            const uint32_t q = (uint32_t)c * (128 * kHalves) + xhalf(i) * 128 + xpiece(i);
            load_lds16(xr, st + kW + i * 1024,
                       xoff[i] != kRsrcPastEnd && e < row_bytes * kRuns ? xoff[i] + q : kRsrcPastEnd);
        }
    }
};

// Until what the wave's LDS reads and loads so far asked for is there.
__device__ __forceinline__ void wait_lds() { asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory"); }

__device__ __forceinline__ bool active(const LayerShape& s, const LayerArgs& a, int t, int k)
{
    return s.mask_kind == 0 || a.mask[s.mask_kind == 1 ? t : t * s.K + k] != 0;
}

// A wave's own notes.
struct UpNotes {
    uint32_t present[kMaxIds / 32];             // experts with tokens
    uint32_t who[kLayerTokens / 32];            // tokens of the wave's expert
    int token[kLayerTokens];                    // the same in ascending order
    float scales[2][kMaxChunks];                // of the gate's and the up rows' block
};

// Inclusive sums over the first 32 lanes (the others' values do not matter).
__device__ __forceinline__ int scan32(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, true);      // row_shr 1, 2, 4, 8
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, true);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, true);
    const int low = __builtin_amdgcn_readlane(v, 15);
    return (threadIdx.x & (kWave - 1)) >= 16 ? v + low : v;
}

// The expert of slot j (the j-th of those that have tokens, by id) and its tokens in ascending order.
// A lane holds every 64th pick.  The picks' ids (-1: inactive) and weights are left in LDS for
// sum_weights; all waves of a workgroup write the same there, and one that reads them has written them.
__device__ __forceinline__ Slot find_slot(const LayerShape& s, const LayerArgs& a, int j, UpNotes& notes,
                                          int* ids, float* weights)
{
    const int lane = threadIdx.x & (kWave - 1);
    const int picks = s.T * s.K;
    constexpr int kPasses = kLayerTokens * kMaxK / kWave;
    const uint32_t magic = 65536u / (uint32_t)s.K + 1;       // p / K for p < 1024
    const auto token_of = [&](int p) { return (int)((uint32_t)p * magic >> 16); };
    const __amdgpu_buffer_rsrc_t ir = make_rsrc(a.ids, (uint32_t)picks * 4);
    const __amdgpu_buffer_rsrc_t fr = make_rsrc(a.weights, (uint32_t)picks * 4);
    const __amdgpu_buffer_rsrc_t mr =
        make_rsrc(a.mask, s.mask_kind == 0 ? 0 : s.mask_kind == 1 ? (uint32_t)s.T : (uint32_t)picks);
    int id[kPasses], on[kPasses];
    float weight[kPasses];
    // all loads at once
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
        const int p = i * kWave + lane;
        id[i] = -1;
        on[i] = 1;
        weight[i] = 0.0f;
        if (i * kWave < picks) {
            id[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(ir, p * 4, 0, 0);
            weight[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(fr, p * 4, 0, 0));
            if (s.mask_kind != 0)
                on[i] = (int)__builtin_amdgcn_raw_buffer_load_b8(mr, s.mask_kind == 1 ? token_of(p) : p, 0, 0);
        }
    }
    if (lane < kMaxIds / 32) notes.present[lane] = 0;
    if (lane < kLayerTokens / 32) notes.who[lane] = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        if (i * kWave < picks) {
            const int p = i * kWave + lane;
            if (p >= picks || on[i] == 0 || id[i] < 0 || id[i] >= s.E) id[i] = -1;
            else atomicOr(&notes.present[id[i] >> 5], 1u << (id[i] & 31));
            if (p < picks) {
                ids[p] = id[i];
                weights[p] = weight[i];
            }
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const uint32_t word = lane < kMaxIds / 32 ? notes.present[lane] : 0;
    const int upto = scan32(__popc(word));
    const uint64_t holds = __ballot(lane < kMaxIds / 32 && upto > j && upto - __popc(word) <= j);
    Slot slot = {-1, 0, 0, 0};
    if (holds == 0) return slot;
    const int src = __ffsll((unsigned long long)holds) - 1;
    uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)word, src);
    const int skip = j - (__builtin_amdgcn_readlane(upto, src) - __popc(bits));
    for (int i = 0; i < skip; ++i) bits &= bits - 1;
    slot.expert = src * 32 + __ffs((int)bits) - 1;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
        if (i * kWave < picks) {
            slot.first += __popcll((unsigned long long)__ballot(id[i] >= 0 && id[i] < slot.expert));
            if (id[i] == slot.expert) {
                const int t = token_of(i * kWave + lane);
                atomicOr(&notes.who[t >> 5], 1u << (t & 31));
            }
        }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    const uint64_t who = (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)notes.who[0]) |
                         (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)notes.who[1]) << 32;
    slot.rows = __popcll((unsigned long long)who);
    if (who >> lane & 1) notes.token[__popcll((unsigned long long)(who & ((1ull << lane) - 1)))] = lane;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    return slot;
}

// The sum, in the picks' order, of the weights with which each of the slot's tokens (a lane each) chose
// its expert.
__device__ __forceinline__ float sum_weights(const LayerShape& s, const Slot& slot, const int* ids,
                                             const float* weights, const UpNotes& notes)
{
    const int lane = threadIdx.x & (kWave - 1);
    float total = 0.0f;
    if (lane >= slot.rows) return total;
    const int p0 = notes.token[lane] * s.K;
    for (int k = 0; k < s.K; ++k)
        if (ids[p0 + k] == slot.expert) total += weights[p0 + k];
    return total;
}

// What a rounded value leaves, 0 where it is infinite or NaN.
template <bool F16>
__device__ __forceinline__ float rest(float v, uint32_t rounded)
{
    const float r = tok_lo<F16>(rounded & 0xFFFF);
    return __builtin_fabsf(r) < INFINITY ? v - r : 0.0f;
}

// Four elements of a row of h from element n on, both parts.
template <bool F16>
__device__ __forceinline__ void store_h(char* row, int n, const float (&v)[4])
{
    char* o = row + n / 64 * 256 + n % 64 * 2;
    const uint2 hi = make_uint2(pack_out2(v[0], v[1], F16), pack_out2(v[2], v[3], F16));
    *reinterpret_cast<uint2*>(o) = hi;
    *reinterpret_cast<uint2*>(o + 128) =
        make_uint2(pack_out2(rest<F16>(v[0], hi.x), rest<F16>(v[1], hi.x >> 16), F16),
                   pack_out2(rest<F16>(v[2], hi.y), rest<F16>(v[3], hi.y >> 16), F16));
}

// RP: rows of an expert that share a sweep over its weights.
template <bool F16, bool BLOCK, int RP, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void up_kernel(LayerShape s, LayerArgs a)
{
    typedef Stage<F16, BLOCK, 2, RP, 1> S;
    constexpr int kRows = S::kTiles;
    __shared__ __align__(1024) char ring[WAVES][kRing][S::kBytes];
    __shared__ UpNotes all_notes[WAVES];
    static_assert(kRing * S::kBytes >= kRows * 2 * kWave * 16, "a wave's sums take its ring's place");
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    UpNotes& notes = all_notes[wave];
    const int j = blockIdx.y;
    extern __shared__ __align__(16) char picks[];            // ids, then weights
    int* ids = reinterpret_cast<int*>(picks);
    float* weights = reinterpret_cast<float*>(ids + s.T * s.K);
    const Slot slot = find_slot(s, a, j, notes, ids, weights);
    const bool writes = blockIdx.x == 0 && wave == 0;        // the slot and its rows
    if (writes && lane == 0) a.slots[j] = slot;
    if (slot.expert < 0) return;
    const int n0 = blockIdx.x * 16;
    const uint32_t row_bytes = (uint32_t)s.H * (BLOCK ? 1 : 2);
    const int chunks = (int)((row_bytes + 127) / 128);
    const int left = s.F - n0 < 16 ? s.F - n0 : 16;
    const char* base = static_cast<const char*>(a.up) + ((size_t)slot.expert * 2 * s.F + n0) * row_bytes;
    const __amdgpu_buffer_rsrc_t wr[2] = {make_rsrc(base, (uint32_t)left * row_bytes),
                                          make_rsrc(base + (size_t)s.F * row_bytes, (uint32_t)left * row_bytes)};
    const __amdgpu_buffer_rsrc_t xr = make_rsrc(a.x, (uint32_t)s.T * s.H * 2);
    if (BLOCK) {
        const int blocks = (s.F + 127) / 128;
        const float* scales = a.up_scales + ((size_t)slot.expert * 2 * blocks + n0 / 128) * chunks;
#pragma unroll
        for (int t = 0; t < 2; ++t)
            load_lds4(make_rsrc(scales + (size_t)t * blocks * chunks, (uint32_t)chunks * 4),
                      reinterpret_cast<char*>(notes.scales[t]), (uint32_t)lane * 4);
    }
    // Each workgroup begins at another chunk, so that rows of a length that is a multiple of a large
    // power of two are not read in step all over the chip (H = 4096, F = 1024: 44.5 -> 40.8 us).
    const int rot = (int)(blockIdx.x * 5 % chunks);
    const auto turn = [&](int c) { return c >= chunks ? c : c + rot >= chunks ? c + rot - chunks : c + rot; };
    for (int r0 = 0; r0 < slot.rows; r0 += RP) {
        uint32_t xoff[S::kXLoads];
#pragma unroll
        for (int i = 0; i < S::kXLoads; ++i) {
            const int r = r0 + S::xrow(i);
            xoff[i] = S::xrow(i) < RP && r < slot.rows ? (uint32_t)notes.token[r] * s.H * 2 : kRsrcPastEnd;
        }
        v4f_t acc[kRows][2];
#pragma unroll
        for (int m = 0; m < kRows; ++m) acc[m][0] = acc[m][1] = v4f_t{0, 0, 0, 0};
#pragma unroll
        for (int d = 0; d < kRing; ++d) S::fill(ring[wave][d], wr, xr, row_bytes, xoff, turn(wave + d * WAVES));
        if (r0 == 0 && writes) {
            const float weight = sum_weights(s, slot, ids, weights, notes);
            if (lane < slot.rows) a.rows[slot.first + lane] = Row{notes.token[lane], weight};
        }
        for (int c = wave; c < chunks; c += kRing * WAVES) {
#pragma unroll
            for (int d = 0; d < kRing; ++d) {
                const int now = c + d * WAVES;
                typename S::Regs r;
                wait_loads<(kRing - 1) * S::kLoads>();
                S::read(ring[wave][d], r);
                float sc[2];
                if (BLOCK) {
                    sc[0] = notes.scales[0][turn(now) & (kMaxChunks - 1)];
                    sc[1] = notes.scales[1][turn(now) & (kMaxChunks - 1)];
                }
                wait_lds();
                S::fill(ring[wave][d], wr, xr, row_bytes, xoff, turn(now + kRing * WAVES));
#pragma unroll
                for (int m = 0; m < kRows; ++m)
#pragma unroll
                    for (int t = 0; t < 2; ++t) {
                        if constexpr (BLOCK) {
                            const v4f_t sum = S::mma(r.w[t], r.x[m], v4f_t{0, 0, 0, 0});
                            if (now < chunks) add_scaled(acc[m][t], sum, sc[t]);
                        } else {
                            acc[m][t] = S::mma(r.w[t], r.x[m], acc[m][t]);
                        }
                    }
            }
        }
        wait_loads<0>();                        // nothing lands in LDS any more
        v4f_t* mine = reinterpret_cast<v4f_t*>(ring[wave][0]);
#pragma unroll
        for (int m = 0; m < kRows; ++m)
#pragma unroll
            for (int t = 0; t < 2; ++t) mine[(m * 2 + t) * kWave + lane] = acc[m][t];
        __syncthreads();
        // one row tile a wave
        for (int m = wave; m < kRows; m += WAVES) {
            float r[2][4];
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                v4f_t v = reinterpret_cast<const v4f_t*>(ring[0][0])[(m * 2 + t) * kWave + lane];
#pragma unroll
                for (int o = 1; o < WAVES; ++o)
                    v += reinterpret_cast<const v4f_t*>(ring[o][0])[(m * 2 + t) * kWave + lane];
#pragma unroll
                for (int q = 0; q < 4; ++q) r[t][q] = v[q];
            }
            const int row = r0 + m * 16 + l16;
            if (m * 16 + l16 >= RP || row >= slot.rows) continue;
            silu_mul4(r[0], r[1], r[0]);
            if (g * 4 < left)                   // F is a multiple of 8
                store_h<F16>(static_cast<char*>(a.h) + (size_t)(slot.first + row) * layer_h_row(s.F), n0 + g * 4, r[0]);
        }
        if (r0 + RP < slot.rows) __syncthreads();            // before the rings are filled again
    }
}

// Dynamic LDS of down_kernel after its rings: sums [wave][token][column], the slots cut to RP rows,
// the rows' tokens and weights, scales [wave][2][64 units].
struct DownLds {
    size_t ring, sums, slots, rows, scales;
};
__host__ __device__ inline DownLds down_lds(const LayerShape& s, int waves, int stages, int cols, int rp)
{
    DownLds l;
    l.ring = (size_t)waves * stages;
    l.sums = (size_t)waves * s.T * cols * 4;
    l.slots = ((size_t)s.slots + (s.T > rp ? s.T * s.K / rp : 0)) * sizeof(Slot);
    l.rows = (size_t)s.T * s.K * sizeof(Row);
    l.scales = s.block ? (size_t)waves * 2 * kWave * 4 : 0;
    return l;
}

template <bool F16, bool BLOCK, int NT, int RP, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void down_kernel(LayerShape s, LayerArgs a)
{
    typedef Stage<F16, BLOCK, NT, RP, 2> S;
    constexpr int kCols = NT * 16;
    constexpr int kThreads = WAVES * kWave;
    extern __shared__ __align__(1024) char lds[];
    __shared__ int count_lds;
    const DownLds parts = down_lds(s, WAVES, kRing * S::kBytes, kCols, RP);
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int l16 = lane & 15, g = lane >> 4;
    char* ring = lds + (size_t)wave * kRing * S::kBytes;
    float* sums = reinterpret_cast<float*>(lds + parts.ring);
    Slot* slots = reinterpret_cast<Slot*>(lds + parts.ring + parts.sums);
    Row* rows = reinterpret_cast<Row*>(lds + parts.ring + parts.sums + parts.slots);
    float* scales = reinterpret_cast<float*>(lds + parts.ring + parts.sums + parts.slots + parts.rows) +
                    wave * 2 * kWave;
    // The first wave cuts the slots to at most RP rows each.
    if (wave == 0) {
        int count = 0;
        for (int i0 = 0; i0 < s.slots; i0 += kWave) {
            Slot slot = {-1, 0, 0, 0};
            if (i0 + lane < s.slots) slot = a.slots[i0 + lane];
            const int pieces = slot.expert < 0 ? 0 : (slot.rows + RP - 1) / RP;
            int upto = __popcll((unsigned long long)(__ballot(pieces > 0) & (~0ull >> (kWave - 1 - lane))));
            if (__ballot(pieces > 1) != 0) {
                upto = pieces;
#pragma unroll
                for (int off = 1; off < kWave; off <<= 1) {
                    const int o = __shfl_up(upto, off, kWave);
                    if (lane >= off) upto += o;
                }
            }
            for (int p = 0; p < pieces; ++p)
                slots[count + upto - pieces + p] = {slot.expert, slot.first + p * RP,
                                                    slot.rows - p * RP < RP ? slot.rows - p * RP : RP, 0};
            count += __builtin_amdgcn_readlane(upto, kWave - 1);
        }
        if (lane == 0) count_lds = count;
    }
    for (int i = threadIdx.x; i < s.T * s.K; i += kThreads) rows[i] = a.rows[i];
    for (int i = threadIdx.x; i < WAVES * s.T * kCols; i += kThreads) sums[i] = 0.0f;
    __syncthreads();
    const int count = __builtin_amdgcn_readfirstlane(count_lds);
    const char* h = static_cast<const char*>(a.h);
    const uint32_t row_bytes = (uint32_t)s.F * (BLOCK ? 1 : 2);
    const uint32_t h_bytes = (uint32_t)layer_h_row(s.F);
    const int chunks = (int)((row_bytes + 127) / 128);
    const int n0 = blockIdx.x * kCols;
    const int blocks = (s.H + 127) / 128;

    // Units (slot, chunk), one after another; a wave takes as many in a row as any other, so that it
    // seldom goes on to another slot.
    struct Place { int slot, chunk; };
    const auto step = [&](Place p) {
        if (++p.chunk == chunks) {
            p.chunk = 0;
            ++p.slot;
        }
        return p;
    };
    const int first = (int)((int64_t)count * chunks * wave / WAVES);
    const int units = (int)((int64_t)count * chunks * (wave + 1) / WAVES) - first;
    const auto slot_at = [&](int i) {
        Slot r;
        r.expert = __builtin_amdgcn_readfirstlane(slots[i].expert);
        r.first = __builtin_amdgcn_readfirstlane(slots[i].first);
        r.rows = __builtin_amdgcn_readfirstlane(slots[i].rows);
        return r;
    };
    const int rot = (int)(blockIdx.x * 3 % chunks);          // as in the up kernel
    const auto turn = [&](int c) { return c + rot >= chunks ? c + rot - chunks : c + rot; };
    Place ahead = {first / chunks, first % chunks};
    Slot next = {0, 0, 0, 0};
    int held = -1;                              // the slot that `next` describes
    int filled = 0;                             // fills asked for
    const auto fill = [&](int d) {
        if (filled++ >= units) return;
        if (held != ahead.slot) {
            next = slot_at(ahead.slot);
            held = ahead.slot;
        }
        __amdgpu_buffer_rsrc_t wr[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int left = s.H - n0 - t * 16 < 16 ? s.H - n0 - t * 16 : 16;
            wr[t] = make_rsrc(static_cast<const char*>(a.down) +
                                  ((size_t)next.expert * s.H + n0 + t * 16) * row_bytes,
                              left > 0 ? (uint32_t)left * row_bytes : 0);
        }
        const __amdgpu_buffer_rsrc_t hr =
            make_rsrc(h + (size_t)next.first * h_bytes, (uint32_t)next.rows * h_bytes);
        uint32_t xoff[S::kXLoads];
#pragma unroll
        for (int i = 0; i < S::kXLoads; ++i)
            xoff[i] = S::xrow(i) < RP ? (uint32_t)S::xrow(i) * h_bytes : kRsrcPastEnd;
        S::fill(ring + d * S::kBytes, wr, hr, row_bytes, xoff, turn(ahead.chunk));
        ahead = step(ahead);
    };
    // The scales of units 64 * batch + 0..63 of the wave, a lane each.
    const auto fetch_scales = [&](int batch) {
        const int unit = first + batch * kWave + lane;
        const int i = unit / chunks;
        const uint32_t off = i < count ? (uint32_t)(((size_t)slots[i].expert * blocks + n0 / 128) * chunks +
                                                    turn(unit - i * chunks)) * 4
                                       : kRsrcPastEnd;
        load_lds4(make_rsrc(a.down_scales, (uint32_t)s.E * blocks * chunks * 4),
                  reinterpret_cast<char*>(scales + (batch & 1) * kWave), off);
    };
    if (BLOCK) fetch_scales(0);
    v4f_t acc[S::kTiles][NT];
    const auto clear = [&]() {
#pragma unroll
        for (int m = 0; m < S::kTiles; ++m)
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[m][t] = v4f_t{0, 0, 0, 0};
    };
    clear();
    float* mine = sums + wave * s.T * kCols;
    // Adds an expert's sums, times the weights, to those of its tokens.
    const auto flush = [&](int i) {
        const Slot slot = slot_at(i);
#pragma unroll
        for (int m = 0; m < S::kTiles; ++m) {
            const int row = m * 16 + l16;
            if (row < slot.rows) {
                const Row r = rows[slot.first + row];
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    v4f_t* to = reinterpret_cast<v4f_t*>(mine + r.token * kCols + t * 16 + g * 4);
                    v4f_t sum = *to;
                    add_scaled(sum, acc[m][t], r.weight);
                    *to = sum;
                }
            }
        }
        clear();
    };
    Place now = ahead;
    int open = now.slot, unit = 0;
#pragma unroll
    for (int d = 0; d < kRing; ++d) fill(d);
    while (unit < units) {
#pragma unroll
        for (int d = 0; d < kRing; ++d) {
            if (unit >= units) break;
            typename S::Regs r;
            // no fetch is sent past the last unit (12.5 -> 12.0 us on a small layer, 164 -> 162 on a larger
            // one), and with none behind this unit's there is nothing to leave in flight
            if (unit + 1 < units) wait_loads<S::kLoads>();
            else wait_loads<0>();
            S::read(ring + d * S::kBytes, r);
            float sc = 0.0f;
            if (BLOCK) sc = scales[unit & (2 * kWave - 1)];
            wait_lds();
            if (BLOCK && (unit & (kWave - 1)) == 0) fetch_scales(unit / kWave + 1);
            fill(d);
            if (now.slot != open) {
                flush(open);
                open = now.slot;
            }
#pragma unroll
            for (int m = 0; m < S::kTiles; ++m)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    if constexpr (BLOCK)
                        add_scaled(acc[m][t], S::mma(r.w[t], r.x[m], v4f_t{0, 0, 0, 0}), sc);
                    else
                        acc[m][t] = S::mma(r.w[t], r.x[m], acc[m][t]);
                }
            now = step(now);
            ++unit;
        }
    }
    wait_loads<0>();                            // nothing lands in LDS any more
    if (units > 0) flush(open);
    __syncthreads();
    for (int i = threadIdx.x; i < s.T * kCols; i += kThreads) {
        const int t = i / kCols, n = n0 + i % kCols;
        if (n >= s.H) continue;
        float v = 0.0f;
#pragma unroll
        for (int o = 0; o < WAVES; ++o) v += sums[o * s.T * kCols + i];
        const size_t at = (size_t)t * s.H + n;
        if (s.id_end > s.zero_end)
            for (int k = 0; k < s.K; ++k) {
                const int id = a.ids[t * s.K + k];
                if (id >= s.zero_end && id < s.id_end && active(s, a, t, k))
                    v += a.weights[t * s.K + k] * tok_lo_rt(static_cast<const uint16_t*>(a.x)[at], F16);
            }
        if (a.shared) v += tok_lo_rt(static_cast<const uint16_t*>(a.shared)[at], F16);
        static_cast<uint16_t*>(a.y)[at] = (uint16_t)f32_to_tok_rt(v, F16);
    }
}

template <bool F16, bool BLOCK, int NT, int RP, int WAVES>
hipError_t launch_down(const LayerShape& s, const LayerArgs& a, hipStream_t stream)
{
    const DownLds l = down_lds(s, WAVES, kRing * Stage<F16, BLOCK, NT, RP, 2>::kBytes, NT * 16, RP);
    const size_t bytes = l.ring + l.sums + l.slots + l.rows + l.scales;
    down_kernel<F16, BLOCK, NT, RP, WAVES><<<(unsigned)((s.H + NT * 16 - 1) / (NT * 16)), WAVES * kWave, bytes,
                                             stream>>>(s, a);
    return hipGetLastError();
}

template <bool F16, bool BLOCK, int RP, int WAVES>
hipError_t launch_up(const LayerShape& s, const LayerArgs& a, hipStream_t stream)
{
    up_kernel<F16, BLOCK, RP, WAVES><<<dim3((unsigned)((s.F + 15) / 16), (unsigned)s.slots), WAVES * kWave,
                                       (size_t)s.T * s.K * 8, stream>>>(s, a);
    return hipGetLastError();
}

template <bool F16, bool BLOCK, int RP>
hipError_t launch_rows(const LayerShape& s, const LayerArgs& a, hipStream_t stream)
{
    const hipError_t e = (int64_t)s.slots * s.F <= kFewUp ? launch_up<F16, BLOCK, RP, 4>(s, a, stream)
                                                          : launch_up<F16, BLOCK, RP, 2>(s, a, stream);
    if (e != hipSuccess) return e;
    // The rings fit the 160 KB of LDS beside up to 62 KB of sums, slots and rows: with codes, whose chunks
    // meet 512 bytes of a row of h, fewer rows share a sweep.  16 columns and codes, eight rows with eight
    // waves against 16 with four, us: 2048 x 1024, 16 tokens on 16 experts 28.3 and 35.3; 4096 x 1024, 32
    // tokens on 32 experts 87.5 and 94.6, 64 on 64 186 and 186; but with more than 8 rows an expert in the mean,
    // 4096 x 4096, 64 tokens on 8 experts 129 and 121.
    constexpr int kRows = BLOCK && RP == 32 ? 16 : RP, kNarrowRows = BLOCK && RP == 16 ? 8 : kRows;
    constexpr bool kEight = 8 * kRing * Stage<F16, BLOCK, 1, kNarrowRows, 2>::kBytes <= 96 << 10;
    if (s.H >= kWideDown) return launch_down<F16, BLOCK, 2, kRows, 4>(s, a, stream);
    return launch_down<F16, BLOCK, 1, kNarrowRows, kEight ? 8 : 4>(s, a, stream);
}

template <bool F16, bool BLOCK>
hipError_t launch(const LayerShape& s, const LayerArgs& a, hipStream_t stream)
{
    // An expert's rows beyond RP read its weights again, from the caches.  TB/s of weights with uniform
    // experts, with one that every token picks and with weights of 1 / rank: 64 tokens on 256 experts x 7168 x
    // 2048 E4M3 (7, 64, 50 rows at most, four a sweep) 5.88, 5.75, 4.79, 32 tokens (5, 32, 24) 5.96, 5.83,
    // 5.18; 64 tokens on 64 experts bf16 (18, 64, 58, sixteen a sweep) 5.61, 5.74, 5.04.
    constexpr int kFew = BLOCK ? 4 : 8;         // rows that one load brings a chunk of
    if (s.T <= kFew || s.T * s.K <= 2 * s.E) return launch_rows<F16, BLOCK, kFew>(s, a, stream);
    if (s.T <= 16 || s.T * s.K <= 8 * s.E) return launch_rows<F16, BLOCK, 16>(s, a, stream);
    return launch_rows<F16, BLOCK, 32>(s, a, stream);
}

}  // namespace

hipError_t launch_experts_layer(const LayerShape& s, const LayerArgs& a, hipStream_t stream)
{
    if (s.tok_f16) return s.block ? launch<true, true>(s, a, stream) : launch<true, false>(s, a, stream);
    return s.block ? launch<false, true>(s, a, stream) : launch<false, false>(s, a, stream);
}

}  // namespace moe_dc
