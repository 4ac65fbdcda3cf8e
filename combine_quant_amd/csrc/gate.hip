// gate.hip -- the router: K best of n scores per token, with an optional group limit.
//
// One wave per token; lane l holds ids l, l + 64, ...  The choice of an id (score + bias) is
// formed in binary64 and ordered through a 32-bit key of its binary32 rounding: rounding never
// reverses an order, so a key that is alone at the top is the best choice, found by one 32-bit
// wave maximum; only keys that tie are compared in binary64, then by id.  Without a bias the
// logits are the choices (score rises with them) and the keys are exact.
#include "experts_internal.h"
#include "dc_device.h"

namespace moe_dc {
namespace {

constexpr int kGateWaves = 4;             // tokens per workgroup
constexpr int kGateMaxIds = 2048;

// Order-preserving keys: 0 is kept for ids out of play, 1 for NaN.
__device__ __forceinline__ uint32_t choice_key(float f)
{
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
    if (u == 0x80000000u) return 0x80000000u;             // -0 equals +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// CH: ids per lane.  WIDE: choices are binary64 values (a bias was added); otherwise logits.
template <int CH, bool WIDE>
__global__ __launch_bounds__(kGateWaves * kWave) void gate_kernel(
    GateShape s, const float* __restrict__ logits, const float* __restrict__ bias,
    int32_t* __restrict__ expert_ids, float* __restrict__ expert_scales)
{
    extern __shared__ double group_lds[];                  // [waves][n], with a group limit only
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int token = blockIdx.x * kGateWaves + wave;
    if (token >= s.tokens) return;                         // no workgroup barrier below
    const float* z = logits + (size_t)token * s.n;

    float v[CH];
    uint32_t key[CH];
    double c[CH];                                          // WIDE: the choices
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int id = lane + i * kWave;
        v[i] = id < s.n ? z[id] : -INFINITY;
        top = fmaxf(top, v[i]);
    }
    double total = 1.0;
    double peak = 0.0;
    if (!s.sigmoid) {
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, kWave));
        peak = top;
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (lane + i * kWave < s.n && top > -INFINITY) part += exp((double)v[i] - peak);
        total = wave_sum(part);
    }
    const auto score = [&](float x) -> double {
        if (s.sigmoid) return 1.0 / (1.0 + exp(-(double)x));
        return top > -INFINITY ? exp((double)x - peak) / total : 0.0;
    };
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int id = lane + i * kWave;
        c[i] = 0.0;
        if (WIDE && id < s.n) c[i] = score(v[i]) + (double)bias[id];
        key[i] = id < s.n ? choice_key(WIDE ? (float)c[i] : v[i]) : 0u;
    }

    if (s.groups > 1) {
        // A group's value from its group_top best choices, one group per lane; then each group
        // counts the groups ahead of it and the keep first ones stay.
        const int size = s.n / s.groups;
        double* mine = group_lds + (size_t)wave * s.n;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int id = lane + i * kWave;
            if (id < s.n) mine[id] = WIDE ? c[i] : s.top == 2 ? score(v[i]) : (double)v[i];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        double value = -INFINITY;
        if (lane < s.groups) {
            double a = -INFINITY, b = -INFINITY;
            for (int j = 0; j < size; ++j) {
                const double w = mine[lane * size + j];
                if (w > a) {
                    b = a;
                    a = w;
                } else if (w > b) {
                    b = w;
                }
            }
            value = s.top == 2 ? a + b : a;
        }
        int ahead = 0;
        for (int g = 0; g < s.groups; ++g) {
            const double other = __shfl(value, g, kWave);
            if (other > value || (other == value && g < lane)) ++ahead;
        }
        const uint64_t kept = __ballot(lane < s.groups && ahead < s.keep);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int id = lane + i * kWave;
            if (id < s.n && !((kept >> (id / size)) & 1)) key[i] = 0u;
        }
    }

    int my_id = 0;               // lane k < K: the k-th choice and its score
    double my_score = 0.0;
    for (int k = 0; k < s.K; ++k) {
        uint32_t best = 0;
#pragma unroll
        for (int i = 0; i < CH; ++i) best = best > key[i] ? best : key[i];
        const uint32_t m = wave_max_u32(best);
        int hits = 0, slot = 0;
#pragma unroll
        for (int i = CH - 1; i >= 0; --i)
            if (key[i] == m) {
                ++hits;
                slot = i;
            }
        uint64_t who = __ballot(hits > 0);
        int winner = __ffsll((unsigned long long)who) - 1;
        if (__popcll(who) > 1 || __ballot(hits > 1)) {
            // Tied keys: the largest binary64 choice (WIDE), then the lowest id.
            double d = -INFINITY;
            int id = 1 << 30;
            if (hits > 0) {
#pragma unroll
                for (int i = 0; i < CH; ++i) {
                    if (key[i] != m) continue;
                    const double w = WIDE && m > 1u ? c[i] : 0.0;
                    if (id == (1 << 30) || w > d) {
                        d = w;
                        id = lane + i * kWave;
                        slot = i;
                    }
                }
            }
            double bd = d;
            int bid = id;
#pragma unroll
            for (int off = 32; off > 0; off >>= 1) {
                const double od = __shfl_xor(bd, off, kWave);
                const int oid = __shfl_xor(bid, off, kWave);
                if (oid != (1 << 30) && (bid == (1 << 30) || od > bd || (od == bd && oid < bid))) {
                    bd = od;
                    bid = oid;
                }
            }
            winner = bid & (kWave - 1);
        }
        float x = 0.0f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (i == slot) {
                x = v[i];
                if (lane == winner) key[i] = 0u;
            }
        const int id = __shfl(lane + slot * kWave, winner, kWave);
        const float xw = __shfl(x, winner, kWave);
        if (lane == k) {
            my_id = id;
            my_score = (double)xw;
        }
    }
    // The K scores, one per lane.
    double w = lane < s.K ? score((float)my_score) : 0.0;
    if (s.renormalize) w = w / (wave_sum(w) + 1e-20);
    if (lane < s.K) {
        expert_ids[(size_t)token * s.K + lane] = my_id;
        expert_scales[(size_t)token * s.K + lane] = (float)(w * (double)s.factor);
    }
}

template <int CH>
hipError_t launch_ch(const GateShape& s, const float* logits, const float* bias, int32_t* ids,
                     float* scales, hipStream_t stream)
{
    const dim3 grid((s.tokens + kGateWaves - 1) / kGateWaves), block(kGateWaves * kWave);
    const size_t lds = s.groups > 1 ? (size_t)kGateWaves * s.n * sizeof(double) : 0;
    if (bias)
        gate_kernel<CH, true><<<grid, block, lds, stream>>>(s, logits, bias, ids, scales);
    else
        gate_kernel<CH, false><<<grid, block, lds, stream>>>(s, logits, bias, ids, scales);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gate_topk(const GateShape& s, const float* logits, const float* bias,
                            int32_t* expert_ids, float* expert_scales, hipStream_t stream)
{
    static_assert(kGateWaves * kGateMaxIds * sizeof(double) <= 65536, "LDS of a workgroup");
    if (s.n <= 4 * kWave) return launch_ch<4>(s, logits, bias, expert_ids, expert_scales, stream);
    if (s.n <= 10 * kWave) return launch_ch<10>(s, logits, bias, expert_ids, expert_scales, stream);
    if (s.n <= 16 * kWave) return launch_ch<16>(s, logits, bias, expert_ids, expert_scales, stream);
    return launch_ch<32>(s, logits, bias, expert_ids, expert_scales, stream);
}

}  // namespace moe_dc
