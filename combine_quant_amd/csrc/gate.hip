// gate.hip -- the router: K best of n scores per token, with an optional group limit.
//
// The choice of an id (score + bias) is defined in binary64, where scores next to each other keep
// their order.  Two kernels:
//
// gate_scores_kernel (a bias, or groups measured by sums of scores): one wave per token forms the
// choices in binary64 and orders them through a 32-bit key of their binary32 rounding: rounding
// never reverses an order, so a key that is alone at the top is the best choice, found by one
// 32-bit wave maximum; only keys that tie are compared in binary64, then by id.  15.4 us for 8192
// tokens x 256 ids, K = 8, 8 groups (8.9 MB), 6.5 us for 2 tokens: bound by its instructions and,
// with few tokens, by one wave's latency.  (With the library's exponential, one lane to a group
// and the winner's id by a lane shuffle it took 18.3 and 8.3 us.  16 lanes a token need half the
// instructions but leave two waves a SIMD, which wait: with 4096 tokens 15.9 us against 10.8, with
// 8192 19.8 against 17.0 in one run, and only from 16384 on less, 25.6 against 29.3.)
//
// gate_logits_kernel (the logits themselves are compared, which is the order of the scores): the
// scores are needed only for the K chosen.  LANES lanes per token; each lane first sorts its
// DEPTH largest keys (its slot in a key's low bits), and a round takes the largest head among the
// lanes and moves the winner's list up; with tokens enough to fill the chip, one wave serves four
// tokens of 16 lanes each.  Keys that agree but for the slot bits are settled by the logits and
// ids of the K + 2 candidates, and if that is not enough (many equal logits) by the whole wave in
// a plain loop.  16384 tokens x 516 ids, K = 16 (34 MB): 33 us, against 54 us by the first
// kernel.
#include "experts_internal.h"
#include "dc_device.h"
#include "gate_math.h"

namespace moe_dc {
namespace {

constexpr int kGateWaves = 4;
constexpr int kGateMaxIds = 2048;
// Tokens from which a wave serves four; below, the waves are too few for the CUs.  With a wave
// each and with four to a wave: 2048 x 256, K = 8, 8.4 and 9.4 us, 4096 x 256 11.5 and 9.8; 2048 x
// 516, K = 16, 13.5 and 16.6, 4096 x 516 19.8 and 18.6, 16384 x 516 50 and 31.
constexpr int kGateQuarterTokens = 4096;
// Order-preserving keys: 0 is kept for ids out of play, 1 for NaN.
__device__ __forceinline__ uint32_t choice_key(float f)
{
    const uint32_t u = __float_as_uint(f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 1u;
    if (u == 0x80000000u) return 0x80000000u;             // -0 equals +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_choice(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

// 1 / (1 + e^-z) as (1 or t) / (1 + t) with t = e^-|z|: the divisor lies in [1, 2], so its
// reciprocal needs no scaling; two Newton steps, and one on the quotient.
__device__ __forceinline__ double sigmoid(double z)
{
    const double t = exp_below(-__builtin_fabs(z));
    const double d = 1.0 + t, num = z < 0.0 ? t : 1.0;
    double y = __builtin_amdgcn_rcp(d);
    y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
    y = __builtin_fma(__builtin_fma(-d, y, 1.0), y, y);
    const double q = num * y;
    return __builtin_fma(__builtin_fma(-d, q, num), y, q);
}

template <int LANES, typename T>
__device__ __forceinline__ T group_sum(T v)
{
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}
template <int LANES>
__device__ __forceinline__ float group_max(float v)
{
#pragma unroll
    for (int off = LANES / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor(v, off, kWave));
    return v;
}

__device__ __forceinline__ double fine_score(const GateShape& s, float z, double peak, double total)
{
    if (s.sigmoid) return sigmoid((double)z);
    return peak > -INFINITY ? exp_below((double)z - peak) / total : 0.0;
}

// a is chosen before b: the larger one, NaN last, then the lower id.
__device__ __forceinline__ bool precedes(float a, int ia, float b, int ib)
{
    if (a != a || b != b) return a == a || (b != b && ia < ib);
    return a > b || (a == b && ia < ib);
}

// One token by the whole wave.  Returns the lane's choice (lane k < K: the k-th id).
__device__ __noinline__ int plain_token(const GateShape& s, const float* __restrict__ z, uint64_t kept,
                                        int shift)
{
    const int lane = threadIdx.x & (kWave - 1);
    uint32_t out = 0;                                      // the lane's ids that are out of play
    if (s.groups > 1)
        for (int i = 0, id = lane; id < s.n; ++i, id += kWave)
            if (!((kept >> (s.group_of(id) << shift)) & 1)) out |= 1u << i;
    int chosen = 0;
    for (int k = 0; k < s.K; ++k) {
        float best = 0.0f;
        int at = kGateMaxIds;
        for (int i = 0, id = lane; id < s.n; ++i, id += kWave) {
            const float v = z[id];
            if (!((out >> i) & 1) && (at == kGateMaxIds || precedes(v, id, best, at))) {
                best = v;
                at = id;
            }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
            const float ov = __shfl_xor(best, off, kWave);
            const int oi = __shfl_xor(at, off, kWave);
            if (oi != kGateMaxIds && (at == kGateMaxIds || precedes(ov, oi, best, at))) {
                best = ov;
                at = oi;
            }
        }
        if ((at & (kWave - 1)) == lane) out |= 1u << (at / kWave);
        if (lane == k) chosen = at;
    }
    return chosen;
}

// Slots of a lane are held in the low kSlotBits bits of its keys.
constexpr int slot_bits(int ch) { return ch <= 4 ? 2 : ch <= 8 ? 3 : ch <= 16 ? 4 : ch <= 32 ? 5 : 6; }

// CH: ids per lane: lane l of a token's LANES holds ids l + LANES * i.  DEPTH: keys a lane sorts
// at a time.
template <int LANES, int CH, int DEPTH>
__global__ __launch_bounds__(kGateWaves * kWave) void gate_logits_kernel(
    GateShape s, const float* __restrict__ logits, int32_t* __restrict__ expert_ids,
    float* __restrict__ expert_scales)
{
    extern __shared__ float lds[];                         // [waves][tokens][n]
    constexpr int kTokens = kWave / LANES;                 // per wave
    constexpr uint32_t kSlots = (1u << slot_bits(CH)) - 1;
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = threadIdx.x / kWave;
    const int sub = lane / LANES, l = lane % LANES;
    const int token0 = (blockIdx.x * kGateWaves + wave) * kTokens;
    if (token0 >= s.tokens) return;                        // no workgroup barrier below
    const int token = token0 + sub < s.tokens ? token0 + sub : token0;
    const bool live = token0 + sub < s.tokens;
    const float* z = logits + (size_t)token * s.n;
    float* mem = lds + (size_t)wave * kTokens * s.n;
    const auto id_of = [&](int i) { return l + i * LANES; };
    const uint64_t tokens_lanes = LANES == kWave ? ~0ull : ((1ull << (LANES & 63)) - 1) << (sub * LANES);

    float v[CH];
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        v[i] = id_of(i) < s.n ? z[id_of(i)] : -INFINITY;
        top = fmaxf(top, v[i]);
    }
    double total = 1.0, peak = 0.0;
    if (!s.sigmoid) {
        top = group_max<LANES>(top);
        peak = top;
        double part = 0.0;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (id_of(i) < s.n && top > -INFINITY)
                part += exp2_fine(((double)v[i] - peak) * 1.4426950408889634);
        total = group_sum<LANES>(part);
    }

    bool again = false;                                    // the token needs the plain loop
    uint64_t kept = ~0ull;                                 // group g: bit g << shift
    int shift = 0;
    const int size = s.n / s.groups;
    if (s.groups > 1) {
        // A group's value is its largest logit (group_top 1), NaN without one, as a key, since
        // NaN ranks below -infinity; 2^shift lanes share a group.  A group counts the groups
        // ahead of it and the keep first ones stay.
        float* mine = mem + sub * s.n;
#pragma unroll
        for (int i = 0; i < CH; ++i)
            if (id_of(i) < s.n) mine[id_of(i)] = v[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        while ((s.groups << (shift + 1)) <= LANES) ++shift;
        const int share = 1 << shift, group = l >> shift;
        float value = NAN;                                 // (fmaxf leaves NaN out)
        if (group < s.groups)
#pragma unroll 8
            for (int i = l & (share - 1); i < size; i += share)
                value = fmaxf(value, mine[group * size + i]);
        for (int off = 1; off < share; off <<= 1) value = fmaxf(value, __shfl_xor(value, off, kWave));
        const uint32_t rank = choice_key(value);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (group < s.groups) mine[group] = __uint_as_float(rank);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        int ahead = 0;
#pragma unroll 8
        for (int g = 0; g < s.groups; ++g) {
            const uint32_t other = __float_as_uint(mine[g]);
            if (other > rank || (other == rank && g < group)) ++ahead;
        }
        kept = __ballot(group < s.groups && ahead < s.keep);
        if (LANES != kWave) kept = (kept >> (sub * LANES)) & ((1ull << (LANES & 63)) - 1);
    }

#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int id = id_of(i);
        bool in = id < s.n;
        if (s.groups > 1) in = in && ((kept >> (s.group_of(id) << shift)) & 1);
        again |= in && v[i] != v[i];
        // (a number's key has bit 31 or bits of 23-30 set, so clearing low bits leaves it in
        // play)
        const uint32_t k = in ? (choice_key(v[i]) & ~kSlots) | (uint32_t)(kSlots - i) : 0u;
        v[i] = __uint_as_float(k);
    }
    // The lane's DEPTH largest keys below `limit`, largest first.
    uint32_t head[DEPTH];
    const auto sort_heads = [&](uint32_t limit) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) head[d] = 0u;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            uint32_t k = __float_as_uint(v[i]);
            k = k < limit ? k : 0u;
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                const uint32_t hi = head[d] > k ? head[d] : k;
                k = head[d] > k ? k : head[d];
                head[d] = hi;
            }
        }
    };
    sort_heads(0xFFFFFFFFu);

    int my_id = 0;                                         // lane k < K: the k-th choice
    int spare = -1;                                        // the next one, in every lane
    bool doubt = false;                                    // the order of the K
    bool edge = false, far_edge = false;                   // K or K + 1 against the next one
    float before = 0.0f;
    int held = DEPTH;                                      // keys left in the lane's list
    const int rounds = s.K + 2;
    for (int k = 0; k < rounds; ++k) {
        const uint32_t m = LANES == kWave ? wave_max_u32(head[0]) : group_max_u32<LANES>(head[0]);
        const uint64_t who = __ballot(head[0] == m) & tokens_lanes;
        const int winner = __ffsll((unsigned long long)who) - 1;
        const float now = key_choice(m & ~kSlots);
        const bool any = m != 0u;                          // fewer ids than rounds
        if (k > 0 && any) {
            const bool c = !(before > now);
            if (k < s.K) doubt |= c;
            if (k == s.K) edge = c;
            if (k == s.K + 1) far_edge = c;
        }
        before = now;
        const int id = (winner & (LANES - 1)) + (int)(kSlots - (m & kSlots)) * LANES;
        if (l == k && k < s.K) my_id = id;
        if (k == s.K && any) spare = id;
        if (lane == winner) {
#pragma unroll
            for (int d = 0; d + 1 < DEPTH; ++d) head[d] = head[d + 1];
            head[DEPTH - 1] = 0u;
            --held;
        }
        if (CH > DEPTH && __ballot(held == 0)) {
            const uint32_t limit = m;
            if (held == 0) {
                sort_heads(limit);
                held = DEPTH;
            }
        }
    }
    again |= edge && far_edge;
    const uint64_t redo = __ballot(again);
    const bool redone = (redo & tokens_lanes) != 0;
    if (redo) {
#pragma unroll
        for (int t = 0; t < kTokens; ++t) {
            const uint64_t lanes = LANES == kWave ? ~0ull : ((1ull << (LANES & 63)) - 1) << (t * LANES);
            if (!(redo & lanes) || token0 + t >= s.tokens) continue;
            const int chosen = plain_token(s, logits + (size_t)(token0 + t) * s.n,
                                           __shfl((unsigned long long)kept, t * LANES, kWave), shift);
            const int got = __shfl(chosen, l, kWave);
            if (sub == t) my_id = got;
        }
    }
    int place = l;
    if (__ballot((doubt || edge) && !redone)) {
        float mine = l < s.K ? z[my_id] : 0.0f;
        const auto rank = [&]() {
            int ahead = 0;
            for (int k = 0; k < s.K; ++k) {
                const float other = __shfl(mine, sub * LANES + k, kWave);
                const int oid = __shfl(my_id, sub * LANES + k, kWave);
                if (precedes(other, oid, mine, my_id)) ++ahead;
            }
            return ahead;
        };
        int ahead = rank();
        if (__ballot(edge && !redone)) {
            // the spare candidate takes the place of the last one if it precedes it
            const float other = spare < 0 ? 0.0f : z[spare];
            if (!redone && edge && spare >= 0 && l < s.K && ahead == s.K - 1 &&
                precedes(other, spare, mine, my_id)) {
                my_id = spare;
                mine = other;
            }
            ahead = rank();
        }
        if (!redone) place = ahead;
    }
    const double score = l < s.K ? fine_score(s, z[my_id], peak, total) : 0.0;
    double weight = score;
    if (s.renormalize) weight = weight / (group_sum<LANES>(score) + 1e-20);
    if (l < s.K && live) {
        expert_ids[(size_t)token * s.K + place] = my_id;
        expert_scales[(size_t)token * s.K + place] = (float)(weight * (double)s.factor);
    }
}

__device__ __forceinline__ double wave_sum(double v)
{
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, kWave);
    return v;
}

// CH: ids per lane.  WIDE: choices are binary64 values (a bias was added); otherwise logits, and
// groups are measured by the sum of their two best scores.
template <int CH, bool WIDE>
__global__ __launch_bounds__(kGateWaves * kWave) void gate_scores_kernel(
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
    double c[CH];                                          // scores; WIDE: the choices
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
        for (int i = 0; i < CH; ++i) {
            c[i] = 0.0;
            if (lane + i * kWave < s.n && top > -INFINITY) c[i] = exp_below((double)v[i] - peak);
            part += c[i];
        }
        total = wave_sum(part);
        const double inverse = top > -INFINITY ? 1.0 / total : 0.0;
#pragma unroll
        for (int i = 0; i < CH; ++i) c[i] *= inverse;
    } else {
#pragma unroll
        for (int i = 0; i < CH; ++i) c[i] = lane + i * kWave < s.n ? sigmoid((double)v[i]) : 0.0;
    }
#pragma unroll
    for (int i = 0; i < CH; ++i) {
        const int id = lane + i * kWave;
        if (WIDE && id < s.n) c[i] += (double)bias[id];
        key[i] = id < s.n ? choice_key(WIDE ? (float)c[i] : v[i]) : 0u;
    }

    if (s.groups > 1) {
        // A group's value from its group_top best choices, 2^shift lanes sharing a group; then
        // each group counts the groups ahead of it and the keep first ones stay.  NaN ranks below
        // -infinity, as a choice and as a value: here -infinity is kLow, below every finite
        // choice, and NaN -infinity.
        constexpr double kLow = -1e300;
        const int size = s.n / s.groups;
        double* mine = group_lds + (size_t)wave * s.n;
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int id = lane + i * kWave;
            if (id < s.n) mine[id] = c[i] == c[i] ? fmax(c[i], kLow) : -INFINITY;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        int shift = 0;
        while ((s.groups << (shift + 1)) <= kWave) ++shift;
        const int share = 1 << shift, group = lane >> shift;
        double a = -INFINITY, b = -INFINITY;
        if (group < s.groups)
#pragma unroll 4
            for (int j = lane & (share - 1); j < size; j += share) {
                const double w = mine[group * size + j];
                b = fmax(b, fmin(a, w));
                a = fmax(a, w);
            }
        for (int off = 1; off < share; off <<= 1) {
            const double oa = __shfl_xor(a, off, kWave), ob = __shfl_xor(b, off, kWave);
            b = fmax(fmin(a, oa), fmax(b, ob));
            a = fmax(a, oa);
        }
        const double last = s.top == 2 ? b : a;
        double value = s.top == 2 ? a + b : a;
        if (!(last > kLow)) value = last == kLow && a < INFINITY ? kLow : -INFINITY;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (group < s.groups) mine[group] = value;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        int ahead = 0;
#pragma unroll 8
        for (int g = 0; g < s.groups; ++g) {
            const double other = mine[g];
            if (other > value || (other == value && g < group)) ++ahead;
        }
        const uint64_t kept = __ballot(group < s.groups && ahead < s.keep);
#pragma unroll
        for (int i = 0; i < CH; ++i) {
            const int id = lane + i * kWave;
            if (id < s.n && !((kept >> (s.group_of(id) << shift)) & 1)) key[i] = 0u;
        }
    }

    int my_id = 0;                                         // lane k < K: the k-th choice
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
        winner = __builtin_amdgcn_readfirstlane(winner);
        const int id = lane_value(lane + slot * kWave, winner);
        if (lane == k) my_id = id;
        if (lane == winner) {
#pragma unroll
            for (int i = 0; i < CH; ++i)
                if (i == slot) key[i] = 0u;
        }
    }
    // The K scores, one per lane.
    double w = lane < s.K ? fine_score(s, z[my_id], peak, total) : 0.0;
    if (s.renormalize) w = w / (wave_sum(w) + 1e-20);
    if (lane < s.K) {
        expert_ids[(size_t)token * s.K + lane] = my_id;
        expert_scales[(size_t)token * s.K + lane] = (float)(w * (double)s.factor);
    }
}

template <int LANES, int CH, int DEPTH>
hipError_t launch_logits(const GateShape& s, const float* logits, int32_t* ids, float* scales,
                         hipStream_t stream)
{
    constexpr int kTokens = kWave / LANES;
    const dim3 grid((s.tokens + kGateWaves * kTokens - 1) / (kGateWaves * kTokens));
    const size_t lds = s.groups > 1 ? sizeof(float) * kGateWaves * kTokens * s.n : 0;
    gate_logits_kernel<LANES, CH, DEPTH><<<grid, kGateWaves * kWave, lds, stream>>>(s, logits, ids, scales);
    return hipGetLastError();
}

template <int LANES, int CH>
hipError_t launch_depth(const GateShape& s, const float* logits, int32_t* ids, float* scales,
                        hipStream_t stream)
{
    // A list that runs out is sorted anew: with four keys in 0.2 % of the tokens for K = 8, with
    // six in 0.1 % for K = 16.
    if (CH <= 4 || s.K <= 8) return launch_logits<LANES, CH, 4>(s, logits, ids, scales, stream);
    return launch_logits<LANES, CH, 6>(s, logits, ids, scales, stream);
}

template <int CH>
hipError_t launch_scores(const GateShape& s, const float* logits, const float* bias, int32_t* ids,
                         float* scales, hipStream_t stream)
{
    const dim3 grid((s.tokens + kGateWaves - 1) / kGateWaves), block(kGateWaves * kWave);
    const size_t lds = s.groups > 1 ? (size_t)kGateWaves * s.n * sizeof(double) : 0;
    if (bias)
        gate_scores_kernel<CH, true><<<grid, block, lds, stream>>>(s, logits, bias, ids, scales);
    else
        gate_scores_kernel<CH, false><<<grid, block, lds, stream>>>(s, logits, bias, ids, scales);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gate_topk(const GateShape& s, const float* logits, const float* bias,
                            int32_t* expert_ids, float* expert_scales, hipStream_t stream)
{
    static_assert(kGateWaves * kGateMaxIds * sizeof(double) <= 65536, "LDS of a workgroup");
    // An id more than a kernel holds takes the next one, of more ids per lane: 8192 tokens with a
    // bias, K = 8, 256 ids 12.1 us, 257 17.1, 640 21.6, 641 26.4, 1024 30.9, 1025 45.2; without,
    // K = 16, 576 20.8 (16 lanes a token), 577 29.8 (64); 128 tokens 256 6.8, 257 8.4, 1025 11.4.
    // 640 and 576 leave room for special ids beside 512 experts.
    if (bias || (s.groups > 1 && s.top == 2)) {
        if (s.n <= 256) return launch_scores<4>(s, logits, bias, expert_ids, expert_scales, stream);
        if (s.n <= 640) return launch_scores<10>(s, logits, bias, expert_ids, expert_scales, stream);
        if (s.n <= 1024) return launch_scores<16>(s, logits, bias, expert_ids, expert_scales, stream);
        return launch_scores<32>(s, logits, bias, expert_ids, expert_scales, stream);
    }
    if (s.tokens >= kGateQuarterTokens && s.groups <= 16) {      // (a lane or more per group)
        if (s.n <= 256) return launch_depth<16, 16>(s, logits, expert_ids, expert_scales, stream);
        if (s.n <= 576) return launch_depth<16, 36>(s, logits, expert_ids, expert_scales, stream);
    }
    if (s.n <= 256) return launch_depth<64, 4>(s, logits, expert_ids, expert_scales, stream);
    if (s.n <= 1024) return launch_depth<64, 16>(s, logits, expert_ids, expert_scales, stream);
    return launch_depth<64, 32>(s, logits, expert_ids, expert_scales, stream);
}

}  // namespace moe_dc
