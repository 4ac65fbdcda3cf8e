// experts_api.cpp -- C ABI of the router and the experts' products: host validation and launch.
//
// As in api.cpp, nothing here allocates device memory or synchronises the host; each call is
// one kernel on the caller's stream.
#include "moe_dc.h"
#include "experts_internal.h"

#include <cmath>
#include <cstdarg>
#include <cstdio>

namespace {

using moe_dc::MatmulArgs;
using moe_dc::MatmulShape;

moe_status fail(moe_status st, const char* fmt, ...)
{
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return moe_dc::set_error(st, buf);
}

moe_status launched(hipError_t e, const char* what)
{
    if (e != hipSuccess) return fail(MOE_ERR_DEVICE, "%s: %s", what, hipGetErrorString(e));
    return moe_dc::set_ok();
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Whether two ranges of bytes share any (a NULL one shares none).
bool overlap(const void* p, int64_t n, const void* q, int64_t m)
{
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return p && q && (a < b ? b - a < (uintptr_t)n : a - b < (uintptr_t)m);
}

// The rows that a product may touch.
int64_t touched(const MatmulShape& s) { return s.rows < s.cap ? s.rows : s.cap; }

// The output of a product against everything that it reads, in bytes.
moe_status check_overlap(const MatmulShape& s, const MatmulArgs& a, int64_t x, int64_t x_scales,
                         int64_t w, int64_t w_scales)
{
    const int64_t out = touched(s) * (s.swiglu ? s.out / 2 : s.out) * 2;
    const int64_t counts = (int64_t)s.E * s.W * 4, offsets = (int64_t)(s.W + 1) * 8;
    if (overlap(a.out, out, a.x, x) || overlap(a.out, out, a.x_scales, x_scales) ||
        overlap(a.out, out, a.w, w) || overlap(a.out, out, a.w_scales, w_scales) ||
        overlap(a.out, out, a.ep_recv_count, counts) || overlap(a.out, out, a.recv_offsets, offsets))
        return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
    return MOE_OK;
}

// The rules the two products share: the config, the sizes and the activation.
moe_status check_matmul(const moe_dc_config* cfg, const moe_matmul* mm, MatmulShape* s)
{
    moe_dc::Shape sh;
    moe_status st = moe_dc::check_config(cfg, &sh);
    if (st != MOE_OK) return st;
    if (!mm) return fail(MOE_ERR_INVALID_ARG, "matmul description is NULL");
    if (mm->in_features < 1 || mm->in_features > 65536)
        return fail(MOE_ERR_INVALID_ARG, "in_features %d outside [1, 65536]", mm->in_features);
    if (mm->out_features < 1 || mm->out_features > 65536)
        return fail(MOE_ERR_INVALID_ARG, "out_features %d outside [1, 65536]", mm->out_features);
    if (mm->activation != MOE_ACT_NONE && mm->activation != MOE_ACT_SWIGLU)
        return fail(MOE_ERR_INVALID_ARG, "activation %d is not one of 0 (none), 1 (SwiGLU)",
                    mm->activation);
    if (mm->activation == MOE_ACT_SWIGLU && mm->out_features % 2 != 0)
        return fail(MOE_ERR_INVALID_ARG, "SwiGLU needs an even out_features, got %d",
                    mm->out_features);
    if (mm->reserved != 0) return fail(MOE_ERR_INVALID_ARG, "reserved must be 0");
    s->W = sh.W;
    s->E = sh.E;
    s->L = sh.L;
    s->in = mm->in_features;
    s->out = mm->out_features;
    s->swiglu = mm->activation == MOE_ACT_SWIGLU ? 1 : 0;
    s->tok_f16 = sh.tok_f16;
    s->type = sh.tok_f16 ? moe_dc::kMmF16 : moe_dc::kMmBf16;
    s->w4 = 0;
    s->group = 0;
    s->rows = (int64_t)sh.W * sh.BS * sh.K;
    s->cap = sh.cap;
    return MOE_OK;
}

hipError_t launch_grouped_matmul(const MatmulShape& s, const MatmulArgs& a, hipStream_t stream)
{
    switch (s.type) {
    case moe_dc::kMmBf16: return moe_dc::launch_grouped_bf16(s, a, stream);
    case moe_dc::kMmF16: return moe_dc::launch_grouped_f16(s, a, stream);
    case moe_dc::kMmInt8: return moe_dc::launch_grouped_int8(s, a, stream);
    case moe_dc::kMmE4m3: return moe_dc::launch_grouped_e4m3(s, a, stream);
    case moe_dc::kMmE5m2: return moe_dc::launch_grouped_e5m2(s, a, stream);
    case moe_dc::kMmMxE4m3: return moe_dc::launch_grouped_mxe4m3(s, a, stream);
    default: return moe_dc::launch_grouped_mxe5m2(s, a, stream);
    }
}

moe_status check_pointers(const MatmulArgs& a)
{
    if (!a.x || !a.w || !a.ep_recv_count || !a.recv_offsets || !a.out)
        return fail(MOE_ERR_INVALID_ARG, "a required tensor pointer is NULL");
    if (!aligned(a.x, 16) || !aligned(a.w, 16))
        return fail(MOE_ERR_INVALID_ARG, "x and weight must be 16-byte aligned");
    return MOE_OK;
}

}  // namespace

extern "C" {

moe_status moe_grouped_matmul(const moe_dc_config* cfg, const moe_matmul* mm, const void* x,
                              const void* x_scales, const void* weight,
                              const void* weight_scales, const int32_t* ep_recv_count,
                              const int64_t* recv_offsets, void* out, void* stream)
{
    MatmulShape s;
    moe_status st = check_matmul(cfg, mm, &s);
    if (st != MOE_OK) return st;
    if (mm->weight_dtype != 0 || mm->group_size != 0)
        return fail(MOE_ERR_INVALID_ARG, "weight_dtype and group_size belong to the 4-bit product");
    if (mm->scaling < MOE_MM_SCALE_NONE || mm->scaling > MOE_MM_SCALE_MX)
        return fail(MOE_ERR_INVALID_ARG, "scaling %d is not one of 0..2", mm->scaling);
    const bool codes = mm->x_dtype != MOE_DTYPE_DEFAULT;
    int32_t step = 8;
    switch (mm->x_dtype) {
    case MOE_DTYPE_DEFAULT:
        if (mm->scaling != MOE_MM_SCALE_NONE)
            return fail(MOE_ERR_INVALID_ARG, "token rows take no scales (scaling %d)", mm->scaling);
        break;
    case MOE_DTYPE_INT8:
        if (mm->scaling != MOE_MM_SCALE_ROW)
            return fail(MOE_ERR_INVALID_ARG, "int8 rows need scaling MOE_MM_SCALE_ROW");
        s.type = moe_dc::kMmInt8;
        step = 16;
        break;
    case MOE_DTYPE_E4M3:
    case MOE_DTYPE_E5M2:
        if (mm->scaling == MOE_MM_SCALE_NONE)
            return fail(MOE_ERR_INVALID_ARG, "fp8 rows need scaling MOE_MM_SCALE_ROW or _MX");
        if (mm->scaling == MOE_MM_SCALE_ROW) {
            s.type = mm->x_dtype == MOE_DTYPE_E4M3 ? moe_dc::kMmE4m3 : moe_dc::kMmE5m2;
            step = 16;
        } else {
            s.type = mm->x_dtype == MOE_DTYPE_E4M3 ? moe_dc::kMmMxE4m3 : moe_dc::kMmMxE5m2;
            step = 128;
        }
        break;
    case MOE_DTYPE_E2M1:
        return fail(MOE_ERR_UNSUPPORTED, "E2M1 rows are not supported");
    default:
        return fail(MOE_ERR_INVALID_ARG, "x_dtype %d is not a moe_dtype", mm->x_dtype);
    }
    if (s.in % step != 0)
        return fail(MOE_ERR_INVALID_ARG, "in_features %d must be a multiple of %d for these rows",
                    s.in, step);
    const MatmulArgs a{x, x_scales, weight, weight_scales, ep_recv_count, recv_offsets, out};
    st = check_pointers(a);
    if (st != MOE_OK) return st;
    if (!codes && (x_scales || weight_scales))
        return fail(MOE_ERR_INVALID_ARG, "token rows take no x_scales or weight_scales");
    if (codes && !weight_scales)
        return fail(MOE_ERR_INVALID_ARG, "weight_scales is required for scaling %d", mm->scaling);
    if (mm->scaling == MOE_MM_SCALE_MX && !x_scales)
        return fail(MOE_ERR_INVALID_ARG, "x_scales is required for MX rows");
    if (!aligned(x_scales, 4) || !aligned(weight_scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "x_scales and weight_scales must be 4-byte aligned");
    const int64_t rows = touched(s), xn = rows * s.in, wrows = (int64_t)s.E * s.out, wn = wrows * s.in;
    const bool mx = mm->scaling == MOE_MM_SCALE_MX;
    st = check_overlap(s, a, codes ? xn : xn * 2, mx ? xn / 32 : rows * 4, codes ? wn : wn * 2,
                       mx ? wn / 32 : wrows * 4);
    if (st != MOE_OK) return st;
    return launched(launch_grouped_matmul(s, a, static_cast<hipStream_t>(stream)),
                    "grouped matmul launch");
}

moe_status moe_grouped_matmul_w4(const moe_dc_config* cfg, const moe_matmul* mm, const void* x,
                                 const void* weight, const void* weight_scales,
                                 const int32_t* ep_recv_count, const int64_t* recv_offsets,
                                 void* out, void* stream)
{
    MatmulShape s;
    moe_status st = check_matmul(cfg, mm, &s);
    if (st != MOE_OK) return st;
    if (mm->x_dtype != MOE_DTYPE_DEFAULT || mm->scaling != MOE_MM_SCALE_NONE)
        return fail(MOE_ERR_INVALID_ARG, "the 4-bit product takes token rows without scales");
    if (mm->weight_dtype != MOE_W4_INT4 && mm->weight_dtype != MOE_W4_E2M1)
        return fail(MOE_ERR_INVALID_ARG, "weight_dtype %d is not one of 1 (int4), 2 (E2M1)",
                    mm->weight_dtype);
    if (mm->group_size != 32 && mm->group_size != 64 && mm->group_size != 128)
        return fail(MOE_ERR_INVALID_ARG, "group_size %d is not one of 32, 64, 128", mm->group_size);
    if (mm->weight_dtype == MOE_W4_E2M1 && mm->group_size != 32)
        return fail(MOE_ERR_INVALID_ARG, "E2M1 weights have one scale per 32 elements");
    if (s.in % mm->group_size != 0)
        return fail(MOE_ERR_INVALID_ARG, "in_features %d must be a multiple of group_size %d", s.in,
                    mm->group_size);
    s.w4 = mm->weight_dtype;
    s.group = mm->group_size;
    const MatmulArgs a{x, nullptr, weight, weight_scales, ep_recv_count, recv_offsets, out};
    st = check_pointers(a);
    if (st != MOE_OK) return st;
    if (!weight_scales) return fail(MOE_ERR_INVALID_ARG, "weight_scales is required");
    if (!aligned(weight_scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "weight_scales must be 4-byte aligned");
    const int64_t wn = (int64_t)s.E * s.out * s.in;
    st = check_overlap(s, a, touched(s) * s.in * 2, 0, wn / 2,
                       wn / s.group * (mm->weight_dtype == MOE_W4_INT4 ? 2 : 1));
    if (st != MOE_OK) return st;
    return launched(moe_dc::launch_grouped_matmul_w4(s, a, static_cast<hipStream_t>(stream)),
                    "4-bit grouped matmul launch");
}

moe_status moe_gate_topk(const moe_dc_config* cfg, const moe_gate* gate, const float* logits,
                         const float* bias, int32_t* expert_ids, float* expert_scales,
                         void* stream)
{
    moe_dc::Shape sh;
    moe_status st = moe_dc::check_config(cfg, &sh);
    if (st != MOE_OK) return st;
    if (!gate) return fail(MOE_ERR_INVALID_ARG, "gate description is NULL");
    if (gate->score != MOE_SCORE_SOFTMAX && gate->score != MOE_SCORE_SIGMOID)
        return fail(MOE_ERR_INVALID_ARG, "score %d is not one of 0 (softmax), 1 (sigmoid)",
                    gate->score);
    const int32_t n = sh.id_end;
    if (n > 2048)
        return fail(MOE_ERR_UNSUPPORTED, "%d expert ids: the router takes up to 2048", n);
    const int32_t g = gate->group_count;
    if (g < 1 || g > 64 || n % g != 0)
        return fail(MOE_ERR_INVALID_ARG, "group_count %d must be in [1, 64] and divide the %d ids", g,
                    n);
    if (gate->group_keep < 1 || gate->group_keep > g)
        return fail(MOE_ERR_INVALID_ARG, "group_keep %d outside [1, %d]", gate->group_keep, g);
    if (gate->group_top < 1 || gate->group_top > 2 || gate->group_top > n / g)
        return fail(MOE_ERR_INVALID_ARG, "group_top %d must be 1 or 2 and at most the group's %d ids",
                    gate->group_top, n / g);
    if (sh.K > n / g * gate->group_keep)
        return fail(MOE_ERR_INVALID_ARG, "topk %d exceeds the %d ids of the kept groups", sh.K,
                    n / g * gate->group_keep);
    if (gate->renormalize != 0 && gate->renormalize != 1)
        return fail(MOE_ERR_INVALID_ARG, "renormalize must be 0 or 1");
    if (!std::isfinite(gate->factor))
        return fail(MOE_ERR_INVALID_ARG, "factor must be finite");
    if (!logits || !expert_ids || !expert_scales)
        return fail(MOE_ERR_INVALID_ARG, "a required tensor pointer is NULL");
    const int64_t tokens = (int64_t)sh.W * sh.BS, outs = tokens * sh.K * 4;
    if (overlap(expert_ids, outs, logits, tokens * n * 4) || overlap(expert_ids, outs, bias, n * 4) ||
        overlap(expert_scales, outs, logits, tokens * n * 4) ||
        overlap(expert_scales, outs, bias, n * 4) || overlap(expert_ids, outs, expert_scales, outs))
        return fail(MOE_ERR_INVALID_ARG, "expert_ids or expert_scales overlaps another tensor");
    const moe_dc::GateShape s{sh.W * sh.BS, n, sh.K, gate->score == MOE_SCORE_SIGMOID ? 1 : 0,
                              g, gate->group_keep, gate->group_top, gate->renormalize,
                              gate->factor, (1u << 21) / (uint32_t)(n / g) + 1};
    return launched(moe_dc::launch_gate_topk(s, logits, bias, expert_ids, expert_scales,
                                             static_cast<hipStream_t>(stream)),
                    "router kernel launch");
}

}  // extern "C"
