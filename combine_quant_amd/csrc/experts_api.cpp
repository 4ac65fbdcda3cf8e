// experts_api.cpp -- C ABI of the norm, the router, the experts' products and the layer of a few
// tokens: host validation and launch.
//
// As in api.cpp, nothing here allocates device memory or synchronises the host; each call is
// one kernel on the caller's stream (the layer two).
#include "moe_dc.h"
#include "experts_internal.h"
#include "layer_internal.h"
#include "norm_internal.h"

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

// Scales of `n` elements in groups of 128.
int64_t groups_of(int64_t n) { return (n + moe_dc::kBlock - 1) / moe_dc::kBlock; }

// The outputs of a product against each other and everything that it reads, in bytes.
moe_status check_overlap(const MatmulShape& s, const MatmulArgs& a, int64_t x, int64_t x_scales,
                         int64_t w, int64_t w_scales)
{
    const int64_t cols = s.swiglu ? s.out / 2 : s.out;
    const int64_t out = touched(s) * cols * (s.out_code ? 1 : 2);
    const int64_t scales = touched(s) * groups_of(cols) * 4;
    const int64_t counts = (int64_t)s.E * s.W * 4, offsets = (int64_t)(s.W + 1) * 8;
    const struct { const void* p; int64_t n; } outs[2] = {{a.out, out}, {a.out_scales, scales}};
    for (const auto& o : outs)
        if (overlap(o.p, o.n, a.x, x) || overlap(o.p, o.n, a.x_scales, x_scales) ||
            overlap(o.p, o.n, a.w, w) || overlap(o.p, o.n, a.w_scales, w_scales) ||
            overlap(o.p, o.n, a.ep_recv_count, counts) || overlap(o.p, o.n, a.recv_offsets, offsets))
            return fail(MOE_ERR_INVALID_ARG, "out overlaps an input");
    if (overlap(a.out, out, a.out_scales, scales))
        return fail(MOE_ERR_INVALID_ARG, "codes and out_scales overlap");
    return MOE_OK;
}

// The rules of the layer's attributes; fills *s.
moe_status check_layer(const moe_dc_config* cfg, const moe_experts* experts, moe_dc::LayerShape* s)
{
    moe_dc::Shape sh;
    moe_status st = moe_dc::check_config(cfg, &sh);
    if (st != MOE_OK) return st;
    if (!experts) return fail(MOE_ERR_INVALID_ARG, "experts description is NULL");
    if (experts->scaling != MOE_MM_SCALE_NONE && experts->scaling != MOE_MM_SCALE_BLOCK)
        return fail(MOE_ERR_INVALID_ARG, "scaling %d is not one of 0 (token weights), 3 (block)",
                    experts->scaling);
    const int32_t step = experts->scaling == MOE_MM_SCALE_BLOCK ? 16 : 8;
    if (experts->intermediate < 1 || experts->intermediate > 32768)
        return fail(MOE_ERR_INVALID_ARG, "intermediate %d outside [1, 32768]", experts->intermediate);
    if (sh.H % step != 0 || experts->intermediate % step != 0)
        return fail(MOE_ERR_INVALID_ARG, "hidden %d and intermediate %d must be multiples of %d", sh.H,
                    experts->intermediate, step);
    if ((int64_t)sh.W * sh.BS > moe_dc::kLayerTokens)
        return fail(MOE_ERR_UNSUPPORTED, "%lld tokens: the layer takes up to %d", (long long)sh.W * sh.BS,
                    moe_dc::kLayerTokens);
    const int32_t T = sh.W * sh.BS, picks = T * sh.K;
    *s = moe_dc::LayerShape{T, sh.K, sh.E, sh.zero_end, sh.id_end, sh.H, experts->intermediate,
                            experts->scaling == MOE_MM_SCALE_BLOCK ? 1 : 0, sh.tok_f16, sh.mask_kind,
                            sh.E < picks ? sh.E : picks};
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
    s->out_code = 0;
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
    case moe_dc::kMmMxE5m2: return moe_dc::launch_grouped_mxe5m2(s, a, stream);
    case moe_dc::kMmBlockE4m3:
        return s.out_code ? moe_dc::launch_grouped_coded_e4m3(s, a, stream)
                          : moe_dc::launch_grouped_block_e4m3(s, a, stream);
    default:
        return s.out_code ? moe_dc::launch_grouped_coded_e5m2(s, a, stream)
                          : moe_dc::launch_grouped_block_e5m2(s, a, stream);
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

// moe_grouped_matmul, with tokens in `out`, or moe_grouped_matmul_quantize, with codes of out_code
// and out_scales.
moe_status grouped_matmul(const moe_dc_config* cfg, const moe_matmul* mm, const void* x, const void* x_scales,
                          const void* weight, const void* weight_scales, const int32_t* ep_recv_count,
                          const int64_t* recv_offsets, int32_t out_code, void* out, float* out_scales,
                          void* stream)
{
    MatmulShape s;
    moe_status st = check_matmul(cfg, mm, &s);
    if (st != MOE_OK) return st;
    if (mm->weight_dtype != 0 || mm->group_size != 0)
        return fail(MOE_ERR_INVALID_ARG, "weight_dtype and group_size belong to the 4-bit product");
    if (mm->scaling < MOE_MM_SCALE_NONE || mm->scaling > MOE_MM_SCALE_BLOCK)
        return fail(MOE_ERR_INVALID_ARG, "scaling %d is not one of 0..3", mm->scaling);
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
            return fail(MOE_ERR_INVALID_ARG, "fp8 rows need scaling MOE_MM_SCALE_ROW, _MX or _BLOCK");
        if (mm->scaling == MOE_MM_SCALE_ROW) {
            s.type = mm->x_dtype == MOE_DTYPE_E4M3 ? moe_dc::kMmE4m3 : moe_dc::kMmE5m2;
            step = 16;
        } else if (mm->scaling == MOE_MM_SCALE_BLOCK) {
            s.type = mm->x_dtype == MOE_DTYPE_E4M3 ? moe_dc::kMmBlockE4m3 : moe_dc::kMmBlockE5m2;
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
    s.out_code = out_code;
    const MatmulArgs a{x, x_scales, weight, weight_scales, ep_recv_count, recv_offsets, out, out_scales};
    st = check_pointers(a);
    if (st != MOE_OK) return st;
    if (!codes && (x_scales || weight_scales))
        return fail(MOE_ERR_INVALID_ARG, "token rows take no x_scales or weight_scales");
    if (codes && !weight_scales)
        return fail(MOE_ERR_INVALID_ARG, "weight_scales is required for scaling %d", mm->scaling);
    const bool mx = mm->scaling == MOE_MM_SCALE_MX, block = mm->scaling == MOE_MM_SCALE_BLOCK;
    if ((mx || block) && !x_scales)
        return fail(MOE_ERR_INVALID_ARG, "x_scales is required for %s rows", mx ? "MX" : "block-scaled");
    if (!aligned(x_scales, 4) || !aligned(weight_scales, 4))
        return fail(MOE_ERR_INVALID_ARG, "x_scales and weight_scales must be 4-byte aligned");
    const int64_t rows = touched(s), xn = rows * s.in, wrows = (int64_t)s.E * s.out, wn = wrows * s.in;
    const int64_t parts = s.swiglu ? 2 : 1;
    st = check_overlap(s, a, codes ? xn : xn * 2,
                       mx ? xn / 32 : block ? rows * groups_of(s.in) * 4 : rows * 4, codes ? wn : wn * 2,
                       mx ? wn / 32 : block ? s.E * parts * groups_of(s.out / parts) * groups_of(s.in) * 4
                                            : wrows * 4);
    if (st != MOE_OK) return st;
    return launched(launch_grouped_matmul(s, a, static_cast<hipStream_t>(stream)),
                    "grouped matmul launch");
}

}  // namespace

extern "C" {

moe_status moe_grouped_matmul(const moe_dc_config* cfg, const moe_matmul* mm, const void* x,
                              const void* x_scales, const void* weight,
                              const void* weight_scales, const int32_t* ep_recv_count,
                              const int64_t* recv_offsets, void* out, void* stream)
{
    return grouped_matmul(cfg, mm, x, x_scales, weight, weight_scales, ep_recv_count, recv_offsets, 0,
                          out, nullptr, stream);
}

moe_status moe_grouped_matmul_quantize(const moe_dc_config* cfg, const moe_matmul* mm, int32_t out_dtype,
                                       const void* x, const float* x_scales, const void* weight,
                                       const float* weight_scales, const int32_t* ep_recv_count,
                                       const int64_t* recv_offsets, void* codes, float* out_scales,
                                       void* stream)
{
    if (mm && mm->scaling != MOE_MM_SCALE_BLOCK)
        return fail(MOE_ERR_INVALID_ARG, "coded results need scaling MOE_MM_SCALE_BLOCK, got %d", mm->scaling);
    if (out_dtype != MOE_DTYPE_E4M3 && out_dtype != MOE_DTYPE_E5M2)
        return fail(MOE_ERR_INVALID_ARG, "out_dtype %d is not one of 2 (E4M3), 3 (E5M2)", out_dtype);
    if (!out_scales) return fail(MOE_ERR_INVALID_ARG, "out_scales is NULL");
    if (!aligned(out_scales, 4)) return fail(MOE_ERR_INVALID_ARG, "out_scales must be 4-byte aligned");
    return grouped_matmul(cfg, mm, x, x_scales, weight, weight_scales, ep_recv_count, recv_offsets,
                          out_dtype, codes, out_scales, stream);
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
    const MatmulArgs a{x, nullptr, weight, weight_scales, ep_recv_count, recv_offsets, out, nullptr};
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

moe_status moe_rms_norm(const moe_dc_config* cfg, const moe_norm* norm, const void* x,
                        const void* residual, const void* gamma, void* residual_out, void* y,
                        void* codes, void* dynamic_scales, void* stream)
{
    moe_dc::Shape sh;
    moe_status st = moe_dc::check_config(cfg, &sh);
    if (st != MOE_OK) return st;
    if (!norm) return fail(MOE_ERR_INVALID_ARG, "norm description is NULL");
    if (!std::isfinite(norm->epsilon) || norm->epsilon <= 0.0f)
        return fail(MOE_ERR_INVALID_ARG, "epsilon must be finite and above 0");
    if (norm->reserved != 0) return fail(MOE_ERR_INVALID_ARG, "reserved must be 0");
    if (sh.quant_mode == 1 || sh.scales_kind != MOE_SCALES_NONE)
        return fail(MOE_ERR_UNSUPPORTED, "the norm's codes take no scales tensor");
    if (sh.code_type == moe_dc::kCodeE2m1) return fail(MOE_ERR_UNSUPPORTED, "E2M1 codes are not supported");
    if (!x || !gamma) return fail(MOE_ERR_INVALID_ARG, "a required tensor pointer is NULL");
    if (residual_out && !residual)
        return fail(MOE_ERR_INVALID_ARG, "residual_out is the sum with a residual, which is NULL");
    const bool coded = sh.quant_mode != 0;
    if (coded != (codes != nullptr) || coded != (dynamic_scales != nullptr))
        return fail(MOE_ERR_INVALID_ARG, "codes and dynamic_scales must be given iff quant_mode is not 0");
    if (!coded && !y) return fail(MOE_ERR_INVALID_ARG, "y is required for quant_mode 0");
    if (!aligned(x, 2) || !aligned(residual, 2) || !aligned(gamma, 2) || !aligned(residual_out, 2) ||
        !aligned(y, 2) || (sh.scale_format != MOE_SCALE_E8M0 && !aligned(dynamic_scales, 4)))
        return fail(MOE_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
    const int64_t tokens = (int64_t)sh.W * sh.BS, rows = tokens * sh.H * 2;
    const int64_t scales = tokens * sh.scales_per_row * (sh.scale_format == MOE_SCALE_E8M0 ? 1 : 4);
    const struct { const void* p; int64_t n; } outs[4] = {
        {residual_out, rows}, {y, rows}, {codes, rows / 2}, {dynamic_scales, scales}};
    for (int i = 0; i < 4; ++i) {
        // a token is read whole before any of it is written: the sum may take its addends' place
        // and y that of x
        if ((overlap(outs[i].p, outs[i].n, x, rows) && !(i < 2 && outs[i].p == x)) ||
            (overlap(outs[i].p, outs[i].n, residual, rows) && !(i < 2 && outs[i].p == residual)) ||
            overlap(outs[i].p, outs[i].n, gamma, sh.H * 2))
            return fail(MOE_ERR_INVALID_ARG, "an output overlaps an input without being in its place");
        for (int j = 0; j < i; ++j)
            if (overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n))
                return fail(MOE_ERR_INVALID_ARG, "two outputs overlap");
    }
    const bool vectorized = sh.H % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(gamma, 16) &&
                            aligned(residual_out, 16) && aligned(y, 16) && aligned(codes, 8);
    const moe_dc::NormShape s{(int32_t)tokens, sh.H, sh.tok_f16, sh.quant_mode, sh.code_type,
                              sh.scale_format, sh.scales_per_row, norm->epsilon};
    const moe_dc::NormArgs a{x, residual, gamma, residual_out, y, codes, dynamic_scales};
    return launched(moe_dc::launch_rms_norm(s, a, vectorized, static_cast<hipStream_t>(stream)),
                    "norm kernel launch");
}

size_t moe_dc_experts_layer_workspace_bytes(const moe_dc_config* cfg, const moe_experts* experts)
{
    moe_dc::LayerShape s;
    return check_layer(cfg, experts, &s) == MOE_OK ? moe_dc::layer_workspace_bytes(s) : 0;
}

moe_status moe_experts_layer(const moe_dc_config* cfg, const moe_experts* experts, const void* x,
                             const int32_t* expert_ids, const float* expert_scales,
                             const uint8_t* x_active_mask, const void* up, const float* up_scales,
                             const void* down, const float* down_scales, const void* shared_x, void* y,
                             void* workspace, size_t workspace_bytes, void* stream)
{
    moe_dc::LayerShape s;
    moe_status st = check_layer(cfg, experts, &s);
    if (st != MOE_OK) return st;
    if (!x || !expert_ids || !expert_scales || !up || !down || !y)
        return fail(MOE_ERR_INVALID_ARG, "a required tensor pointer is NULL");
    if ((s.mask_kind != 0) != (x_active_mask != nullptr))
        return fail(MOE_ERR_INVALID_ARG, "x_active_mask must be given iff mask_kind != 0");
    if ((s.block != 0) != (up_scales != nullptr) || (s.block != 0) != (down_scales != nullptr))
        return fail(MOE_ERR_INVALID_ARG, "up_scales and down_scales must be given iff scaling is _BLOCK");
    const size_t need = moe_dc::layer_workspace_bytes(s);
    if (!workspace || workspace_bytes < need)
        return fail(MOE_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
    if (!aligned(x, 16) || !aligned(up, 16) || !aligned(down, 16) || !aligned(workspace, 16))
        return fail(MOE_ERR_INVALID_ARG, "x, up, down and workspace must be 16-byte aligned");
    if (!aligned(expert_ids, 4) || !aligned(expert_scales, 4) || !aligned(up_scales, 4) ||
        !aligned(down_scales, 4) || !aligned(shared_x, 2) || !aligned(y, 2))
        return fail(MOE_ERR_INVALID_ARG, "a tensor is not aligned to its elements");
    const int64_t rows = (int64_t)s.T * s.H * 2, picks = (int64_t)s.T * s.K, each = s.block ? 1 : 2;
    const int64_t weights = (int64_t)s.E * s.F * s.H * each, gf = groups_of(s.F), gh = groups_of(s.H);
    const struct { const void* p; int64_t n; } ins[9] = {
        {x, rows}, {expert_ids, picks * 4}, {expert_scales, picks * 4},
        {x_active_mask, s.mask_kind == 1 ? s.T : picks}, {up, 2 * weights}, {down, weights},
        {up_scales, s.E * 2 * gf * gh * 4}, {down_scales, s.E * gf * gh * 4}, {shared_x, rows}};
    for (const auto& in : ins)
        if (overlap(y, rows, in.p, in.n) || overlap(workspace, (int64_t)need, in.p, in.n))
            return fail(MOE_ERR_INVALID_ARG, "y or workspace overlaps an input");
    if (overlap(y, rows, workspace, (int64_t)need))
        return fail(MOE_ERR_INVALID_ARG, "y and workspace overlap");
    char* ws = static_cast<char*>(workspace);
    const moe_dc::LayerArgs a{x, expert_ids, expert_scales, x_active_mask, up, up_scales, down, down_scales,
                              shared_x, y, reinterpret_cast<moe_dc::Slot*>(ws),
                              reinterpret_cast<moe_dc::Row*>(ws + moe_dc::layer_rows_offset(s)),
                              ws + moe_dc::layer_h_offset(s)};
    return launched(moe_dc::launch_experts_layer(s, a, static_cast<hipStream_t>(stream)),
                    "experts' layer launch");
}

}  // extern "C"
