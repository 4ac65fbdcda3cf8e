/*
 * moe_dc.h -- MoE Dispatch/Combine for one AMD Instinct MI355X (gfx950), C ABI.
 *
 * The library implements the data path of the MoE dispatch and combine operators described
 * by these pages (cited below by the tags in brackets):
 *   [DDD] "MoeDistributeDispatch和MoeDistributeCombine算子设计介绍" (gitcode design doc)
 *   [LLD] "low_latency_dispatch" (hiascend API doc): 计算公式, 约束说明
 *   [OPS] "CANN ops-transformer 算子解析：MoeDistributeDispatchV3 的 EP 域 Token 分发与动态量化
 *         通信实现" (mwwr.cn): 功能说明, 参数说明, 约束说明, 调用说明, 接口级量化模式扩展
 *   [SMP] "CANN MoE Dispatch/Combine 通信算子性能优化实践：Kernel 直调与 ACL SHMEM 实现专家分发
 *         与聚合" (lqnn.cn): Dispatch 功能介绍, Combine 功能介绍, 通信前量化
 *
 * All W logical expert-parallel (EP) ranks live in the HBM of one GPU.  The pages' all-to-all
 * exchange therefore becomes a device-local permutation: dispatch writes every routed pick
 * straight to its final row of the receivers' packed buffer, and combine gathers from there.
 *
 * Notation: W ranks, E routed experts (L = E / W per rank, rank r owns [r*L, (r+1)*L)),
 * BS tokens per source rank, H hidden size, K picks per token.  A "pick" is (s, i, k):
 * source rank s, token i, k-th choice, with expert e = expert_ids[s][i][k].
 *
 * Conventions shared by every entry point:
 *   - Tensor arguments are DEVICE pointers into the memory of the current HIP device;
 *     arrays are dense, C-contiguous, in the shapes given.  bf16 is the 16-bit brain-float
 *     bit pattern; every token tensor below written "bf16" (x, ori_x, shared_x, expert_out,
 *     y, mode-0 expand_x) holds IEEE binary16 instead when cfg->token_dtype is
 *     MOE_TOKEN_F16, and y then rounds to binary16.  Device pointers should be 16-byte
 *     aligned for the vectorised kernels;
 *     unaligned pointers (or H not a multiple of 8) select slower element-wise kernels.
 *   - `stream` is a hipStream_t passed as void* (NULL = the legacy default stream).  Every
 *     call is asynchronous on that stream: it validates on the host, enqueues kernels and
 *     returns; outputs are valid in stream order.  No call synchronises the host, and no
 *     call allocates or frees memory: the caller owns every buffer and the stream.
 *   - A negative status other than MOE_ERR_DEVICE means nothing was enqueued (after
 *     MOE_ERR_DEVICE, kernels enqueued before the failing launch may still run and the
 *     outputs are undefined); moe_dc_last_error() then describes the
 *     problem (thread-local, valid until the next call on the same thread).
 */
#ifndef MOE_DC_H
#define MOE_DC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    MOE_OK = 0,
    MOE_ERR_INVALID_ARG = -1,   /* a range, divisibility, pointer or size rule is broken   */
    MOE_ERR_UNSUPPORTED = -2,   /* allowed by the pages but not built (const experts)      */
    MOE_ERR_WORKSPACE = -3,     /* workspace missing or smaller than the query returned    */
    MOE_ERR_DEVICE = -4         /* a HIP runtime call failed                               */
} moe_status;

/* Element type of expand_x ([LLD] 约束说明 lists the types each quant mode allows). */
typedef enum {
    MOE_DTYPE_DEFAULT = 0,      /* the mode's default: bf16 (mode 0), int8 (modes 1, 2),
                                   E4M3 (modes 3, 4, 5)                                     */
    MOE_DTYPE_INT8 = 1,         /* modes 1, 2                                              */
    MOE_DTYPE_E4M3 = 2,         /* OCP E4M3 ("fn": bias 7, max 448); modes 2-5             */
    MOE_DTYPE_E5M2 = 3,         /* OCP E5M2 (bias 15, max 57344); modes 2-5                */
    MOE_DTYPE_E2M1 = 4          /* OCP E2M1 fp4 (max 6), two codes per byte, the element of
                                   even index in the low nibble; modes 4/5, H even          */
} moe_dtype;

/* Shape of the quantization scales tensor ([LLD] 约束说明: for mode 1 a scalar quant
 * coefficient, a row shared by every expert, or one row per expert; modes 2 and 3 take the
 * same shapes as smooth scales). */
typedef enum {
    MOE_SCALES_NONE = 0,        /* no scales tensor (modes 0, 2, 3, 4, 5)                  */
    MOE_SCALES_SCALAR = 1,      /* fp32 [1]                                                */
    MOE_SCALES_SHARED = 2,      /* fp32 [H], the same row for every expert                 */
    MOE_SCALES_PER_EXPERT = 3   /* fp32 [E][H]; the routed expert's row, so quantization is
                                   per pick                                                */
} moe_scales_kind;

/* Storage of the MX block scales (modes 4/5). */
typedef enum {
    MOE_SCALE_FP32 = 0,         /* fp32 2^shared_exp                                        */
    MOE_SCALE_E8M0 = 1,         /* one byte shared_exp + 127 ([SMP] 通信前量化 stores the MX
                                   scale as an E8M0 value)                                  */
    MOE_SCALE_FP32_RECIPROCAL = 2 /* fp32 2^-shared_exp, exact: the value that the [LLD]
                                   计算公式 of modes 4/5 writes out, 1.0 divided by the
                                   block's 2^shared_exp; the pad entry 0                     */
} moe_scale_format;

/* Element type of the tokens: x, ori_x, shared_x, expert_out, y and the mode-0 rows of
 * expand_x ([LLD] and [OPS] 参数说明: the token dtype is float16 or bfloat16). */
typedef enum {
    MOE_TOKEN_BF16 = 0,         /* bfloat16                                                */
    MOE_TOKEN_F16 = 1           /* IEEE binary16; y rounds to nearest even, overflow to inf */
} moe_token_dtype;

/* Bits of moe_dc_config.flags. */
typedef enum {
    /* moe_dispatch always runs the routing and the prefix sums as kernels of their own.  By
     * default a small batch (W*BS*K <= 2048 picks and E*W <= 4096, with the vectorised
     * scatter) computes them inside the scatter launch instead, one launch in place of
     * three; the results are identical either way. */
    MOE_DC_FLAG_SEPARATE_ROUTE = 1,
    /* moe_dispatch also counts the active picks whose expert id lies outside
     * [0, E + zero + copy) -- a contract violation the kernels otherwise skip silently -- and
     * stores the count as the int32 at byte 0 of the workspace (valid in stream order, until
     * the workspace is used again). */
    MOE_DC_FLAG_CHECK_IDS = 2
} moe_dc_flag;

/* Operator attributes ([OPS] 参数说明; [LLD] 约束说明).  One struct serves both calls; the
 * pages require the same values on every rank and for dispatch and its combine
 * ([OPS] 约束说明, cross-card consistency), which one struct gives for free.
 * Layout: sixteen int32 then one int64, 72 bytes, no padding. */
typedef struct {
    int32_t ep_world_size;          /* W, in [2, 768]                                        */
    int32_t moe_expert_num;         /* E, in (0, 1024], E % W == 0; L*W <= 2048               */
    int32_t bs;                     /* BS tokens per rank, in [1, 512]                        */
    int32_t hidden;                 /* H, in [1024, 8192]                                     */
    int32_t topk;                   /* K, in (0, 16], K <= E + zero + copy + const            */
    int32_t quant_mode;             /* 0 none, 1 static int8, 2 dynamic per token,
                                       3 dynamic per 128-element group, 4 MX, 5 MX clip       */
    int32_t zero_expert_num;        /* >= 0; ids [E, E+Z) are zero experts                    */
    int32_t copy_expert_num;        /* >= 0; ids [E+Z, E+Z+C) are copy experts               */
    int32_t const_expert_num;       /* must be 0 (its parameters are not on the pages)        */
    int32_t expert_token_nums_type; /* 0 = running sum over local experts, 1 = counts         */
    int32_t mask_kind;              /* 0 none, 1 per token [W][BS], 2 per pick [W][BS][K]     */
    int32_t out_dtype;              /* moe_dtype: mode 0 DEFAULT only; mode 1 DEFAULT/INT8;
                                       mode 2 DEFAULT/INT8/E4M3/E5M2; mode 3 DEFAULT/E4M3/
                                       E5M2; modes 4/5 DEFAULT/E4M3/E5M2/E2M1                */
    int32_t scales_kind;            /* moe_scales_kind: mode 1 SCALAR/SHARED/PER_EXPERT;
                                       modes 2, 3 any; modes 0, 4, 5 NONE                     */
    int32_t scale_format;           /* moe_scale_format: E8M0 and FP32_RECIPROCAL only with
                                       modes 4/5                                              */
    int32_t flags;                  /* moe_dc_flag bits; 0 for the defaults                   */
    int32_t token_dtype;            /* moe_token_dtype of x, ori_x, shared_x, expert_out, y
                                       and mode-0 expand_x: BF16 (0, the default) or F16      */
    int64_t expand_rows_capacity;   /* rows of expand_x / dynamic_scales / assist_info and of
                                       expert_out; must be >= W*BS*K                           */
} moe_dc_config;

/* Host-only check of every rule the pages state for the attributes ([OPS] 约束说明 and the
 * wrapper's checks under 调用说明; [LLD] 约束说明): the ranges above, E % W == 0,
 * L*W <= 2048, K <= E+Z+C+const, E+Z+C+const < INT32_MAX, capacity >= W*BS*K and < 2^31,
 * and the pairings of quant_mode with out_dtype, scales_kind and scale_format above.
 * Returns MOE_OK, MOE_ERR_INVALID_ARG or MOE_ERR_UNSUPPORTED.  Touches no device. */
moe_status moe_dc_validate(const moe_dc_config* cfg);

/* Scales per expand_x row for cfg->quant_mode (the dynamic_scales shape rule of [LLD]
 * 约束说明): 0 for modes 0 and 1, 1 for mode 2, Ceil(H, 128) for mode 3 and
 * Align2(Ceil(H, 32)) for modes 4/5.  Each scale is an fp32, or one byte with
 * MOE_SCALE_E8M0.  Returns -1 for an invalid config. */
int32_t moe_dc_scales_per_row(const moe_dc_config* cfg);

/* Workspace bytes moe_dispatch needs for this config (the pages' two-phase pattern:
 * query the workspace size, then execute; [OPS] 调用说明).  0 for an invalid config.
 * The workspace is scratch: its contents need no initialisation and are meaningless after
 * the call (except the checked-ids count of MOE_DC_FLAG_CHECK_IDS at byte 0); one workspace
 * must not be used by two dispatches that may run concurrently. */
size_t moe_dc_dispatch_workspace_bytes(const moe_dc_config* cfg);

/* moe_dispatch -- quantize, route and scatter every pick to its receiver's packed rows.
 *
 * Defined by: [DDD] §2.2 (index computation: per source rank, a pick's expand_idx is the
 * count of that rank's earlier picks, in row-major (token, pick) order, that chose the same
 * expert; the target rank is e / L rounded down and the local expert e % L); [DDD] §2.4
 * (receive side: the W x L count matrix is transposed and prefix-summed row-major into
 * ep_recv_count; expert_token_nums is its last column); [OPS] 功能说明 情形 1/2 and
 * [LLD] 计算公式 (quantization formulas of modes 0-5); [SMP] Dispatch 功能介绍
 * (each row carries its source triple, output as assist_info_for_combine).
 *
 * Quantization of a token x (x_fp32 = x widened to fp32, times the scales tensor if any):
 *   mode 1  codes = int8(x_fp32)
 *   mode 2  dyn = type_max / max|x_fp32| over the token; codes = type(x_fp32 * dyn);
 *           scale = 1/dyn (type_max 127 int8, 448 E4M3, 57344 E5M2)
 *   mode 3  as mode 2 for each group of 128 consecutive elements (the last may be short)
 *   mode 4  per 32-element block: shared_exp = floor(log2 max|x|) - emax, at least -127
 *           (emax 8 for E4M3, 15 for E5M2; an all-zero block takes -127)
 *   mode 5  per block: shared_exp = ceil(log2(max(max|x|, 1e-4) / type_max))
 *   modes 4/5: codes = fp8(x / 2^shared_exp); scale = 2^shared_exp (the dequant multiplier);
 *           E2M1 elements use emax 2 and type_max 6
 *
 * Inputs:
 *   x              bf16  [W][BS][H]   tokens of every source rank (finite values)
 *   expert_ids     int32 [W][BS][K]   picks; ids >= E are the special experts
 *   scales         fp32, shaped by cfg->scales_kind ([1], [H] or [E][H]); NULL iff
 *                  scales_kind is MOE_SCALES_NONE
 *   x_active_mask  uint8 [W][BS] (mask_kind 1) or [W][BS][K] (mask_kind 2), or NULL when
 *                  mask_kind is 0; nonzero = active.  An inactive pick is not dispatched.
 *   expert_scales  fp32 [W][BS][K] pick weights, or NULL; given exactly when expand_scales
 *                  is given (each routed row then carries its pick's weight)
 * Outputs (row = a receiver row in the packed layout below; cap = expand_rows_capacity):
 *   expand_x       [cap][H] bf16 (mode 0), [cap][H/2] bytes for E2M1 (two codes per byte),
 *                  else [cap][H] bytes: int8 or fp8 codes
 *   dynamic_scales [cap][moe_dc_scales_per_row(cfg)] fp32 (or bytes with MOE_SCALE_E8M0):
 *                  mode 2 one 1/dyn per row; mode 3 one 1/dyn per group; modes 4/5 one scale
 *                  per 32-element block (2^shared_exp, its E8M0 byte, or 2^-shared_exp, as
 *                  scale_format says) and 0 in the Align2 pad slot.  NULL allowed for
 *                  modes 0 and 1, which have no scales
 *   expand_idx     int32 [W][BS][K]   ordinal of each pick among its source rank's picks of
 *                  the same expert; -1 for inactive picks and special experts
 *   assist_info    int32 [cap][3]     (s, i, k) of the pick stored in each row
 *   ep_recv_count  int32 [W][L*W]     receiver r, entry j*W+s: inclusive running total of
 *                  the rows r receives, over (local expert j, source s) in that order
 *   expert_token_nums int64 [W][L]    type 1: rows per local expert; type 0: running sum
 *   recv_offsets   int64 [W+1]        first row of each receiver; [W] = total routed rows
 *   expand_scales  fp32 [cap] or NULL: each row's pick weight ([OPS] 参数说明,
 *                  expand_scales_out: the weight travels with its token)
 *   workspace      moe_dc_dispatch_workspace_bytes(cfg) bytes, 4-byte aligned
 * Packed layout: receiver r owns rows [recv_offsets[r], recv_offsets[r+1]); inside, rows go
 * by local expert, then source rank, then expand_idx.  So the whole buffer is one stable sort
 * of the routed picks by (expert, s, i, k).  Rows at or past recv_offsets[W] are not written.
 * Numerics: every fp32 operation is a single IEEE binary32 operation rounded to nearest
 * even, in the order of the formulas; int8 codes round half to even and saturate at +-127
 * (NaN -> 0); fp8 codes round to nearest even and saturate at +-448 (E4M3) or +-57344
 * (E5M2); in modes 2/3 an all-zero segment gives codes 0 and scale 0; fp32 subnormals are
 * kept.  The results are deterministic: identical inputs give identical bytes.
 * Errors: host validation first (MOE_ERR_INVALID_ARG / _UNSUPPORTED / _WORKSPACE); a HIP
 * launch failure gives MOE_ERR_DEVICE.  Out-of-range expert ids are a contract violation:
 * the kernels never access memory out of bounds for them and treat such picks as not
 * dispatched; MOE_DC_FLAG_CHECK_IDS counts them.  A per-token mask needs no particular order (the pages ask for trues before
 * falses; any order works here). */
moe_status moe_dispatch(const moe_dc_config* cfg,
                        const void* x, const int32_t* expert_ids,
                        const float* scales, const uint8_t* x_active_mask,
                        const float* expert_scales,
                        void* expand_x, void* dynamic_scales, int32_t* expand_idx,
                        int32_t* assist_info, int32_t* ep_recv_count,
                        int64_t* expert_token_nums, int64_t* recv_offsets,
                        float* expand_scales,
                        void* workspace, size_t workspace_bytes, void* stream);

/* moe_dispatch_no_workspace -- moe_dispatch without a workspace argument, for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation).  It runs the same kernels and writes the same outputs as
 * moe_dispatch; its workspace is a 1 MiB array in the library's own device memory, one per
 * GPU, held from the library's load until the process ends.
 *
 * Arguments: as for moe_dispatch, less workspace and workspace_bytes.
 * Limits and errors: a config whose moe_dc_dispatch_workspace_bytes exceeds 1 MiB
 * (E * W above about 260,000 counts) returns MOE_ERR_WORKSPACE, and MOE_DC_FLAG_CHECK_IDS
 * (whose count lands in the caller's workspace) returns MOE_ERR_INVALID_ARG; both are checked
 * on the host before anything is enqueued.  The first call on a device looks up that device's
 * copy of the array (MOE_ERR_DEVICE if the lookup fails).  Nothing is allocated or freed.
 * Every call on one GPU uses the same array: calls that may run concurrently on one GPU
 * (other streams, other threads) race and must be ordered by the caller. */
moe_status moe_dispatch_no_workspace(const moe_dc_config* cfg,
                                     const void* x, const int32_t* expert_ids,
                                     const float* scales, const uint8_t* x_active_mask,
                                     const float* expert_scales,
                                     void* expand_x, void* dynamic_scales, int32_t* expand_idx,
                                     int32_t* assist_info, int32_t* ep_recv_count,
                                     int64_t* expert_token_nums, int64_t* recv_offsets,
                                     float* expand_scales, void* stream);

/* moe_combine -- gather each token's K expert outputs and form their weighted sum.
 *
 * Defined by: [DDD] §3.4 (a pick's expert output sits at its rank's window + the expert's
 * offset + expand_idx; the K outputs are weighted and summed back to the token); [SMP]
 * Combine 功能介绍 (each expert row times its expert scale, accumulated in fp32, then cast
 * down); [LLD] 计算公式 特殊专家场景 (a zero expert outputs 0, a copy expert outputs ori_x).
 *
 * Inputs:
 *   expert_out     bf16 [cap][H]      expert outputs, row-aligned with dispatch's expand_x
 *   expert_ids, expand_idx, ep_recv_count, recv_offsets: as produced by moe_dispatch for
 *                  this config (the addressing uses exactly these)
 *   expert_scales  fp32 [W][BS][K]    weight of each pick
 *   x_active_mask  as for moe_dispatch (inactive picks contribute nothing)
 *   ori_x          bf16 [W][BS][H]    dispatch's x; required iff copy_expert_num > 0
 * Output:
 *   y              bf16 [W][BS][H]    y[s][i] = bf16_rne( sum over active picks in k order of
 *                  w * expert_row ), accumulated in fp32 starting from +0 with one multiply
 *                  and one add per pick (zero experts add nothing); all-inactive tokens -> +0
 * Errors: as for moe_dispatch; ori_x NULL with copy experts is MOE_ERR_INVALID_ARG.
 * Needs no workspace. */
moe_status moe_combine(const moe_dc_config* cfg,
                       const void* expert_out, const int32_t* expert_ids,
                       const int32_t* expand_idx, const float* expert_scales,
                       const int32_t* ep_recv_count, const int64_t* recv_offsets,
                       const uint8_t* x_active_mask, const void* ori_x, void* y,
                       void* stream);

/* Workspace bytes moe_combine_scatter needs: one int32 per pick slot (W*BS*K), rounded up
 * to 256.  0 for an invalid config.  Scratch, as for dispatch. */
size_t moe_dc_combine_scatter_workspace_bytes(const moe_dc_config* cfg);

/* moe_combine_scatter -- the scatter-back combine: rows return to their sources by their
 * source triples, then each token sums its K slots and adds the shared expert's output.
 *
 * Defined by: [SMP] Combine 功能介绍 计算步骤 and 源码实现: each expert-side row r is sent back
 * using its triple (s, i, k) = assist_info[r] to offset epOffset = i * K + k of source rank s;
 * the source then multiplies each of a token's K results by its expert scale, sums them in
 * fp32 and adds the shared expert's result.  All ranks share this GPU's memory, so a slot
 * stores the row's index (in the workspace) and the sum reads the row through it: the same
 * values as copying the row, without moving its bytes twice.
 *
 * Inputs:
 *   expert_out     bf16 [cap][H]      expert outputs, row-aligned with expand_x
 *   assist_info    int32 [cap][3]     from moe_dispatch; rows [0, recv_offsets[W]) are sent
 *   recv_offsets   int64 [W+1]        from moe_dispatch
 *   expert_ids     int32 [W][BS][K]   which picks are routed, zero or copy experts
 *   expert_scales  fp32 [W][BS][K]    the source's pick weights
 *   x_active_mask  as for moe_dispatch
 *   ori_x          bf16 [W][BS][H]    required iff copy_expert_num > 0
 *   shared_x       bf16 [W][BS][H]    the shared expert's output per token, or NULL
 * Output:
 *   y              bf16 [W][BS][H] = bf16_rne( sum over active picks in k order of w * row,
 *                  then + shared_x ), accumulated in fp32 from +0
 * Errors: as for moe_combine; a workspace smaller than the query is MOE_ERR_WORKSPACE. */
moe_status moe_combine_scatter(const moe_dc_config* cfg, const void* expert_out,
                               const int32_t* assist_info, const int64_t* recv_offsets,
                               const int32_t* expert_ids, const float* expert_scales,
                               const uint8_t* x_active_mask, const void* ori_x,
                               const void* shared_x, void* y, void* workspace,
                               size_t workspace_bytes, void* stream);

/* moe_combine_quantize -- expert-side int8 block quantization of the expert outputs, the
 * compression the pages apply before the combine's return transfer.
 *
 * Defined by: [SMP] 通信前量化 (Combine 的 INT8 block 量化): each expert-output row is cut into
 * blocks of 8 elements (32 bytes of fp32); per block scale = amax * (1/127) (the reciprocal of
 * 127 rounded once to fp32), and each code = int8(fp16(x / scale)), where the division is one
 * IEEE fp32 division and each narrowing rounds to nearest even (int8 saturates at +-127; an
 * all-zero block gives codes 0 and scale 0).
 *
 * Inputs:
 *   expert_out     bf16 [cap][H]      as for moe_combine
 *   recv_offsets   int64 [W+1]        from moe_dispatch; rows [0, recv_offsets[W]) are coded
 * Outputs:
 *   codes          int8 [cap][H]
 *   block_scales   fp32 [cap][Ceil(H, 8)]
 * Rows at or past recv_offsets[W] are not written.  Errors as for moe_combine. */
moe_status moe_combine_quantize(const moe_dc_config* cfg, const void* expert_out,
                                const int64_t* recv_offsets, int8_t* codes,
                                float* block_scales, void* stream);

/* moe_combine_int8 -- moe_combine over block-quantized expert outputs.
 *
 * Defined by: moe_combine's definition with each routed pick's row dequantized first
 * ([SMP] 通信前量化: int8 -> fp16 -> float, both exact, times the block's scale, one fp32
 * multiply); zero experts add nothing, copy experts add w * ori_x (ori_x is not quantized).
 *
 * Inputs: codes and block_scales as written by moe_combine_quantize; the other arguments as
 * for moe_combine.  Output: y bf16 [W][BS][H] = bf16_rne( sum over active picks in k order
 * of w * (code * scale) ), accumulated in fp32 from +0.  Errors as for moe_combine. */
moe_status moe_combine_int8(const moe_dc_config* cfg, const int8_t* codes,
                            const float* block_scales, const int32_t* expert_ids,
                            const int32_t* expand_idx, const float* expert_scales,
                            const int32_t* ep_recv_count, const int64_t* recv_offsets,
                            const uint8_t* x_active_mask, const void* ori_x, void* y,
                            void* stream);

/* ---- the router and the experts' products -------------------------------------------------
 *
 * The calls on either side of the exchange: moe_gate_topk makes the expert_ids and
 * expert_scales that moe_dispatch and moe_combine take, and the products turn the packed rows
 * of expand_x into the rows of expert_out.  They follow the conventions at the top of this
 * header, except that x and weight must be 16-byte and their scales 4-byte aligned (there is
 * no element-wise fallback), and that an output that overlaps another tensor of the same call is
 * refused (MOE_ERR_INVALID_ARG).  They need no workspace; each is one kernel. */

/* How the products' codes are scaled. */
typedef enum {
    MOE_MM_SCALE_NONE = 0,      /* token rows and weights                                  */
    MOE_MM_SCALE_ROW = 1,       /* one fp32 per row of x and one per weight row            */
    MOE_MM_SCALE_MX = 2,        /* one E8M0 byte per 32 elements of x and of the weights   */
    MOE_MM_SCALE_BLOCK = 3      /* one fp32 per 128 elements of a row of x and per block of 128
                                   x 128 elements of the weights                            */
} moe_mm_scaling;

typedef enum {
    MOE_ACT_NONE = 0,
    MOE_ACT_SWIGLU = 1          /* weight rows [0, N/2) are the gate, [N/2, N) the up rows  */
} moe_activation;

/* 4-bit weights: two codes per byte, the element of even index in the low nibble. */
typedef enum {
    MOE_W4_INT4 = 1,            /* two's complement, -8..7                                 */
    MOE_W4_E2M1 = 2             /* OCP E2M1 with E8M0 scales (MX)                          */
} moe_w4_dtype;

/* One product of the packed rows with the experts' weights.  Eight int32, 32 bytes. */
typedef struct {
    int32_t in_features;        /* I, in [1, 65536]: elements of a row of x                 */
    int32_t out_features;       /* N, in [1, 65536]: weight rows per expert                 */
    int32_t x_dtype;            /* moe_dtype of the rows: DEFAULT = the token type, INT8,
                                   E4M3 or E5M2 (moe_grouped_matmul only)                   */
    int32_t scaling;            /* moe_mm_scaling: NONE for tokens, ROW for INT8, ROW, MX or
                                   BLOCK for E4M3 and E5M2                                  */
    int32_t activation;         /* moe_activation                                           */
    int32_t weight_dtype;       /* moe_w4_dtype for moe_grouped_matmul_w4, else 0            */
    int32_t group_size;         /* moe_grouped_matmul_w4: 32, 64 or 128 elements per scale
                                   (E2M1: 32), else 0                                        */
    int32_t reserved;           /* 0                                                        */
} moe_matmul;

/* moe_grouped_matmul -- every packed row times its expert's weights.
 *
 * For the rows p of expert e (receiver r = e / L, local expert j = e % L: rows from
 * recv_offsets[r] + ep_recv_count[r][j*W - 1] (0 for j = 0) up to recv_offsets[r] +
 * ep_recv_count[r][j*W + W - 1]), with X and V the values of x and weight:
 *   S[p][n]   = sum over i of X[p][i] * V[e][n][i]
 *   out[p][n] = S[p][n]                                        MOE_ACT_NONE,   n < N
 *   out[p][n] = silu(S[p][n]) * S[p][N/2 + n], silu(t) = t / (1 + exp(-t))
 *                                                              MOE_ACT_SWIGLU, n < N/2
 * X and V are the tokens themselves, code * scale of the row (ROW), code * 2^(byte - 127) of
 * the block (MX), or code * scale of the group or block (BLOCK).
 *
 * Inputs:
 *   x              [cap][I] in x_dtype (mode-0 expand_x, or its codes)
 *   x_scales       ROW: fp32 [cap] (mode 2's dynamic_scales), or NULL for all 1 (mode 1, whose
 *                  static scale belongs into weight_scales); MX: bytes [cap][I/32] (the
 *                  dynamic_scales of MOE_SCALE_E8M0); BLOCK: fp32 [cap][Ceil(I, 128)] (mode 3's
 *                  dynamic_scales); NULL for tokens
 *   weight         [E][N][I]: tokens for token rows, int8 for INT8, E4M3 for E4M3 and E5M2
 *   weight_scales  ROW: fp32 [E][N]; MX: bytes [E][N][I/32]; BLOCK: fp32
 *                  [E][Ceil(N, 128)][Ceil(I, 128)], with SwiGLU [E][2 Ceil(N/2, 128)][Ceil(I, 128)]:
 *                  the blocks of the gate rows, then those of the up rows, which begin anew at row
 *                  N/2; NULL for tokens
 *   ep_recv_count, recv_offsets: as produced by moe_dispatch for this config
 * Output:
 *   out            token type [cap][N], or [cap][N/2] with SwiGLU.  Rows at or past
 *                  recv_offsets[W] are not written
 * I must be a multiple of 8 (tokens), 16 (ROW, BLOCK) or 128 (MX).
 * Numerics: products are exact; int8 sums are exact in 32 bits; the other sums are fp32 in an
 * order that depends on the sizes only (the same inputs give the same bytes); ROW scales
 * multiply the sum (weight's, then row's); BLOCK sums 128 products, multiplies them by the
 * product of their two scales and adds, each in fp32; SwiGLU is within 2^-17 of its value for S[p][n] down
 * to -176, below that 0; out is rounded once, to nearest even.  The fp8
 * matrix instructions add eight consecutive products at a time and drop, of each product, what
 * lies below 2^-13 of the largest one's power of two.  An infinity or NaN stays within its own
 * row (or weight row).
 * Errors: MOE_ERR_UNSUPPORTED for E2M1 rows; otherwise as for moe_dispatch. */
moe_status moe_grouped_matmul(const moe_dc_config* cfg, const moe_matmul* mm, const void* x,
                              const void* x_scales, const void* weight,
                              const void* weight_scales, const int32_t* ep_recv_count,
                              const int64_t* recv_offsets, void* out, void* stream);

/* moe_grouped_matmul_quantize -- moe_grouped_matmul of block-scaled rows, its results coded for
 * another such product.
 *
 * With M = N, or N/2 with SwiGLU, and out[p][n] as moe_grouped_matmul defines it, before its last
 * rounding: each row's columns in groups of 128 (the last may be short) are coded as moe_dispatch
 * codes a token in mode 3: dyn = type_max / max|out| over the group, codes = type(out * dyn), scale =
 * 1/dyn; a group of zeros has codes 0 and scale 0.  A group that holds an infinity or a NaN has scale
 * NaN and codes 0.
 *
 * Inputs as for moe_grouped_matmul with scaling MOE_MM_SCALE_BLOCK (no other is taken).
 *   out_dtype      MOE_DTYPE_E4M3 or MOE_DTYPE_E5M2 (moe_dtype), whatever the rows of x hold
 * Outputs:
 *   codes          bytes [cap][M]
 *   out_scales     fp32 [cap][Ceil(M, 128)]
 * Rows at or past recv_offsets[W] are not written.  Numerics and errors as for
 * moe_grouped_matmul, but tiles of up to 64 rows drop nothing of the products: those of an expert with up
 * to 64 rows, and without SwiGLU of every expert where the product is small.  In taller ones what is dropped
 * shows as another code, one step away, in about one of 1000 (7168 x 4096, 512 rows an expert: 8 to 16 of
 * 10 000, values off by 0.0012 of their norm).  The codes of a row may therefore depend on how many rows
 * its expert has; the same inputs give the same bytes. */
moe_status moe_grouped_matmul_quantize(const moe_dc_config* cfg, const moe_matmul* mm,
                                       int32_t out_dtype, const void* x, const float* x_scales,
                                       const void* weight, const float* weight_scales,
                                       const int32_t* ep_recv_count, const int64_t* recv_offsets,
                                       void* codes, float* out_scales, void* stream);

/* moe_grouped_matmul_w4 -- moe_grouped_matmul of token rows with 4-bit weights.
 *
 * V[e][n][i] = code * scale of the group of group_size elements that i belongs to.
 *   x              token type [cap][I]
 *   weight         bytes [E][N][I/2], two codes per byte
 *   weight_scales  int4: token type [E][N][I/group_size]; E2M1: E8M0 bytes [E][N][I/32]
 * I must be a multiple of group_size.  The codes enter the matrix instructions exactly; each
 * group's sum (int4 with bf16 rows: a sixteenth of it) is formed in fp32, multiplied by its scale
 * and added in fp32.  (E2M1 codes may enter as bf16 code * scale, which is exact for scale bytes
 * up to 252; with 253 or 254 the larger codes may turn infinite.)
 * Everything else as for moe_grouped_matmul. */
moe_status moe_grouped_matmul_w4(const moe_dc_config* cfg, const moe_matmul* mm, const void* x,
                                 const void* weight, const void* weight_scales,
                                 const int32_t* ep_recv_count, const int64_t* recv_offsets,
                                 void* out, void* stream);

typedef enum {
    MOE_SCORE_SOFTMAX = 0,
    MOE_SCORE_SIGMOID = 1
} moe_score;

/* Attributes of the router.  Five int32 and one float, 24 bytes. */
typedef struct {
    int32_t score;              /* moe_score                                                */
    int32_t group_count;        /* G >= 1, at most 64, a divisor of n; 1 = no group limit    */
    int32_t group_keep;         /* groups kept per token, in [1, G]                          */
    int32_t group_top;          /* a group's value is the sum of its 1 or 2 best choices     */
    int32_t renormalize;        /* 1: the K weights are divided by their sum + 1e-20          */
    float factor;               /* multiplies the weights                                   */
} moe_gate;

/* moe_gate_topk -- the K best experts of every token, and their weights.
 *
 * Over the n = E + zero + copy ids of the config (n <= 2048, else MOE_ERR_UNSUPPORTED):
 *   score  = softmax over the n logits, or sigmoid of each
 *   choice = score + bias (score alone without a bias)
 *   the ids fall into G groups of n / G in order; with G > 1 only the group_keep groups with
 *   the largest value (sum of the group_top largest choices) stay
 *   expert_ids = the K remaining ids with the largest choice, largest first
 *   expert_scales = their scores (without the bias), divided by (their sum + 1e-20) with
 *   renormalize, times factor
 * Equal choices and equal groups go to the lower id.  Choices are compared in binary64, so
 * that scores next to each other keep their order; without a bias the logits are compared
 * (which is the same order), and only group values with group_top 2 are sums of scores.
 *   logits         fp32 [W][BS][n]
 *   bias           fp32 [n] or NULL
 *   expert_ids     int32 [W][BS][K]
 *   expert_scales  fp32 [W][BS][K]
 * A NaN choice or group value ranks below every number; a softmax row without a finite logit (or with a NaN
 * or +infinity) has weights 0 or NaN, and its ids are distinct and in range all the same.
 * K may not exceed the ids of the kept groups. */
moe_status moe_gate_topk(const moe_dc_config* cfg, const moe_gate* gate, const float* logits,
                         const float* bias, int32_t* expert_ids, float* expert_scales,
                         void* stream);

/* ---- the norm before the router ------------------------------------------------------------ */

/* Attributes of the norm.  One float and one int32, 8 bytes. */
typedef struct {
    float epsilon;              /* finite, > 0                                              */
    int32_t reserved;           /* 0                                                        */
} moe_norm;

/* moe_rms_norm -- the tokens that router and dispatch take: RMS norm, with the residual's addition
 * before it and 8-bit codes behind it.
 *
 * For every token, over its H elements, in fp32:
 *   s = x + residual                      (x alone without a residual)
 *   y = s / sqrt(mean(s^2) + epsilon) * gamma
 *   residual_out = s, y = y, rounded to the token type (nearest even)
 *   codes, dynamic_scales = y (before that rounding) coded as moe_dispatch codes a token with
 *                  cfg->quant_mode 2, 3, 4 or 5, cfg->out_dtype and cfg->scale_format
 * They follow the conventions at the top of this header; H not a multiple of 8 or tensors that are
 * not 16-byte aligned (codes: 8) select a slower kernel.
 *   x              token type [W][BS][H]
 *   residual       token type [W][BS][H] or NULL
 *   gamma          token type [H]
 *   residual_out   token type [W][BS][H], or NULL; may be residual or x itself (in place)
 *   y              token type [W][BS][H], NULL allowed with codes; may be x or residual itself
 *   codes          bytes [W][BS][H]; NULL iff quant_mode is 0
 *   dynamic_scales [W][BS][moe_dc_scales_per_row(cfg)] in cfg->scale_format; NULL iff quant_mode
 *                  is 0
 * The codes are rows for moe_grouped_matmul: mode 2 ROW, mode 3 BLOCK, modes 4/5 with E8M0 MX.
 * Numerics: the mean is a sum in fp32, in an order that depends on H and on the number of tokens;
 * s^2 must not leave the range of fp32.  A token with an infinity or NaN, or whose sum of squares
 * is infinite, has NaN or zeros in y; a scale whose token, group or block holds one is NaN (E8M0:
 * 255) and the code of a NaN is 0.
 * Errors: MOE_ERR_UNSUPPORTED for quant_mode 1, a scales tensor and E2M1; MOE_ERR_INVALID_ARG for
 * outputs that overlap each other or an input other than in its place; otherwise as for
 * moe_dispatch.  Needs no workspace; one kernel. */
moe_status moe_rms_norm(const moe_dc_config* cfg, const moe_norm* norm, const void* x,
                        const void* residual, const void* gamma, void* residual_out, void* y,
                        void* codes, void* dynamic_scales, void* stream);

/* ---- the whole layer for few tokens -------------------------------------------------------- */

/* The experts of a layer.  Two int32, 8 bytes. */
typedef struct {
    int32_t intermediate;       /* F, in [1, 32768]: gate rows (and up rows) of an expert    */
    int32_t scaling;            /* MOE_MM_SCALE_NONE: weights of the token type; _BLOCK: E4M3
                                   with one fp32 per block of 128 x 128 elements             */
} moe_experts;

/* Workspace bytes moe_experts_layer needs (two rows of F tokens a pick, F up to a multiple of 64,
 * and up to 24 KiB).  0 for an invalid config or description.  Scratch, as for dispatch; one workspace must
 * not be used by two calls that may run concurrently. */
size_t moe_dc_experts_layer_workspace_bytes(const moe_dc_config* cfg, const moe_experts* experts);

/* moe_experts_layer -- everything between the router and the residual for up to 64 tokens (W * BS),
 * in two kernels: what moe_dispatch, two products and moe_combine do for many.
 *
 * For every token t, over its active picks k of expert e with weight w:
 *   h = silu(x . gate_e) * (x . up_e), y = sum over k of w * (h . down_e)
 * with up = gate rows [0, F), then up rows [F, 2F).  A zero expert adds nothing, a copy expert
 * w * x; shared_x (the shared expert's output) is added at the end.
 *   x              token type [W][BS][H]
 *   expert_ids     int32 [W][BS][K], expert_scales fp32 [W][BS][K]: as moe_gate_topk gives them
 *   x_active_mask  as for moe_dispatch (an inactive pick contributes nothing)
 *   up             [E][2F][H], down [E][H][F]: tokens, or E4M3 codes
 *   up_scales      fp32 [E][2 Ceil(F, 128)][Ceil(H, 128)] (the gate rows' blocks, then those of the
 *                  up rows, as moe_grouped_matmul takes them), down_scales fp32
 *                  [E][Ceil(H, 128)][Ceil(F, 128)]; NULL without _BLOCK
 *   shared_x       token type [W][BS][H] or NULL
 *   y              token type [W][BS][H]; a token without active picks gets shared_x or +0
 *   workspace      moe_dc_experts_layer_workspace_bytes bytes
 * H and F must be multiples of 8 (tokens) or 16 (_BLOCK); x, up, down and workspace 16-byte aligned.
 * cfg's quantization attributes are not used.
 * Numerics: products of token values and codes are exact (the tokens are not quantized); sums are
 * fp32 in an order that depends on the sizes and ids only; _BLOCK sums the products of a block,
 * multiplies by its scale and adds; SwiGLU as for moe_grouped_matmul.  h is kept as two
 * numbers of the token type between the two products, its rounding and the rest: 16 bits of bf16, 22 of
 * fp16 (down to 2^-25; infinite past 65504).  y is rounded once at the end; w multiplies sums in fp32
 * (it is the sum of the weights where a token picked an expert more than once).  An infinity or NaN
 * in a weight reaches only the tokens that picked its expert, an infinity in `down` as a NaN.
 * Errors: MOE_ERR_UNSUPPORTED for more than 64 tokens; y or the workspace overlapping an input is
 * MOE_ERR_INVALID_ARG; otherwise as for moe_dispatch.  Picks with ids out of range count as
 * inactive. */
moe_status moe_experts_layer(const moe_dc_config* cfg, const moe_experts* experts, const void* x,
                             const int32_t* expert_ids, const float* expert_scales,
                             const uint8_t* x_active_mask, const void* up, const float* up_scales,
                             const void* down, const float* down_scales, const void* shared_x,
                             void* y, void* workspace, size_t workspace_bytes, void* stream);

/* Text of the last non-OK status on this thread ("" if none). */
const char* moe_dc_last_error(void);

/* Library version string. */
const char* moe_dc_version(void);

#ifdef __cplusplus
}
#endif
#endif /* MOE_DC_H */
