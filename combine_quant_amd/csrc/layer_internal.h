// layer_internal.h -- launch interface and workspace of the experts' layer of a few tokens.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stddef.h>
#include <stdint.h>

#include "dc_internal.h"

namespace moe_dc {

constexpr int kLayerTokens = 64;             // most tokens: one lane of a wave each

// One validated layer (see moe_experts in include/moe_dc.h).
struct LayerShape {
    int32_t T, K;            // tokens, picks a token
    int32_t E, zero_end, id_end;
    int32_t H, F;
    int32_t block;           // 1: E4M3 weights with a scale per 128 x 128 block, else tokens
    int32_t tok_f16;
    int32_t mask_kind;       // 0 none, 1 per token, 2 per pick
    int32_t slots;           // experts that can have tokens: min(E, T * K)
};

// Workspace: one Slot per expert that can have tokens; one Row per pick, of each row of h; h, [T * K]
// rows of layer_h_row bytes: of every 64 elements the 64 as tokens, then the 64 rests.  Every part
// that is read is written before in the same call.
struct Slot {
    int32_t expert;          // -1: no more experts
    int32_t first;           // its first row of h
    int32_t rows;
    int32_t unused;
};

struct Row {
    int32_t token;
    float weight;            // with which the token chose the expert
};

struct LayerArgs {
    const void* x;
    const int32_t* ids;
    const float* weights;        // of the picks
    const uint8_t* mask;
    const void* up;
    const float* up_scales;
    const void* down;
    const float* down_scales;
    const void* shared;          // null: none
    void* y;
    Slot* slots;                 // the workspace's parts
    Row* rows;
    void* h;
};

constexpr size_t layer_h_row(int32_t F) { return (size_t)((F + 63) / 64) * 256; }
inline size_t layer_rows_offset(const LayerShape& s) { return round256((size_t)s.slots * sizeof(Slot)); }
inline size_t layer_h_offset(const LayerShape& s)
{
    return layer_rows_offset(s) + round256((size_t)s.T * s.K * sizeof(Row));
}
inline size_t layer_workspace_bytes(const LayerShape& s)
{
    return layer_h_offset(s) + (size_t)s.T * s.K * layer_h_row(s.F);
}

hipError_t launch_experts_layer(const LayerShape& s, const LayerArgs& a, hipStream_t stream);

}  // namespace moe_dc
