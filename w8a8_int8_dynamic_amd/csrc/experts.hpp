// Declarations of the mixture of experts: routing, the plan of the experts'
// rows and the products' launches.
#pragma once

#include "fp8_block.hpp"

namespace w8a8 {

constexpr int kMaxExperts = 1024, kMaxTopK = 64, kMaxGroups = 64;

// ---- routing (routing.hip) ----
constexpr int kScoreSoftmax = 0, kScoreSigmoid = 1;
struct RouteArgs {
    const void *logits;          // [tokens, ld] of element kind `kind`
    int64_t ld, tokens;
    int kind, experts, top_k, score;
    const float *bias;           // [experts] or null
    int groups, top_groups, group_top;
    bool renormalize;
    float scale;
    int *ids;                    // [tokens, top_k]
    float *weights;
    int group_lanes;             // (set by launch_route)
    unsigned size_inverse;
};
hipError_t launch_route(const RouteArgs &a, hipStream_t stream);

// ---- the experts' products (experts.hip) ----
struct ExpertsArgs {
    const void *x;               // [tokens, ldx] of element kind `kind`
    int64_t ldx, tokens;
    int kind;
    int64_t K, inner;
    const int *ids;              // [tokens, top_k]
    const float *weights;
    int top_k, experts;
    const uint8_t *gate_up, *down;
    const float *gate_up_scale, *down_scale;
    void *out;                   // [tokens, ldo], x's kind
    int64_t ldo;
};
// Bytes of workspace for `tokens` tokens (0: out of range).
size_t experts_workspace_bytes(int64_t tokens, int top_k, int experts, int64_t K, int64_t inner);
hipError_t launch_experts(const ExpertsArgs &a, void *workspace, hipStream_t stream);

}  // namespace w8a8
