// C ABI of the mixture of experts: argument checks and dispatch (declared in
// include/w8a8.h).
#include <cmath>

#include "api.hpp"
#include "experts.hpp"

using namespace w8a8::api;

namespace {

bool known_dtype(int t) { return t == W8A8_T_BF16 || t == W8A8_T_F32 || t == W8A8_T_F16; }

bool experts_shape(int64_t tokens, int64_t K, int64_t inner, int experts, int top_k)
{
    return tokens >= 0 && tokens <= kMaxRows && experts >= 1 && experts <= w8a8::kMaxExperts && top_k >= 1 &&
           top_k <= w8a8::kMaxTopK && K >= 16 && K <= W8A8_MAX_K && K % 16 == 0 && inner >= 16 &&
           inner <= W8A8_MAX_K && inner % 16 == 0;
}

}  // namespace

W8A8_API w8a8_status_t route_experts(const void *logits, int dtype, int64_t ld, int64_t tokens, int experts,
                                     const w8a8_routing_t *routing, int32_t *ids, float *weights, void *stream)
{
    const char *what = "route_experts";
    if (!routing)
        return fail(W8A8_ERR_NULL, "%s: NULL routing", what);
    const w8a8_routing_t &r = *routing;
    if (!known_dtype(dtype))
        return fail(W8A8_ERR_MODE, "%s: unknown element type %d", what, dtype);
    if (r.score != W8A8_SCORE_SOFTMAX && r.score != W8A8_SCORE_SIGMOID)
        return fail(W8A8_ERR_MODE, "%s: unknown score %d", what, r.score);
    if (tokens < 0 || tokens > kMaxRows || experts < 1 || experts > w8a8::kMaxExperts || ld < experts)
        return fail(W8A8_ERR_SHAPE, "%s: tokens, experts or ld out of range", what);
    if (r.groups < 1 || r.groups > w8a8::kMaxGroups || experts % r.groups != 0 || r.top_groups < 1 ||
        r.top_groups > r.groups || (r.group_top != 1 && r.group_top != 2))
        return fail(W8A8_ERR_SHAPE, "%s: %d groups of %d experts, %d of them by %d, out of range", what, r.groups,
                    experts, r.top_groups, r.group_top);
    if (r.top_k < 1 || r.top_k > w8a8::kMaxTopK || r.top_k > experts / r.groups * r.top_groups)
        return fail(W8A8_ERR_SHAPE, "%s: top_k %d out of range", what, r.top_k);
    if (!std::isfinite(r.scale))
        return fail(W8A8_ERR_SHAPE, "%s: scale must be finite", what);
    if (tokens == 0)
        return ok();
    if (!logits || !ids || !weights)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    if (!aligned(logits, dtype == W8A8_T_F32 ? 4 : 2) || !aligned(r.bias, 4) || !aligned(ids, 4) ||
        !aligned(weights, 4))
        return fail(W8A8_ERR_ALIGN, "%s: tensors must be aligned to their element size", what);
    w8a8_status_t st = check_device();
    if (st != W8A8_OK)
        return st;
    w8a8::RouteArgs a{};
    a.logits = logits;
    a.ld = ld;
    a.tokens = tokens;
    a.kind = dtype;
    a.experts = experts;
    a.top_k = r.top_k;
    a.score = r.score;
    a.bias = r.bias;
    a.groups = r.groups;
    a.top_groups = r.top_groups;
    a.group_top = r.group_top;
    a.renormalize = r.renormalize != 0;
    a.scale = r.scale;
    a.ids = ids;
    a.weights = weights;
    return launched(w8a8::launch_route(a, reinterpret_cast<hipStream_t>(stream)), what);
}

W8A8_API size_t fp8_block_experts_workspace_bytes(int64_t tokens, int64_t K, int64_t inner, int experts, int top_k)
{
    return experts_shape(tokens, K, inner, experts, top_k)
               ? w8a8::experts_workspace_bytes(tokens, top_k, experts, K, inner) : 0;
}

W8A8_API w8a8_status_t fp8_block_experts(const w8a8_experts_t *layer, const void *x, int x_dtype, int64_t ldx,
                                         int64_t tokens, const int32_t *ids, const float *weights, int top_k,
                                         void *out, int64_t ldo, void *workspace, size_t workspace_bytes,
                                         void *stream)
{
    const char *what = "fp8_block_experts";
    if (!layer)
        return fail(W8A8_ERR_NULL, "%s: NULL layer", what);
    const w8a8_experts_t &l = *layer;
    if (!known_dtype(x_dtype))
        return fail(W8A8_ERR_MODE, "%s: unknown element type %d", what, x_dtype);
    if (!experts_shape(tokens, l.K, l.inner, l.experts, top_k))
        return fail(W8A8_ERR_SHAPE, "%s: tokens, K, inner, experts or top_k out of range", what);
    if (ldx < l.K || ldo < l.K)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    if (tokens == 0)
        return ok();
    if (!x || !ids || !weights || !out || !workspace || !l.gate_up || !l.gate_up_scale || !l.down || !l.down_scale)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    const int64_t vec = x_dtype == W8A8_T_F32 ? 4 : 8;
    if (!aligned(x, 16) || ldx % vec != 0 || !aligned(out, 16) || ldo % vec != 0)
        return fail(W8A8_ERR_ALIGN, "%s: rows of x and out must be 16-byte aligned with ld a multiple of %lld", what,
                    (long long)vec);
    if (!aligned(l.gate_up, 16) || !aligned(l.down, 16) || !aligned(workspace, 256))
        return fail(W8A8_ERR_ALIGN, "%s: packed weights must be 16-byte aligned, the workspace 256-byte", what);
    if (!aligned(ids, 4) || !aligned(weights, 4) || !aligned(l.gate_up_scale, 4) || !aligned(l.down_scale, 4))
        return fail(W8A8_ERR_ALIGN, "%s: ids, weights and scales must be 4-byte aligned", what);
    if (workspace_bytes < w8a8::experts_workspace_bytes(tokens, top_k, l.experts, l.K, l.inner))
        return fail(W8A8_ERR_SHAPE, "%s: the workspace is too small", what);
    w8a8_status_t st = check_device();
    if (st != W8A8_OK)
        return st;
    w8a8::ExpertsArgs a{};
    a.x = x;
    a.ldx = ldx;
    a.tokens = tokens;
    a.kind = x_dtype;
    a.K = l.K;
    a.inner = l.inner;
    a.ids = ids;
    a.weights = weights;
    a.top_k = top_k;
    a.experts = l.experts;
    a.gate_up = static_cast<const uint8_t *>(l.gate_up);
    a.down = static_cast<const uint8_t *>(l.down);
    a.gate_up_scale = l.gate_up_scale;
    a.down_scale = l.down_scale;
    a.out = out;
    a.ldo = ldo;
    return launched(w8a8::launch_experts(a, workspace, reinterpret_cast<hipStream_t>(stream)), what);
}
