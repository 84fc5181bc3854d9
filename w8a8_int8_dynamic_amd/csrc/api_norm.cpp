// C ABI of the norms around a layer: argument checks and dispatch (declared
// in include/w8a8.h).
#include <cmath>

#include "api.hpp"

using namespace w8a8::api;

namespace {

int64_t size_of(int dtype) { return dtype == W8A8_T_F32 ? 4 : 2; }
bool known_dtype(int t) { return t == W8A8_T_BF16 || t == W8A8_T_F32 || t == W8A8_T_F16; }

// Fills `to` from the caller's norm for rows of K in M rows; post: only
// weight and bias may be given.
w8a8_status_t norm_args(const w8a8_norm_t *n, int64_t M, int64_t K, bool post, const char *what,
                        w8a8::NormVectors &to)
{
    if (n->kind != W8A8_NORM_RMS && n->kind != W8A8_NORM_LAYER)
        return fail(W8A8_ERR_MODE, "%s: unknown norm kind %d", what, n->kind);
    if (!(n->eps >= 0.0f) || std::isinf(n->eps))
        return fail(W8A8_ERR_SHAPE, "%s: eps must be finite and not negative", what);
    if ((n->weight || n->bias) && !known_dtype(n->vec_dtype))
        return fail(W8A8_ERR_MODE, "%s: unknown type %d of weight and bias", what, n->vec_dtype);
    const bool mod = n->scale || n->shift;
    if (mod && post)
        return fail(W8A8_ERR_MODE, "%s: the norm of the branch takes no scale or shift", what);
    if (mod && !known_dtype(n->mod_dtype))
        return fail(W8A8_ERR_MODE, "%s: unknown type %d of scale and shift", what, n->mod_dtype);
    if (mod && (n->groups < 1 || M % n->groups != 0))
        return fail(W8A8_ERR_SHAPE, "%s: %lld rows do not split into %lld groups of scale and shift", what,
                    (long long)M, (long long)n->groups);
    if (mod && n->groups > 1 && ((n->scale && n->ld_scale < K) || (n->shift && n->ld_shift < K)))
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension of scale or shift smaller than K", what);
    const uintptr_t v = (uintptr_t)size_of(n->vec_dtype), m = (uintptr_t)size_of(n->mod_dtype);
    if ((n->weight && !aligned(n->weight, v)) || (n->bias && !aligned(n->bias, v)) ||
        (n->scale && !aligned(n->scale, m)) || (n->shift && !aligned(n->shift, m)))
        return fail(W8A8_ERR_ALIGN, "%s: vectors must be aligned to their element size", what);
    to.kind = n->kind;
    to.eps = n->eps;
    to.vec_kind = n->vec_dtype;
    to.mod_kind = n->mod_dtype;
    to.weight = n->weight;
    to.bias = n->bias;
    to.scale = n->scale;
    to.shift = n->shift;
    to.ld_scale = n->ld_scale;
    to.ld_shift = n->ld_shift;
    to.group_rows = mod && M > 0 ? M / n->groups : 1;
    return ok();
}

// What norm_modulate, norm_quant_per_token and gated_residual share.
w8a8_status_t rows_args(int64_t M, int64_t K, const char *what)
{
    if (M < 0 || M > kMaxRows)
        return fail(W8A8_ERR_SHAPE, "%s: rows %lld out of range", what, (long long)M);
    if (K < 1 || K > kMaxRows)
        return fail(W8A8_ERR_SHAPE, "%s: K %lld out of range", what, (long long)K);
    return ok();
}

// The norm's output: kind W8A8_NORM_OUT_16 [M, ldo] in act_dtype, or codes
// [M, ldo] with scales [M].
w8a8_status_t out_args(int out_kind, void *out, int64_t ldo, float *out_scale, int64_t M, int64_t K,
                       const char *what, w8a8::NormRowsArgs &a)
{
    if (out_kind != W8A8_NORM_OUT_16 && out_kind != W8A8_NORM_OUT_INT8 && out_kind != W8A8_NORM_OUT_FP8)
        return fail(W8A8_ERR_MODE, "%s: unknown output kind %d", what, out_kind);
    if (ldo < K)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension of the output smaller than K", what);
    const bool codes = out_kind != W8A8_NORM_OUT_16;
    if (M > 0 && (!out || (codes && !out_scale)))
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    if (M > 0 && codes && (!aligned(out, 8) || ldo % 8 != 0 || !aligned(out_scale, 4)))
        return fail(W8A8_ERR_ALIGN, "%s: codes must be 8-byte aligned with ld a multiple of 8, scales 4-byte aligned",
                    what);
    if (M > 0 && !codes && !aligned(out, 2))
        return fail(W8A8_ERR_ALIGN, "%s: output must be aligned to its element size", what);
    a.out = out;
    a.ldo = ldo;
    a.out_scale = out_scale;
    a.out_kind = out_kind;
    return ok();
}

}  // namespace

W8A8_API w8a8_status_t norm_rows(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                                 const w8a8_norm_t *norm, int act_dtype, int out_kind, void *out, int64_t ldo,
                                 float *out_scale, void *stream)
{
    const char *what = "norm_rows";
    if (!known_dtype(x_dtype) || (act_dtype != W8A8_T_BF16 && act_dtype != W8A8_T_F16) ||
        (x_dtype != W8A8_T_F32 && x_dtype != act_dtype))
        return fail(W8A8_ERR_MODE, "%s: element types must be one 16-bit type, or fp32 with a 16-bit type", what);
    w8a8_status_t st = rows_args(M, K, what);
    if (st != W8A8_OK)
        return st;
    if (ldx < K)
        return fail(W8A8_ERR_SHAPE, "%s: ldx smaller than K", what);
    if (!norm || (M > 0 && !x))
        return fail(W8A8_ERR_NULL, "%s: NULL pointer", what);
    if (M > 0 && !aligned(x, (uintptr_t)size_of(x_dtype)))
        return fail(W8A8_ERR_ALIGN, "%s: rows must be aligned to their element size", what);
    w8a8::NormRowsArgs a{};
    st = norm_args(norm, M, K, false, what, a.next);
    if (st != W8A8_OK)
        return st;
    st = out_args(out_kind, out, ldo, out_scale, M, K, what, a);
    if (st != W8A8_OK || M == 0)
        return st;
    a.x = x;
    a.ldx = ldx;
    a.rows = M;
    a.K = K;
    a.x_kind = x_dtype;
    a.act_kind = act_dtype;
    a.post.kind = w8a8::kNormNone;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_norm_rows(a, reinterpret_cast<hipStream_t>(stream)), what);
}

W8A8_API w8a8_status_t gated_residual_rows(const w8a8_residual_t *res, const w8a8_norm_t *post, int64_t M,
                                           int64_t K, const w8a8_norm_t *norm, int out_kind, void *out, int64_t ldo,
                                           float *out_scale, void *stream)
{
    const char *what = "gated_residual_rows";
    if (!res)
        return fail(W8A8_ERR_NULL, "%s: NULL pointer", what);
    if (!known_dtype(res->x_dtype) || (res->y_dtype != W8A8_T_BF16 && res->y_dtype != W8A8_T_F16) ||
        (res->x_dtype != W8A8_T_F32 && res->x_dtype != res->y_dtype))
        return fail(W8A8_ERR_MODE, "%s: element types must be one 16-bit type, or an fp32 x with a 16-bit y", what);
    w8a8_status_t st = rows_args(M, K, what);
    if (st != W8A8_OK)
        return st;
    if (res->ldx < K || res->ldy < K || res->ldr < K)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension smaller than K", what);
    if (M > 0 && (!res->x || !res->y || !res->r))
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    const uintptr_t xs = (uintptr_t)size_of(res->x_dtype);
    if (M > 0 && (!aligned(res->x, xs) || !aligned(res->r, xs) || !aligned(res->y, 2)))
        return fail(W8A8_ERR_ALIGN, "%s: rows must be aligned to their element size", what);
    w8a8::NormRowsArgs a{};
    a.post.kind = a.next.kind = w8a8::kNormNone;
    if (res->gate) {
        if (!known_dtype(res->gate_dtype))
            return fail(W8A8_ERR_MODE, "%s: unknown type %d of the gate", what, res->gate_dtype);
        if (res->gate_groups < 1 || M % res->gate_groups != 0 || (res->gate_groups > 1 && res->ld_gate < K))
            return fail(W8A8_ERR_SHAPE, "%s: %lld rows do not split into %lld groups of the gate, or its leading "
                        "dimension is smaller than K", what, (long long)M, (long long)res->gate_groups);
        if (!aligned(res->gate, (uintptr_t)size_of(res->gate_dtype)))
            return fail(W8A8_ERR_ALIGN, "%s: vectors must be aligned to their element size", what);
        a.gate = res->gate;
        a.gate_kind = res->gate_dtype;
        a.ld_gate = res->ld_gate;
        a.gate_rows = M > 0 ? M / res->gate_groups : 1;
    }
    if (post) {
        st = norm_args(post, M, K, true, what, a.post);
        if (st != W8A8_OK)
            return st;
    }
    if (norm) {
        st = norm_args(norm, M, K, false, what, a.next);
        if (st == W8A8_OK)
            st = out_args(out_kind, out, ldo, out_scale, M, K, what, a);
        if (st != W8A8_OK)
            return st;
    }
    if (M == 0)
        return ok();
    a.x = res->x;
    a.y = res->y;
    a.r = res->r;
    a.ldx = res->ldx;
    a.ldy = res->ldy;
    a.ldr = res->ldr;
    a.rows = M;
    a.K = K;
    a.x_kind = res->x_dtype;
    a.act_kind = res->y_dtype;
    a.residual_scale = res->residual_scale;
    a.branch_scale = res->branch_scale;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_norm_rows(a, reinterpret_cast<hipStream_t>(stream)), what);
}
