// C ABI of the block-scaled 8-bit layer: argument checks and dispatch (declared
// in include/w8a8.h).
#include "api.hpp"
#include "fp8_block.hpp"

using namespace w8a8::api;

namespace {

constexpr int64_t kStep = 16, kBlock = 128;

bool known_dtype(int t) { return t == W8A8_T_BF16 || t == W8A8_T_F32 || t == W8A8_T_F16; }

w8a8_status_t check_k(int64_t K, const char *what)
{
    if (K < kStep || K > W8A8_MAX_K || K % kStep != 0)
        return fail(W8A8_ERR_SHAPE, "%s: K must be a multiple of %lld in [%lld, %d]", what, (long long)kStep,
                    (long long)kStep, W8A8_MAX_K);
    return ok();
}

// Rows of floats x, their codes and scales.
w8a8_status_t quant_args(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t *xq,
                         int64_t ldq, const float *x_scale, int64_t lds, const char *what)
{
    if (!known_dtype(x_dtype))
        return fail(W8A8_ERR_MODE, "%s: unknown element type %d", what, x_dtype);
    if (M < 0 || M > kMaxRows)
        return fail(W8A8_ERR_SHAPE, "%s: rows %lld out of range", what, (long long)M);
    w8a8_status_t st = check_k(K, what);
    if (st != W8A8_OK)
        return st;
    if (ldx < K || ldq < K || lds < w8a8::ceil_div(K, kBlock))
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    if (M == 0)
        return ok();
    if (!x || !xq || !x_scale)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    const int64_t vec = x_dtype == W8A8_T_F32 ? 4 : 8;
    if (!aligned(x, 16) || ldx % vec != 0)
        return fail(W8A8_ERR_ALIGN, "%s: rows must be 16-byte aligned with ld a multiple of %lld", what,
                    (long long)vec);
    if (!aligned(xq, 8) || ldq % 8 != 0 || !aligned(x_scale, 4))
        return fail(W8A8_ERR_ALIGN, "%s: codes must be 8-byte aligned with ldq a multiple of 8, scales 4-byte", what);
    return ok();
}

// A weight [experts, N, K] and its packed buffer.
w8a8_status_t pack_args(int64_t experts, int64_t N, int64_t K, int gated, const void *a, const void *packed,
                        const char *what)
{
    w8a8_status_t st = check_k(K, what);
    if (st != W8A8_OK)
        return st;
    if (experts < 1 || N < 1 || N > kMaxRows || (gated && N % 32 != 0))
        return fail(W8A8_ERR_SHAPE, "%s: experts or N out of range (gated: N a multiple of 32)", what);
    if (fp8_block_prepack_weight_bytes(experts, N, K) == 0)
        return fail(W8A8_ERR_SHAPE, "%s: packed size overflows", what);
    if (!a || !packed)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    if (!aligned(packed, 16))
        return fail(W8A8_ERR_ALIGN, "%s: the packed buffer must be 16-byte aligned", what);
    return ok();
}

// The matmul's arguments, checked, and the tile.
w8a8_status_t mm_args(const uint8_t *xq, int64_t ldq, const float *x_scale, int64_t lds, const void *w_packed,
                      const float *w_scale, const uint16_t *bias, int64_t M, int64_t N, int64_t K, int mode, void *out,
                      int64_t ldo, int tile, const char *what, w8a8::BlockMmArgs &a, int &t)
{
    if (mode != W8A8_OUT_BF16 && mode != W8A8_OUT_I32 && mode != W8A8_OUT_F16)
        return fail(W8A8_ERR_MODE, "%s: unknown output mode %d", what, mode);
    if (tile < -1 || tile >= w8a8::fp8_block_tile_count())
        return fail(W8A8_ERR_MODE, "%s: unknown tile %d", what, tile);
    if (M < 0 || M > kMaxRows || N < 1 || N > kMaxRows)
        return fail(W8A8_ERR_SHAPE, "%s: M or N out of range", what);
    w8a8_status_t st = check_k(K, what);
    if (st != W8A8_OK)
        return st;
    if (ldq < K || lds < w8a8::ceil_div(K, kBlock) || ldo < N)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    if (ldq > W8A8_MAX_LDQ || lds > W8A8_MAX_LDQ / 4)
        return fail(W8A8_ERR_SHAPE, "%s: ldq above %d or lds above a quarter of that", what, W8A8_MAX_LDQ);
    a = w8a8::BlockMmArgs{};
    t = -1;
    if (M == 0)
        return ok();
    if (!xq || !x_scale || !w_packed || !w_scale || !out)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    if (!aligned(xq, 16) || ldq % 16 != 0 || !aligned(w_packed, 16))
        return fail(W8A8_ERR_ALIGN, "%s: codes and the packed weight must be 16-byte aligned, ldq a multiple of 16",
                    what);
    if (!aligned(x_scale, 16) || lds % 4 != 0)
        return fail(W8A8_ERR_ALIGN, "%s: token scales must be 16-byte aligned with lds a multiple of 4", what);
    const bool raw = mode == W8A8_OUT_I32;
    const uintptr_t esz = raw ? 4 : 2;
    if (!aligned(w_scale, 4) || !aligned(out, esz) || (!raw && bias && !aligned(bias, 2)))
        return fail(W8A8_ERR_ALIGN, "%s: scales, out and bias must be aligned to their element size", what);
    t = tile >= 0 ? tile : w8a8::fp8_block_tile_auto(M, N, K);
    const w8a8::BlockTileEntry &e = w8a8::fp8_block_tile(t);
    if (!w8a8::mm_grid_fits(w8a8::ceil_div(M, e.bm) * w8a8::ceil_div(N, e.bn), e.threads))
        return fail(W8A8_ERR_SHAPE, "%s: M x N needs more workgroups of tile %d than one launch holds", what, t);
    a.xq = xq;
    a.xs = x_scale;
    a.wp = static_cast<const uint8_t *>(w_packed);
    a.ws = w_scale;
    a.bias = raw ? nullptr : bias;
    a.out = out;
    a.ldq = ldq;
    a.lds = lds;
    a.ldo = ldo;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)K;
    a.blocks = (int)w8a8::ceil_div(K, kBlock);
    a.frags = (int)w8a8::fp8_block_frags(N, false);
    const uintptr_t vw = 4 * esz;
    a.vec_store = aligned(out, vw) && ((uint64_t)ldo * esz) % vw == 0;
    a.vec16 = aligned(out, 16) && ((uint64_t)ldo * esz) % 16 == 0;
    return ok();
}

}  // namespace

W8A8_API w8a8_status_t fp8_quant_per_block(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx, uint8_t *xq,
                                           int64_t ldq, float *x_scale, int64_t lds, void *stream)
{
    const char *what = "fp8_quant_per_block";
    w8a8_status_t st = quant_args(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds, what);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_quant_fp8_block(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds,
                                                 reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp8_block_dequant(const uint8_t *xq, int64_t ldq, const float *x_scale, int64_t lds, int64_t M,
                                         int64_t K, int out_dtype, void *out, int64_t ldo, void *stream)
{
    const char *what = "fp8_block_dequant";
    w8a8_status_t st = quant_args(out, out_dtype, M, K, ldo, xq, ldq, x_scale, lds, what);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_dequant_fp8_block(xq, ldq, x_scale, lds, M, K, out_dtype, out, ldo,
                                                   reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API size_t fp8_block_prepack_weight_bytes(int64_t experts, int64_t N, int64_t K)
{
    if (experts < 1 || N < 1 || N > kMaxRows || K < kStep || K > W8A8_MAX_K || K % kStep != 0)
        return 0;
    const int64_t one = w8a8::ceil_div(N, 16) * w8a8::ceil_div(K, kBlock) * 2048;
    return experts > std::numeric_limits<int64_t>::max() / one ? 0 : (size_t)(experts * one);
}

W8A8_API w8a8_status_t fp8_block_prepack_weight(const uint8_t *wq, int64_t ldq, int64_t experts, int64_t N, int64_t K,
                                                int gated, void *w_packed, void *stream)
{
    const char *what = "fp8_block_prepack_weight";
    w8a8_status_t st = pack_args(experts, N, K, gated, wq, w_packed, what);
    if (st != W8A8_OK)
        return st;
    if (ldq < K)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_repack_fp8_block(const_cast<uint8_t *>(wq), ldq, experts, N, K, gated != 0, w_packed,
                                                  true, reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp8_block_unpack_weight(const void *w_packed, int64_t experts, int64_t N, int64_t K, int gated,
                                               uint8_t *wq, int64_t ldq, void *stream)
{
    const char *what = "fp8_block_unpack_weight";
    w8a8_status_t st = pack_args(experts, N, K, gated, wq, w_packed, what);
    if (st != W8A8_OK)
        return st;
    if (ldq < K)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_repack_fp8_block(wq, ldq, experts, N, K, gated != 0, const_cast<void *>(w_packed),
                                                  false, reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp8_block_quant_prepack_weight(const void *w, int w_dtype, int64_t ldw, int64_t experts,
                                                      int64_t N, int64_t K, int gated, void *w_packed, float *w_scale,
                                                      void *stream)
{
    const char *what = "fp8_block_quant_prepack_weight";
    if (w_dtype != W8A8_W_F32 && w_dtype != W8A8_W_BF16)
        return fail(W8A8_ERR_MODE, "%s: unknown weight dtype %d", what, w_dtype);
    w8a8_status_t st = pack_args(experts, N, K, gated, w, w_packed, what);
    if (st != W8A8_OK)
        return st;
    if (!w_scale)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    if (ldw < K)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    const bool f32 = w_dtype == W8A8_W_F32;
    if (!aligned(w, 16) || ldw % (f32 ? 4 : 8) != 0 || !aligned(w_scale, 4))
        return fail(W8A8_ERR_ALIGN, "%s: weight rows must be 16-byte aligned with ldw a multiple of %d", what,
                    f32 ? 4 : 8);
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_quant_prepack_fp8_block(w, f32, ldw, experts, N, K, gated != 0, w_packed, w_scale,
                                                         reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp8_block_scaled_mm_tile(const uint8_t *xq, int64_t ldq, const float *x_scale, int64_t lds,
                                                const void *w_packed, const float *w_scale, const uint16_t *bias,
                                                int64_t M, int64_t N, int64_t K, int mode, void *out, int64_t ldo,
                                                void *stream, int tile)
{
    const char *what = "fp8_block_scaled_mm";
    w8a8::BlockMmArgs a;
    int t;
    w8a8_status_t st = mm_args(xq, ldq, x_scale, lds, w_packed, w_scale, bias, M, N, K, mode, out, ldo, tile, what, a,
                               t);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_fp8_block_mm(a, mode, t, reinterpret_cast<hipStream_t>(stream)), what);
}

W8A8_API w8a8_status_t fp8_block_scaled_mm(const uint8_t *xq, int64_t ldq, const float *x_scale, int64_t lds,
                                           const void *w_packed, const float *w_scale, const uint16_t *bias, int64_t M,
                                           int64_t N, int64_t K, int mode, void *out, int64_t ldo, void *stream)
{
    return fp8_block_scaled_mm_tile(xq, ldq, x_scale, lds, w_packed, w_scale, bias, M, N, K, mode, out, ldo, stream,
                                    -1);
}

W8A8_API w8a8_status_t fp8_block_quant_scaled_mm_tile(const void *x, int x_dtype, int64_t ldx, uint8_t *xq,
                                                      int64_t ldq, float *x_scale, int64_t lds, const void *w_packed,
                                                      const float *w_scale, const uint16_t *bias, int64_t M, int64_t N,
                                                      int64_t K, int mode, void *out, int64_t ldo, void *stream,
                                                      int tile)
{
    const char *what = "fp8_block_quant_scaled_mm";
    w8a8::BlockMmArgs a;
    int t;
    w8a8_status_t st = mm_args(xq, ldq, x_scale, lds, w_packed, w_scale, bias, M, N, K, mode, out, ldo, tile, what, a,
                               t);
    if (st != W8A8_OK)
        return st;
    st = quant_args(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds, what);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    a.x = x;
    a.ldx = ldx;
    hipError_t err = w8a8::launch_fp8_block_quant_mm(a, x_dtype, mode, t, s);
    if (err != hipErrorNotSupported)
        return launched(err, what);
    err = w8a8::launch_quant_fp8_block(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds, s);
    if (err != hipSuccess)
        return launched(err, what);
    return launched(w8a8::launch_fp8_block_mm(a, mode, t, s), what);
}

W8A8_API w8a8_status_t fp8_block_quant_scaled_mm(const void *x, int x_dtype, int64_t ldx, uint8_t *xq, int64_t ldq,
                                                 float *x_scale, int64_t lds, const void *w_packed,
                                                 const float *w_scale, const uint16_t *bias, int64_t M, int64_t N,
                                                 int64_t K, int mode, void *out, int64_t ldo, void *stream)
{
    return fp8_block_quant_scaled_mm_tile(x, x_dtype, ldx, xq, ldq, x_scale, lds, w_packed, w_scale, bias, M, N, K,
                                          mode, out, ldo, stream, -1);
}

W8A8_API int w8a8_fp8_block_tile_count(void) { return w8a8::fp8_block_tile_count(); }

W8A8_API const char *w8a8_fp8_block_tile_name(int tile)
{
    return tile >= 0 && tile < w8a8::fp8_block_tile_count() ? w8a8::fp8_block_tile(tile).name : "";
}

W8A8_API int w8a8_fp8_block_tile_auto(int64_t M, int64_t N, int64_t K)
{
    return w8a8::fp8_block_tile_auto(M, N, K);
}
