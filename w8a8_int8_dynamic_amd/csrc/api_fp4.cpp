// C ABI of the microscaled 4-bit (MX FP4) layer: argument checks and dispatch
// (declared in include/w8a8.h).
#include "api.hpp"

using namespace w8a8::api;

namespace {

constexpr int64_t kBlock = 32;

bool known_dtype(int t) { return t == W8A8_T_BF16 || t == W8A8_T_F32 || t == W8A8_T_F16; }

w8a8_status_t fp4_shape(int64_t rows, int64_t K, int64_t least_rows, const char *what)
{
    if (rows < least_rows || rows > kMaxRows)
        return fail(W8A8_ERR_SHAPE, "%s: rows %lld out of range", what, (long long)rows);
    if (K < kBlock || K > kMaxRows || K % kBlock != 0)
        return fail(W8A8_ERR_SHAPE, "%s: K must be a multiple of %lld, from %lld on", what, (long long)kBlock,
                    (long long)kBlock);
    return ok();
}

// Rows of elements: 16-byte aligned, the pitch a multiple of 16 bytes.
w8a8_status_t fp4_rows(const void *x, int dtype, int64_t ldx, const char *what)
{
    const int64_t vec = dtype == W8A8_T_F32 ? 4 : 8;
    if (!aligned(x, 16) || ldx % vec != 0)
        return fail(W8A8_ERR_ALIGN, "%s: rows must be 16-byte aligned with ld a multiple of %lld", what,
                    (long long)vec);
    return ok();
}

w8a8_status_t quant_args(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx, const uint8_t *xq,
                         int64_t ldq, const uint8_t *x_scale, int64_t lds, const char *what)
{
    if (!known_dtype(x_dtype))
        return fail(W8A8_ERR_MODE, "%s: unknown element type %d", what, x_dtype);
    w8a8_status_t st = fp4_shape(M, K, 0, what);
    if (st != W8A8_OK)
        return st;
    if (ldx < K || ldq < K / 2 || lds < K / kBlock)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    if (M == 0)
        return ok();
    if (!x || !xq || !x_scale)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    st = fp4_rows(x, x_dtype, ldx, what);
    if (st != W8A8_OK)
        return st;
    if (!aligned(xq, 4) || ldq % 4 != 0)
        return fail(W8A8_ERR_ALIGN, "%s: codes must be 4-byte aligned with ldq a multiple of 4", what);
    return ok();
}

w8a8_status_t pack_args(int64_t N, int64_t K, const void *a, const void *b, const void *packed,
                        const void *s_packed, const char *what)
{
    w8a8_status_t st = fp4_shape(N, K, 1, what);
    if (st != W8A8_OK)
        return st;
    if (fp4_prepack_weight_bytes(N, K) == 0)
        return fail(W8A8_ERR_SHAPE, "%s: packed size overflows", what);
    if (!a || !b || !packed || !s_packed)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    if (!aligned(packed, 16) || !aligned(s_packed, 16))
        return fail(W8A8_ERR_ALIGN, "%s: packed buffers must be 16-byte aligned", what);
    return ok();
}

// The matmul's arguments, checked, and the tile.
w8a8_status_t mm_args(const uint8_t *xq, int64_t ldq, const uint8_t *x_scale, int64_t lds, const void *w_packed,
                      const void *s_packed, const uint16_t *bias, int64_t M, int64_t N, int64_t K, int mode,
                      void *out, int64_t ldo, int tile, const char *what, w8a8::MmArgs &a, int &t)
{
    if (mode != W8A8_OUT_BF16 && mode != W8A8_OUT_I32 && mode != W8A8_OUT_F16)
        return fail(W8A8_ERR_MODE, "%s: unknown output mode %d", what, mode);
    if (tile < -1 || tile >= w8a8::fp4_tile_count())
        return fail(W8A8_ERR_MODE, "%s: unknown tile %d", what, tile);
    if (M < 0 || M > kMaxRows || N < 1 || N > kMaxRows)
        return fail(W8A8_ERR_SHAPE, "%s: M or N out of range", what);
    if (K < kBlock || K > W8A8_FP4_MAX_K || K % kBlock != 0)
        return fail(W8A8_ERR_SHAPE, "%s: K must be a multiple of %lld in [%lld, %d]", what, (long long)kBlock,
                    (long long)kBlock, W8A8_FP4_MAX_K);
    if (ldq < K / 2 || lds < K / kBlock || ldo < N)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    if (ldq > W8A8_MAX_LDQ || lds > W8A8_MAX_LDQ)
        return fail(W8A8_ERR_SHAPE, "%s: ldq or lds above %d", what, W8A8_MAX_LDQ);
    a = w8a8::MmArgs{};
    t = -1;
    if (M == 0)
        return ok();
    if (!xq || !x_scale || !w_packed || !s_packed || !out)
        return fail(W8A8_ERR_NULL, "%s: NULL tensor pointer", what);
    if (!aligned(xq, 16) || ldq % 16 != 0 || !aligned(w_packed, 16) || !aligned(s_packed, 16))
        return fail(W8A8_ERR_ALIGN, "%s: codes and packed buffers must be 16-byte aligned, ldq a multiple of 16",
                    what);
    if (!aligned(x_scale, 16) || lds % 16 != 0)
        return fail(W8A8_ERR_ALIGN, "%s: token scales must be 16-byte aligned with lds a multiple of 16", what);
    const bool raw = mode == W8A8_OUT_I32;
    const uintptr_t esz = raw ? 4 : 2;
    if (!aligned(out, esz) || (!raw && bias && !aligned(bias, 2)))
        return fail(W8A8_ERR_ALIGN, "%s: out and bias must be aligned to their element size", what);
    t = tile >= 0 ? tile : w8a8::fp4_tile_auto(M, N, K);
    if (!w8a8::fp4_launch_fits(t, M, N))
        return fail(W8A8_ERR_SHAPE, "%s: M x N needs more workgroups of tile %d than one launch holds", what, t);
    a.xq = reinterpret_cast<const int8_t *>(xq);
    a.wp = reinterpret_cast<const int8_t *>(w_packed);
    a.sx = x_scale;
    a.sw = reinterpret_cast<const uint8_t *>(s_packed);
    a.bias = raw ? nullptr : bias;
    a.out = out;
    a.ldq = ldq;
    a.lds = lds;
    a.ldo = ldo;
    a.M = (int)M;
    a.N = (int)N;
    a.K = (int)(K / 2);
    a.blocks = (int)(K / kBlock);
    a.kblocks = (int)w8a8::ceil_div(K / 2, w8a8::kFragK);
    a.nblocks = (int)w8a8::ceil_div(N, w8a8::kFragN);
    const uintptr_t vw = 4 * esz;
    a.vec_store = aligned(out, vw) && ((uint64_t)ldo * esz) % vw == 0;
    a.vec16 = aligned(out, 16) && ((uint64_t)ldo * esz) % 16 == 0;
    return ok();
}

}  // namespace

W8A8_API w8a8_status_t fp4_quant_per_block(const void *x, int x_dtype, int64_t M, int64_t K, int64_t ldx,
                                           uint8_t *xq, int64_t ldq, uint8_t *x_scale, int64_t lds, void *stream)
{
    const char *what = "fp4_quant_per_block";
    w8a8_status_t st = quant_args(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds, what);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_quant_fp4(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds,
                                           reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp4_dequant(const uint8_t *xq, int64_t ldq, const uint8_t *x_scale, int64_t lds, int64_t M,
                                   int64_t K, int out_dtype, void *out, int64_t ldo, void *stream)
{
    const char *what = "fp4_dequant";
    w8a8_status_t st = quant_args(out, out_dtype, M, K, ldo, xq, ldq, x_scale, lds, what);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_dequant_fp4(xq, ldq, x_scale, lds, M, K, out_dtype, out, ldo,
                                             reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API size_t fp4_prepack_weight_bytes(int64_t N, int64_t K)
{
    return K < kBlock || K % kBlock != 0 ? 0 : int8_prepack_weight_bytes(N, K / 2);
}

W8A8_API size_t fp4_prepack_scale_bytes(int64_t N, int64_t K)
{
    if (fp4_prepack_weight_bytes(N, K) == 0)
        return 0;
    return (size_t)(w8a8::ceil_div(N, 16) * w8a8::ceil_div(K, 512) * 256);
}

W8A8_API w8a8_status_t fp4_prepack_weight(const uint8_t *wq, int64_t ldq, const uint8_t *w_scale, int64_t lds,
                                          int64_t N, int64_t K, void *w_packed, void *s_packed, void *stream)
{
    const char *what = "fp4_prepack_weight";
    w8a8_status_t st = pack_args(N, K, wq, w_scale, w_packed, s_packed, what);
    if (st != W8A8_OK)
        return st;
    if (ldq < K / 2 || lds < K / kBlock)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_prepack_fp4(wq, -1, w_scale, N, K, ldq, lds, w_packed, s_packed,
                                             reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp4_quant_prepack_weight(const void *w, int w_dtype, int64_t N, int64_t K, int64_t ldw,
                                                void *w_packed, void *s_packed, void *stream)
{
    const char *what = "fp4_quant_prepack_weight";
    if (w_dtype != W8A8_W_F32 && w_dtype != W8A8_W_BF16)
        return fail(W8A8_ERR_MODE, "%s: unknown weight dtype %d", what, w_dtype);
    w8a8_status_t st = pack_args(N, K, w, w, w_packed, s_packed, what);
    if (st != W8A8_OK)
        return st;
    if (ldw < K)
        return fail(W8A8_ERR_SHAPE, "%s: ldw smaller than K", what);
    const int kind = w_dtype == W8A8_W_F32 ? w8a8::kElemF32 : w8a8::kElemBF16;
    st = fp4_rows(w, kind, ldw, what);
    if (st != W8A8_OK)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_prepack_fp4(w, kind, nullptr, N, K, ldw, 0, w_packed, s_packed,
                                             reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp4_unpack_weight(const void *w_packed, const void *s_packed, int64_t N, int64_t K,
                                         uint8_t *wq, int64_t ldq, uint8_t *w_scale, int64_t lds, void *stream)
{
    const char *what = "fp4_unpack_weight";
    w8a8_status_t st = pack_args(N, K, wq, w_scale, w_packed, s_packed, what);
    if (st != W8A8_OK)
        return st;
    if (ldq < K / 2 || lds < K / kBlock)
        return fail(W8A8_ERR_SHAPE, "%s: leading dimension too small", what);
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_unpack_fp4(w_packed, s_packed, N, K, wq, ldq, w_scale, lds,
                                            reinterpret_cast<hipStream_t>(stream)),
                    what);
}

W8A8_API w8a8_status_t fp4_scaled_mm_tile(const uint8_t *xq, int64_t ldq, const uint8_t *x_scale, int64_t lds,
                                          const void *w_packed, const void *s_packed, const uint16_t *bias,
                                          int64_t M, int64_t N, int64_t K, int mode, void *out, int64_t ldo,
                                          void *stream, int tile)
{
    const char *what = "fp4_scaled_mm";
    w8a8::MmArgs a;
    int t;
    w8a8_status_t st = mm_args(xq, ldq, x_scale, lds, w_packed, s_packed, bias, M, N, K, mode, out, ldo, tile,
                               what, a, t);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    return launched(w8a8::launch_scaled_mm_fp4(a, mode, t, reinterpret_cast<hipStream_t>(stream)), what);
}

W8A8_API w8a8_status_t fp4_scaled_mm(const uint8_t *xq, int64_t ldq, const uint8_t *x_scale, int64_t lds,
                                     const void *w_packed, const void *s_packed, const uint16_t *bias, int64_t M,
                                     int64_t N, int64_t K, int mode, void *out, int64_t ldo, void *stream)
{
    return fp4_scaled_mm_tile(xq, ldq, x_scale, lds, w_packed, s_packed, bias, M, N, K, mode, out, ldo, stream,
                              -1);
}

W8A8_API w8a8_status_t fp4_quant_scaled_mm_tile(const void *x, int x_dtype, int64_t ldx, uint8_t *xq, int64_t ldq,
                                                uint8_t *x_scale, int64_t lds, const void *w_packed,
                                                const void *s_packed, const uint16_t *bias, int64_t M, int64_t N,
                                                int64_t K, int mode, void *out, int64_t ldo, void *stream, int tile)
{
    const char *what = "fp4_quant_scaled_mm";
    w8a8::MmArgs a;
    int t;
    w8a8_status_t st = mm_args(xq, ldq, x_scale, lds, w_packed, s_packed, bias, M, N, K, mode, out, ldo, tile,
                               what, a, t);
    if (st != W8A8_OK)
        return st;
    st = quant_args(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds, what);
    if (st != W8A8_OK || M == 0)
        return st;
    st = check_device();
    if (st != W8A8_OK)
        return st;
    hipStream_t s = reinterpret_cast<hipStream_t>(stream);
    a.x = reinterpret_cast<const uint16_t *>(x);
    a.ldx = ldx;
    hipError_t err = w8a8::launch_quant_scaled_mm_fp4(a, x_dtype, mode, t, s);
    if (err != hipErrorNotSupported)
        return launched(err, what);
    a.x = nullptr;
    err = w8a8::launch_quant_fp4(x, x_dtype, M, K, ldx, xq, ldq, x_scale, lds, s);
    if (err != hipSuccess)
        return launched(err, what);
    return launched(w8a8::launch_scaled_mm_fp4(a, mode, t, s), what);
}

W8A8_API w8a8_status_t fp4_quant_scaled_mm(const void *x, int x_dtype, int64_t ldx, uint8_t *xq, int64_t ldq,
                                           uint8_t *x_scale, int64_t lds, const void *w_packed,
                                           const void *s_packed, const uint16_t *bias, int64_t M, int64_t N,
                                           int64_t K, int mode, void *out, int64_t ldo, void *stream)
{
    return fp4_quant_scaled_mm_tile(x, x_dtype, ldx, xq, ldq, x_scale, lds, w_packed, s_packed, bias, M, N, K,
                                    mode, out, ldo, stream, -1);
}

W8A8_API int w8a8_fp4_tile_count(void) { return w8a8::fp4_tile_count(); }

W8A8_API const char *w8a8_fp4_tile_name(int tile)
{
    return tile >= 0 && tile < w8a8::fp4_tile_count() ? w8a8::fp4_tile_name(tile) : "";
}

W8A8_API int w8a8_fp4_tile_auto(int64_t M, int64_t N, int64_t K)
{
    return w8a8::fp4_tile_auto(M, N, K);
}
