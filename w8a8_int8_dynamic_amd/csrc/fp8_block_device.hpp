// What the kernels of the block-scaled product share.
#pragma once

#include "fp8_block.hpp"
#include "fp8_block_rule.hpp"

namespace w8a8 {
namespace fp8_block {

// The 128 products of each of 16 channels with each of 16 tokens, summed: a
// fragment's operand and the tokens', each lane the k-chunks l/16 and 4 + l/16
// of its channel and token l%16. Its sums, as measured on MI355X: of each 8
// neighbouring products the bits below 2^-13 of the largest one's power of two are cut
// off, towards zero; the groups of 8 are added in fp32. That is off by 1.3e-5 of the sums'
// rms for normal values, by 5e-5 where codes are spread evenly over their range.
__device__ __forceinline__ f32x4 block_product(const v4i (&w)[2], const v4i (&x)[2])
{
    const v8i ww = __builtin_shufflevector(w[0], w[1], 0, 1, 2, 3, 4, 5, 6, 7);
    const v8i xx = __builtin_shufflevector(x[0], x[1], 0, 1, 2, 3, 4, 5, 6, 7);
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(ww, xx, f32x4{}, 0, 0, 0, 127, 0, 127);
}

// The same of FN fragments with exact products: both operands as bf16 values,
// which hold an e4m3 value exactly, eight k of a lane at a time.
__device__ __forceinline__ v8bf widen(u32 lo, u32 hi)
{
    v8bf o{};
#if defined(__HIP_DEVICE_COMPILE__)
    const bf16x2 p[4] = {__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false),
                         __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true)};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        o[i] = p[i >> 1][i & 1];
#endif
    return o;
}
// Eight k of a lane, part g of 4.
__device__ __forceinline__ v8bf widen(const v4i (&v)[2], int g)
{
    return widen((u32)v[g >> 1][(g & 1) * 2], (u32)v[g >> 1][(g & 1) * 2 + 1]);
}
template <int FN>
__device__ __forceinline__ void wide_products(const v4i (&w)[FN][2], const v4i (&x)[2], f32x4 (&p)[FN])
{
#pragma unroll
    for (int g = 0; g < 4; ++g) {
        const v8bf xw = widen(x, g);
#pragma unroll
        for (int j = 0; j < FN; ++j)
            p[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen(w[j], g), xw, g == 0 ? f32x4{} : p[j], 0, 0, 0);
    }
}

// Scale row of packed fragment nb.
template <int JOB>
__device__ __forceinline__ int scale_row(int nb, int half_scales)
{
    return JOB == kJobGateUp ? (nb & 1) * half_scales + (nb >> 4) : nb >> 3;
}

// v / (1 + e^-v), on the hardware's 2^x and reciprocal (1 ulp each; their
// argument's rounding adds |v| * 2^-24): within 2^-19 for |v| up to 16, 2^-15 of
// the distance between two codes.
__device__ __forceinline__ float silu(float v)
{
    return v * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(v * -1.44269504f));
}

// Four consecutive outputs of a row from channel n on, with the bias, as OUT
// says (kOutI32: raw fp32).
template <int OUT>
__device__ __forceinline__ void store4(const BlockMmArgs &a, int64_t row, int n, f32x4 v)
{
    const bool whole = a.vec_store && n + 3 < a.N;
    if constexpr (OUT == kOutI32) {
        float *o = static_cast<float *>(a.out) + row * a.ldo + n;
        if (whole) {
            *reinterpret_cast<f32x4 *>(o) = v;
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < a.N)
                    o[r] = v[r];
        }
    } else {
        constexpr bool F16 = OUT == kOutF16;
        if (a.bias) {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const unsigned b = a.bias[min(n + r, a.N - 1)];
                v[r] += F16 ? quant_rule::f16_to_float(b) : __uint_as_float(b << 16);
            }
        }
        const u32 lo = pack2<F16>(v[0], v[1]), hi = pack2<F16>(v[2], v[3]);
        uint16_t *o = static_cast<uint16_t *>(a.out) + row * a.ldo + n;
        if (whole) {
            *reinterpret_cast<uint2 *>(o) = make_uint2(lo, hi);
        } else {
            const u32 hv[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (n + r < a.N)
                    o[r] = (uint16_t)hv[r];
        }
    }
}

}  // namespace fp8_block
}  // namespace w8a8
