// The microscaled 4-bit (MX FP4) rule, shared by the quant, repack and
// matmul kernels (the published OCP Microscaling Formats specification v1.0:
// blocks of 32 elements along K, e2m1 elements, one e8m0 scale per block):
//   a = max |x| over the block;  byte = clamp(floor(log2 a) - 2 + 127, 0, 254)
//   code = e2m1(x / 2^(byte - 127)), nearest, ties to even, saturated at 6,
//   the sign kept (zeros too); a = 0 gives byte 0.
// A block that holds an infinity or NaN gets byte 255 (the format's NaN) and
// codes 0. Every step is exact but the one rounding to e2m1: 2 is e2m1's
// largest exponent, so the largest element lands in [4, 8) and x / 2^e is a
// change of exponent alone.
// Codes go two to a byte, the even element in the low nibble.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "quant_rule.hpp"

namespace w8a8 {
namespace fp4_rule {

using quant_rule::kBF16;
using quant_rule::kF16;
using quant_rule::kF32;
using quant_rule::u32;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 32;       // elements per scale

// Scale byte from the fp32 bit pattern of a block's largest |x| (positive):
// the exponent field less 2, from 0 up (fp32 subnormals have field 0, and
// floor(log2) below -125 is clamped there anyway).
__device__ __forceinline__ u32 scale_byte(u32 bits)
{
    const u32 e = bits >> 23;
    return e == 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// 2^(byte - 127) as fp32; byte 0 is the subnormal 2^-127.
__device__ __forceinline__ float scale_value(u32 byte)
{
    return __uint_as_float(byte == 0 ? 0x00400000u : byte << 23);
}

// fp32 bit pattern of the largest |x| among 8 elements held as 16-byte
// words (one word quad for the 16-bit kinds, two for fp32).
template <int E>
__device__ __forceinline__ u32 absmax8(const uint4 &lo, const uint4 &hi)
{
    u32 m = quant_rule::chunk_absmax<E>(lo);
    if (E == kF32)
        return max(m, quant_rule::chunk_absmax<E>(hi));
    return E == kBF16 ? m << 16 : __float_as_uint(quant_rule::f16_to_float(m));
}

// Codes of 8 elements (element j in bits 4j .. 4j+3). gfx950's conversions
// divide by the scale and round to e2m1 to nearest even with saturation,
// two elements at a time; checked on MI355X against the rule for every
// bf16 and fp16 pattern and scales 2^-127 .. 2^127.
template <int E>
__device__ __forceinline__ u32 codes8(const uint4 &lo, const uint4 &hi, u32 byte)
{
    if (byte == 255u)
        return 0;
    const float s = scale_value(byte);
    const u32 a[4] = {lo.x, lo.y, lo.z, lo.w}, b[4] = {hi.x, hi.y, hi.z, hi.w};
    u32 q = 0;
    if constexpr (E == kBF16) {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, a[0]), s, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, a[1]), s, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, a[2]), s, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(q, __builtin_bit_cast(bf16x2, a[3]), s, 3);
    } else if constexpr (E == kF16) {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, a[0]), s, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, a[1]), s, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, a[2]), s, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(q, __builtin_bit_cast(f16x2, a[3]), s, 3);
    } else {
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(a[0]), __uint_as_float(a[1]), s, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(a[2]), __uint_as_float(a[3]), s, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(b[0]), __uint_as_float(b[1]), s, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, __uint_as_float(b[2]), __uint_as_float(b[3]), s, 3);
    }
    return q;
}

// The value of one code times the scale, in fp32 (exact unless it leaves
// fp32's range). Twice the magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6 are whole
// numbers of one hexadecimal digit each.
__device__ __forceinline__ float code_value(u32 code, float scale)
{
    const float v = (float)((0xC8643210u >> (4 * (code & 7u))) & 15u) * 0.5f;
    return (code & 8u ? -v : v) * scale;
}

}  // namespace fp4_rule
}  // namespace w8a8
