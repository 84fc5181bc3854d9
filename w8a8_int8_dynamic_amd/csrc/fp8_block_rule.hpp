// The block-scaled 8-bit rule, shared by the quant, repack and matmul kernels:
// e4m3 codes with one fp32 scale per 128 elements along K (rows), per 128 x
// 128 elements (weights). Over a block
//   a = max |x|;  a < 2^-100 -> scale 0, codes 0;
//   else scale = fl32(a/448), q = e4m3(clamp(fl32(x * f), +-448)),
//        f = fl32(448 * fl32(1/a))
// (quant_rule.hpp's e4m3 rule with a block in place of a row, and the factor by
// way of the reciprocal, as tensor libraries compute a constant over a tensor: f
// differs from fl32(448/a) in its last bit for some a, which moves elements that
// lie halfway between two codes). A block that holds an infinity or NaN gets a scale that is not finite.
//
// Packed weights: fragment F[nb][kb] (kb fastest) is 16 channels x 128 k, 2048
// bytes; unit 16*c + r (16 bytes) holds k 128*kb + 16*c .. +15 of channel 16*nb
// + r, zero outside the weight. A lane l of a wavefront finds its operand of
// v_mfma_scale_f32_16x16x128_f8f6f4 in units l and 64 + l: two loads of 1 KB
// each, every line of them whole, and as LDS images read without bank conflicts.
// That is int8_prepack_weight's layout with an even number of 64-deep
// fragments. Gated weights (gate rows above up rows, [2I, K]) interleave the
// two by fragments: 2*p is 16 gate channels, 2*p + 1 the up channels of the
// same columns, so that one workgroup meets both.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "quant_rule.hpp"

namespace w8a8 {
namespace fp8_block {

using quant_rule::kBF16;
using quant_rule::kF16;
using quant_rule::kF32;
using quant_rule::u32;

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;          // elements per scale along K, and channels per weight scale
constexpr int kFrag = 2048;          // bytes of a packed fragment

// fp32 bit pattern of the largest |x| among 8 elements held as 16-byte words
// (one for the 16-bit kinds, two for fp32).
template <int E>
__device__ __forceinline__ u32 absmax8(const uint4 &lo, const uint4 &hi)
{
    const u32 m = quant_rule::chunk_absmax<E>(lo);
    if (E == kF32)
        return max(m, quant_rule::chunk_absmax<E>(hi));
    return E == kBF16 ? m << 16 : __float_as_uint(quant_rule::f16_to_float(m));
}

// The maximum over each 16 neighbouring lanes, in all of them.
__device__ __forceinline__ u32 row16_max(u32 v)
{
    v = max(v, (u32)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
    v = max(v, (u32)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
    v = max(v, (u32)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x141, 0xF, 0xF, false));   // row_half_mirror
    return max(v, (u32)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x140, 0xF, 0xF, false)); // row_mirror
}

// Scale and factor from the fp32 bit pattern of a block's largest |x|.
__device__ __forceinline__ void scale_of(u32 bits, float &s, float &f)
{
    const float a = __uint_as_float(bits);
    s = a < 0x1p-100f ? 0.0f : a / 448.0f;
    f = a < 0x1p-100f ? 0.0f : (1.0f / a) * 448.0f;
}

// Codes of 8 elements.
template <int E>
__device__ __forceinline__ uint2 codes8(const uint4 &lo, const uint4 &hi, float inv)
{
    uint2 q;
    if constexpr (E == kF32) {
        u32 none;
        quant_rule::chunk_codes<E, true>(lo, inv, q.x, none);
        quant_rule::chunk_codes<E, true>(hi, inv, q.y, none);
    } else {
        quant_rule::chunk_codes<E, true>(lo, inv, q.x, q.y);
    }
    return q;
}

// Two fp32 values rounded to nearest-even 16-bit floats, packed in order.
template <bool F16>
__device__ __forceinline__ u32 pack2(float a, float b)
{
    if constexpr (F16)
        return __builtin_bit_cast(u32, __builtin_convertvector((f32x2){a, b}, f16x2));
    else
        return __builtin_bit_cast(u32, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

}  // namespace fp8_block
}  // namespace w8a8
