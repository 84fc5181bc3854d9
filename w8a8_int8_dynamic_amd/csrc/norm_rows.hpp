// Arithmetic shared by the norm kernels (norm_kernel.hpp): element loads and
// stores with ragged tails, row reductions and the output forms.
#pragma once

#include <utility>

#include "internal.hpp"
#include "quant_rule.hpp"

namespace w8a8 {
namespace norm_rule {

using quant_rule::kBF16;
using quant_rule::kF16;
using quant_rule::kF32;
using quant_rule::u32;

// 16 (or 8) bytes at any element boundary: gfx950 takes unaligned vector
// accesses to global memory, so rows of odd pitch or start need no path of
// their own.
typedef unsigned v4u_any __attribute__((ext_vector_type(4), aligned(2)));
typedef unsigned v2u_any __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// f(std::integral_constant<int, c>) for c = 0 .. N-1: an index that is a
// constant from the start keeps register arrays in registers.
template <class F, int... C>
__device__ __forceinline__ void static_for_impl(F &&f, std::integer_sequence<int, C...>)
{
    (f(std::integral_constant<int, C>{}), ...);
}
template <int N, class F>
__device__ __forceinline__ void static_for(F &&f)
{
    static_for_impl(f, std::make_integer_sequence<int, N>{});
}

template <int E>
__device__ __forceinline__ float widen(u32 bits)
{
    return E == kF32 ? __uint_as_float(bits) : E == kF16 ? quant_rule::f16_to_float(bits) : __uint_as_float(bits << 16);
}

// Elements e .. e+7 of a row of K (zeros past its end; e < K).
template <int E>
__device__ __forceinline__ void load8(const void *row, int64_t e, int64_t K, float (&v)[8])
{
    if (e + 8 <= K) {
        if constexpr (E == kF32) {
            const v4u_any *p = reinterpret_cast<const v4u_any *>(static_cast<const float *>(row) + e);
            const v4u_any a = p[0], b = p[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = __uint_as_float(a[j]);
                v[4 + j] = __uint_as_float(b[j]);
            }
        } else {
            const v4u_any a = *reinterpret_cast<const v4u_any *>(static_cast<const uint16_t *>(row) + e);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[2 * j] = E == kF16 ? widen<E>(a[j]) : __uint_as_float(a[j] << 16);
                v[2 * j + 1] = E == kF16 ? widen<E>(a[j] >> 16) : __uint_as_float(a[j] & 0xffff0000u);
            }
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = 0.0f;
        if (e + j < K)
            v[j] = E == kF32 ? static_cast<const float *>(row)[e + j]
                             : widen<E>(static_cast<const uint16_t *>(row)[e + j]);
    }
}

// The same with the element kind known at run time (uniform over the launch).
__device__ __forceinline__ void load8(const void *row, int kind, int64_t e, int64_t K, float (&v)[8])
{
    if (kind == kF32)
        load8<kF32>(row, e, K, v);
    else if (kind == kF16)
        load8<kF16>(row, e, K, v);
    else
        load8<kBF16>(row, e, K, v);
}

// Two fp32 values rounded to nearest-even 16-bit floats, packed in order.
template <int E>
__device__ __forceinline__ u32 pack2(float a, float b)
{
    if constexpr (E == kF16)
        return __builtin_bit_cast(u32, __builtin_convertvector((f32x2){a, b}, f16x2));
    else
        return __builtin_bit_cast(u32, __builtin_convertvector((f32x2){a, b}, bf16x2));
}

template <int E>
__device__ __forceinline__ void store8(void *row, int64_t e, int64_t K, const float (&v)[8])
{
    if (e + 8 <= K) {
        if constexpr (E == kF32) {
            v4u_any *p = reinterpret_cast<v4u_any *>(static_cast<float *>(row) + e);
            p[0] = v4u_any{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
            p[1] = v4u_any{__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7])};
        } else {
            *reinterpret_cast<v4u_any *>(static_cast<uint16_t *>(row) + e) =
                v4u_any{pack2<E>(v[0], v[1]), pack2<E>(v[2], v[3]), pack2<E>(v[4], v[5]), pack2<E>(v[6], v[7])};
        }
        return;
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (e + j < K) {
            if constexpr (E == kF32)
                static_cast<float *>(row)[e + j] = v[j];
            else
                static_cast<uint16_t *>(row)[e + j] = (uint16_t)pack2<E>(v[j], v[j]);
        }
}

// 1 / sqrt(v) within 1 ulp. v_rsq_f32 takes a subnormal for zero, so one is
// lifted into the normal range first, by a power of two whose root is exact;
// other values are multiplied by 1.
__device__ __forceinline__ float rsqrt_of(float v)
{
    const bool low = v < 0x1p-126f;
    return __builtin_amdgcn_rsqf(low ? v * 0x1p24f : v) * (low ? 0x1p12f : 1.0f);
}

// Sum over a wavefront, the same in every lane and every run: within rows of
// 16 lanes by exchanges, then the four row sums in one fixed order.
__device__ __forceinline__ float wave_sum(float v)
{
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x141, 0xF, 0xF, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x140, 0xF, 0xF, false));
    const int b = __float_as_int(v);
    return (__int_as_float(__builtin_amdgcn_readlane(b, 0)) + __int_as_float(__builtin_amdgcn_readlane(b, 16))) +
           (__int_as_float(__builtin_amdgcn_readlane(b, 32)) + __int_as_float(__builtin_amdgcn_readlane(b, 48)));
}

}  // namespace norm_rule
}  // namespace w8a8
