// Norms around a quantized layer, on gfx950: the modulated norm in front of a
// block, and the gate, residual scale and norm behind it with the next block's
// norm in the same pass (NormRowsArgs in internal.hpp):
//   rms:   n(v) = v * rsqrt(mean(v^2) + eps)
//   layer: n(v) = (v - mean(v)) * rsqrt(mean((v - mean(v))^2) + eps)
//   next(v) = (n(v) * weight + bias) * (1 + scale) + shift
// All in fp32, with the variance taken around the mean in a second pass over
// the values; each output is rounded once, and the codes come from the fp32
// values by the rule of int8_quant_per_token / fp8_quant_per_token.
//
// The simplest form: one workgroup per row, which reads the row again (from
// L2) for each of its passes. It writes nothing before its last pass, so r
// may be x itself.
#include "norm_rows.hpp"

namespace w8a8 {
namespace {

using namespace norm_rule;

__device__ __forceinline__ float block_sum(float v, float *part)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// Mean (0 for rms) and reciprocal deviation of the K values that `value`
// yields, 8 at a time.
template <class F>
__device__ __forceinline__ void stats(F &&value, int64_t K, int kind, float eps, float *part, float &mean, float &inv)
{
    mean = 0.0f;
    if (kind == kNormLayer) {
        float s = 0.0f;
        for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
            float v[8];
            value(e, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += e + j < K ? v[j] : 0.0f;
        }
        mean = block_sum(s, part) / (float)K;
    }
    float q = 0.0f;
    for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
        float v[8];
        value(e, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = e + j < K ? v[j] - mean : 0.0f;
            q += d * d;
        }
    }
    inv = 1.0f / sqrtf(block_sum(q, part) / (float)K + eps);
}

// (v - mean) * inv * weight + bias, then * (1 + scale) + shift.
__device__ __forceinline__ void apply(const NormVectors &n, int64_t row, int64_t e, int64_t K, float mean, float inv,
                                      float (&v)[8])
{
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = (v[j] - mean) * inv;
    if (n.weight) {
        load8(n.weight, n.vec_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= t[j];
    }
    if (n.bias) {
        load8(n.bias, n.vec_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] += t[j];
    }
    const int64_t g = n.scale || n.shift ? row / n.group_rows : 0;
    const int bytes = n.mod_kind == kF32 ? 4 : 2;
    if (n.scale) {
        load8(static_cast<const char *>(n.scale) + g * n.ld_scale * bytes, n.mod_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= 1.0f + t[j];
    }
    if (n.shift) {
        load8(static_cast<const char *>(n.shift) + g * n.ld_shift * bytes, n.mod_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] += t[j];
    }
}

template <int XE, int AE, bool RES>
__global__ __launch_bounds__(256) void norm_rows_looped_kernel(const NormRowsArgs a)
{
    __shared__ float part[4];
    __shared__ u32 most;
    const int64_t K = a.K;
    constexpr int XB = XE == kF32 ? 4 : 2;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char *x = static_cast<const char *>(a.x) + row * a.ldx * XB;
        const char *y = RES ? static_cast<const char *>(a.y) + row * a.ldy * 2 : nullptr;
        const char *gate = nullptr;
        if (RES && a.gate)
            gate = static_cast<const char *>(a.gate) + row / a.gate_rows * a.ld_gate * (a.gate_kind == kF32 ? 4 : 2);
        float pmean = 0.0f, pinv = 1.0f;
        if (RES && a.post.kind != kNormNone)
            stats([&](int64_t e, float (&v)[8]) { load8<AE>(y, e, K, v); }, K, a.post.kind, a.post.eps, part, pmean,
                  pinv);
        auto value = [&](int64_t e, float (&v)[8]) {
            load8<XE>(x, e, K, v);
            if constexpr (RES) {
                float b[8];
                load8<AE>(y, e, K, b);
                if (a.post.kind != kNormNone)
                    apply(a.post, row, e, K, pmean, pinv, b);
                if (gate) {
                    float t[8];
                    load8(gate, a.gate_kind, e, K, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        b[j] *= t[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = a.residual_scale * v[j] + a.branch_scale * b[j];
            }
        };
        float mean = 0.0f, inv = 1.0f;
        const bool next = a.next.kind != kNormNone;
        if (next)
            stats(value, K, a.next.kind, a.next.eps, part, mean, inv);
        // Largest |h| as its bit pattern (which orders NaN above infinity).
        float sc = 0.0f, cinv = 0.0f;
        if (next && a.out_kind != kNormOut16) {
            u32 m = 0;
            for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
                float v[8];
                value(e, v);
                apply(a.next, row, e, K, mean, inv, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = max(m, e + j < K ? __float_as_uint(v[j]) & 0x7fffffffu : 0u);
            }
            m = quant_rule::wave_max(m);
            if (threadIdx.x == 0)
                most = 0;
            __syncthreads();
            if ((threadIdx.x & 63) == 0)
                atomicMax(&most, m);
            __syncthreads();
            m = most;
            quant_rule::scale_of(m, kF32, sc, cinv, a.out_kind == kNormOutFp8);
            if (threadIdx.x == 0)
                a.out_scale[row] = sc;
        }
        for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
            float v[8];
            value(e, v);
            if (RES)
                store8<XE>(static_cast<char *>(a.r) + row * a.ldr * XB, e, K, v);
            if (!next)
                continue;
            apply(a.next, row, e, K, mean, inv, v);
            if (a.out_kind == kNormOut16) {
                store8<AE>(static_cast<char *>(a.out) + row * a.ldo * 2, e, K, v);
            } else {
                u32 lo, hi;
                if (a.out_kind == kNormOutFp8) {
                    lo = quant_rule::codes4_fp8(v[0], v[1], v[2], v[3], cinv);
                    hi = quant_rule::codes4_fp8(v[4], v[5], v[6], v[7], cinv);
                } else {
                    lo = quant_rule::codes4_i8(v[0], v[1], v[2], v[3], cinv);
                    hi = quant_rule::codes4_i8(v[4], v[5], v[6], v[7], cinv);
                }
                quant_rule::store_codes<kBF16, false>(static_cast<int8_t *>(a.out) + row * a.ldo, e, (int)K, lo, hi);
            }
        }
        __syncthreads();                               // part and most are free again
    }
}

template <int XE, int AE>
auto looped(bool res)
{
    return res ? norm_rows_looped_kernel<XE, AE, true> : norm_rows_looped_kernel<XE, AE, false>;
}

}  // namespace

hipError_t launch_norm_rows(const NormRowsArgs &a, hipStream_t stream)
{
    const bool res = a.y != nullptr;
    auto fn = a.x_kind == kElemBF16 ? looped<kBF16, kBF16>(res)
            : a.x_kind == kElemF16  ? looped<kF16, kF16>(res)
            : a.act_kind == kElemF16 ? looped<kF32, kF16>(res) : looped<kF32, kBF16>(res);
    const int64_t blocks = a.rows < kMaxBlocksPerLaunch ? a.rows : kMaxBlocksPerLaunch;
    hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w8a8
