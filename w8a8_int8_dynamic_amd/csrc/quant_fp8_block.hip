// Block-scaled e4m3 quantization, its inverse and the weight repack, on gfx950.
// The rule and the packed layout are fp8_block_rule.hpp's.
//
// quant_fp8_block_kernel (HBM-bound: 2 bytes read and 1 + 1/32 written per
// 16-bit element): 16 neighbouring lanes share a block of 128, 8 elements
// each, so a wavefront's loads are contiguous (16 bytes a lane), four lane
// exchanges give the block's maximum, and its code words are contiguous too.
// A workgroup takes U x 256 such units of one row, or several whole rows where
// a row is shorter than that. Rows whose last block is part full keep their
// units in whole blocks (idle lanes count as zeros). M8192 K12288 bf16: 50 us,
// 6.0 TB/s; the inverse 44 us, 6.9 (part of the codes are still in the caches).
#include <algorithm>

#include "quant_fp8_block.hpp"

namespace w8a8 {
namespace {

using namespace fp8_block;

template <int E, int U>
__global__ __launch_bounds__(256) void quant_fp8_block_kernel(const char *__restrict__ x, int64_t rows, int units,
                                                              int padded, int64_t ldx, uint8_t *__restrict__ q,
                                                              int64_t ldq, float *__restrict__ s, int64_t lds,
                                                              int segs, int rpb)
{
    quant_block_rows<E, U>(blockIdx.x, threadIdx.x, x, rows, units, padded, ldx, q, ldq, s, lds, segs, rpb);
}

// 8 codes a thread back to their values, rounded to the output's type.
template <int E, int U>
__global__ __launch_bounds__(256) void dequant_fp8_block_kernel(const uint8_t *__restrict__ q, int64_t ldq,
                                                                const float *__restrict__ s, int64_t lds,
                                                                int64_t rows, int units, int padded,
                                                                char *__restrict__ out, int64_t ldo, int segs, int rpb)
{
    const Place p = place_of(blockIdx.x, threadIdx.x, rows, padded, segs, rpb, 256 * U);
    constexpr int BYTES = quant_rule::Elem<E>::BYTES;
    if (!p.valid)
        return;
    uint2 w[U];
    float sc[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = min(p.unit0 + i * 256, units - 1);
        w[i] = *reinterpret_cast<const uint2 *>(q + p.row * ldq + (int64_t)u * 8);
        sc[i] = s[p.row * lds + (u >> 4)];
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = p.unit0 + i * 256;
        if (u >= units)
            break;
        const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].x, false) * sc[i];
        const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].x, true) * sc[i];
        const f32x2 c = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].y, false) * sc[i];
        const f32x2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)w[i].y, true) * sc[i];
        char *dst = out + (p.row * ldo + (int64_t)u * 8) * BYTES;
        if constexpr (E == kF32) {
            *reinterpret_cast<f32x4 *>(dst) = f32x4{a[0], a[1], b[0], b[1]};
            *reinterpret_cast<f32x4 *>(dst + 16) = f32x4{c[0], c[1], d[0], d[1]};
        } else {
            constexpr bool H = E == kF16;
            __builtin_nontemporal_store(
                quant_rule::v4u{pack2<H>(a[0], a[1]), pack2<H>(b[0], b[1]), pack2<H>(c[0], c[1]), pack2<H>(d[0], d[1])},
                reinterpret_cast<quant_rule::v4u *>(dst));
        }
    }
}

// Weight row of channel r of fragment nb: gated weights hold `half` gate rows,
// then the up rows.
__device__ __forceinline__ int64_t weight_row(int64_t nb, int r, int half, int64_t N)
{
    if (half == 0)
        return nb * 16 + r;
    const int64_t col = (nb >> 1) * 16 + r;
    return col < half ? (nb & 1) * half + col : N;
}

// One 16-byte unit of a fragment per thread, from codes made before (PACK) or
// back to them. `experts` weights of N rows follow each other.
template <bool PACK>
__global__ __launch_bounds__(256) void repack_fp8_block_kernel(uint8_t *__restrict__ w, int64_t ldw, int64_t N, int K,
                                                               int half, int blocks, int64_t frags,
                                                               uint4 *__restrict__ packed, int64_t units, int64_t u0)
{
    const int64_t u = u0 + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= units)
        return;
    const int r = (int)(u & 15), c = (int)((u >> 4) & 7);
    const int64_t frag = u >> 7;
    const int kb = (int)(frag % blocks);
    const int64_t row = frag / blocks, e = row / frags, nb = row - e * frags;
    const int64_t n = weight_row(nb, r, half, N);
    const int k = kb * kBlock + c * 16;
    const bool in = n < N && k < K;                       // K is a multiple of 16
    uint8_t *p = w + (e * N + n) * ldw + k;
    if constexpr (PACK) {
        u32 o[4] = {0, 0, 0, 0};
        if (in)
            for (int j = 0; j < 16; ++j)
                o[j >> 2] |= (u32)p[j] << (8 * (j & 3));
        packed[u] = make_uint4(o[0], o[1], o[2], o[3]);
    } else if (in) {
        const uint4 v = packed[u];
        const u32 o[4] = {v.x, v.y, v.z, v.w};
        for (int j = 0; j < 16; ++j)
            p[j] = (uint8_t)(o[j >> 2] >> (8 * (j & 3)));
    }
}

// Online quantization: one workgroup per 128 x 128 block (of the gate or up
// half, where there are halves). Thread t holds rows t/8 + 32*i, elements
// 16*(t%8) .. +15 of them.
template <int E>
__global__ __launch_bounds__(256) void quant_prepack_fp8_block_kernel(const char *__restrict__ w, int64_t ldw,
                                                                      int64_t N, int K, int half, int blocks,
                                                                      int64_t srows, int64_t frags,
                                                                      uint4 *__restrict__ packed,
                                                                      float *__restrict__ scale, int64_t b0)
{
    constexpr int B = quant_rule::Elem<E>::BYTES, W = B;  // 16-byte words per 16 elements
    __shared__ u32 wave_top[4];
    const int64_t b = b0 + blockIdx.x;
    const int kb = (int)(b % blocks);
    const int64_t row = b / blocks, e = row / srows, sr = row - e * srows;
    const int64_t per_half = half ? srows / 2 : srows;
    const int which = half ? (int)(sr / per_half) : 0;
    const int64_t col0 = (sr - which * per_half) * kBlock;   // first channel of the block in its half
    const int64_t end = half ? half : N;
    const int c = (int)(threadIdx.x & 7), k = kb * kBlock + c * 16;
    uint4 v[4][W];
    u32 top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t col = col0 + (threadIdx.x >> 3) + 32 * i;
#pragma unroll
        for (int j = 0; j < W; ++j)
            v[i][j] = make_uint4(0, 0, 0, 0);
        if (col < end && k < K) {
            const uint4 *src = reinterpret_cast<const uint4 *>(w + ((e * N + which * half + col) * ldw + k) * B);
#pragma unroll
            for (int j = 0; j < W; ++j)
                v[i][j] = src[j];
        }
        top = max(top, max(absmax8<E>(v[i][0], v[i][1]), absmax8<E>(v[i][W / 2], v[i][W - 1])));
    }
    top = quant_rule::wave_max(top);
    if ((threadIdx.x & 63) == 0)
        wave_top[threadIdx.x >> 6] = top;
    __syncthreads();
    top = max(max(wave_top[0], wave_top[1]), max(wave_top[2], wave_top[3]));
    float s, inv;
    scale_of(top, s, inv);
    if (threadIdx.x == 0)
        scale[row * blocks + kb] = s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t col = col0 + (threadIdx.x >> 3) + 32 * i;
        // (columns past the end up to a whole fragment are packed as zeros)
        if (col >= (end + 15) / 16 * 16)
            continue;
        const uint2 lo = codes8<E>(v[i][0], v[i][E == kF32 ? 1 : 0], inv);
        const uint2 hi = codes8<E>(v[i][W / 2], v[i][W - 1], inv);
        const int64_t nb = half ? (col >> 4) * 2 + which : col >> 4;
        packed[((e * frags + nb) * blocks + kb) * 128 + c * 16 + (col & 15)] = make_uint4(lo.x, lo.y, hi.x, hi.y);
    }
}

template <int E>
auto quant_pick(int u)
{
    return u == 1 ? quant_fp8_block_kernel<E, 1> : u == 2 ? quant_fp8_block_kernel<E, 2>
         : u == 3 ? quant_fp8_block_kernel<E, 3> : quant_fp8_block_kernel<E, 4>;
}
template <int E>
auto dequant_pick(int u)
{
    return u == 1 ? dequant_fp8_block_kernel<E, 1> : u == 2 ? dequant_fp8_block_kernel<E, 2>
         : u == 3 ? dequant_fp8_block_kernel<E, 3> : dequant_fp8_block_kernel<E, 4>;
}

// launch(first row, rows, cut) over slices of rows whose workgroups fit one
// launch.
template <class F>
hipError_t in_row_slices(int64_t rows, int padded, F &&launch)
{
    const Cut whole = cut_of(rows, padded);
    const int64_t step = std::max<int64_t>(1, kMaxBlocksPerLaunch / whole.segs) * whole.rpb;
    for (int64_t r0 = 0; r0 < rows; r0 += step) {
        Cut c = whole;
        const int64_t n = std::min(rows - r0, step);
        c.blocks = whole.rpb == 1 ? n * c.segs : ceil_div(n, c.rpb);
        launch(r0, n, c);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_quant_fp8_block(const void *x, int kind, int64_t rows, int64_t K, int64_t ldx, uint8_t *q,
                                  int64_t ldq, float *s, int64_t lds, hipStream_t stream)
{
    const int units = (int)(K / 8), padded = (int)round_up(units, 16), bytes = kind == kElemF32 ? 4 : 2;
    return in_row_slices(rows, padded, [&](int64_t r0, int64_t n, const Cut &c) {
        auto fn = kind == kElemF32 ? quant_pick<kF32>(c.u) : kind == kElemF16 ? quant_pick<kF16>(c.u)
                                                                              : quant_pick<kBF16>(c.u);
        hipLaunchKernelGGL(fn, dim3((unsigned)c.blocks), dim3(256), 0, stream,
                           static_cast<const char *>(x) + r0 * ldx * bytes, n, units, padded, ldx, q + r0 * ldq, ldq,
                           s + r0 * lds, lds, c.segs, c.rpb);
    });
}

hipError_t launch_dequant_fp8_block(const uint8_t *q, int64_t ldq, const float *s, int64_t lds, int64_t rows,
                                    int64_t K, int kind, void *out, int64_t ldo, hipStream_t stream)
{
    const int units = (int)(K / 8), padded = (int)round_up(units, 16), bytes = kind == kElemF32 ? 4 : 2;
    return in_row_slices(rows, padded, [&](int64_t r0, int64_t n, const Cut &c) {
        auto fn = kind == kElemF32 ? dequant_pick<kF32>(c.u) : kind == kElemF16 ? dequant_pick<kF16>(c.u)
                                                                                : dequant_pick<kBF16>(c.u);
        hipLaunchKernelGGL(fn, dim3((unsigned)c.blocks), dim3(256), 0, stream, q + r0 * ldq, ldq, s + r0 * lds, lds,
                           n, units, padded, static_cast<char *>(out) + r0 * ldo * bytes, ldo, c.segs, c.rpb);
    });
}

hipError_t launch_repack_fp8_block(uint8_t *w, int64_t ldw, int64_t experts, int64_t N, int64_t K, bool gated,
                                   void *packed, bool pack, hipStream_t stream)
{
    const int blocks = (int)ceil_div(K, kBlock);
    const int half = gated ? (int)(N / 2) : 0;
    const int64_t frags = fp8_block_frags(N, gated), units = experts * frags * blocks * 128;
    auto fn = pack ? repack_fp8_block_kernel<true> : repack_fp8_block_kernel<false>;
    for (int64_t u0 = 0; u0 < units; u0 += kMaxBlocksPerLaunch * 256) {
        const int64_t n = std::min(ceil_div(units - u0, 256), kMaxBlocksPerLaunch);
        hipLaunchKernelGGL(fn, dim3((unsigned)n), dim3(256), 0, stream, w, ldw, N, (int)K, half, blocks, frags,
                           static_cast<uint4 *>(packed), units, u0);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

hipError_t launch_quant_prepack_fp8_block(const void *w, bool w_f32, int64_t ldw, int64_t experts, int64_t N,
                                          int64_t K, bool gated, void *packed, float *scale, hipStream_t stream)
{
    const int blocks = (int)ceil_div(K, kBlock);
    const int half = gated ? (int)(N / 2) : 0;
    const int64_t srows = fp8_block_scale_rows(N, gated), total = experts * srows * blocks;
    auto fn = w_f32 ? quant_prepack_fp8_block_kernel<kF32> : quant_prepack_fp8_block_kernel<kBF16>;
    for (int64_t b0 = 0; b0 < total; b0 += kMaxBlocksPerLaunch) {
        hipLaunchKernelGGL(fn, dim3((unsigned)std::min(total - b0, kMaxBlocksPerLaunch)), dim3(256), 0, stream,
                           static_cast<const char *>(w), ldw, N, (int)K, half, blocks, srows,
                           fp8_block_frags(N, gated), static_cast<uint4 *>(packed), scale, b0);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace w8a8
