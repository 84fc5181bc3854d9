// The microscaled 4-bit (MX FP4) matmul:
//   acc[m,n] = sum over blocks b of 2^(sx[m,b] + sw[n,b] - 254) *
//              sum over k in b of e2m1(xq[m,k]) * e2m1(wq[n,k])
//   out[m,n] = 16-bit float of acc [+ bias[n]], or acc itself
// on v_mfma_scale_f32_32x32x64_f8f6f4, which applies one e8m0 scale per
// operand row and 32 elements inside the instruction and adds in fp32: 64
// products of e2m1 values are exact in it, so only the sum across blocks of
// different scales rounds.
//
// The simplest form: one wavefront per 32 x 32 output tile, four of them
// (2 x 2) per workgroup, every operand read straight from memory.
#include "mm_kernel.hpp"

namespace w8a8 {
namespace {

template <int OUT>
__global__ __launch_bounds__(256) void fp4_mm_kernel(const MmArgs a)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int tiles_m = (a.M + 63) / 64;
    const int m0 = ((int)blockIdx.x % tiles_m) * 64 + (wave & 1) * 32;
    const int n0 = ((int)blockIdx.x / tiles_m) * 64 + (wave >> 1) * 32;
    const int m = min(m0 + (lane & 31), a.M - 1);
    const int nb = min(n0 / 16 + ((lane >> 4) & 1), a.nblocks - 1);
    const int8_t *xrow = a.xq + (int64_t)m * a.ldq;
    const uint8_t *srow = a.sx + (int64_t)m * a.lds;
    const int chunks = (a.kblocks + 3) / 4;
    v16f acc = {};
    for (int kb = 0; kb < a.kblocks; ++kb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            // Lane l takes block 4*kb + 2*h + l/32 of token l%32 and channel
            // l%32; past the row's last block the last one is read again and
            // meets zero weights.
            const int c = 2 * h + (lane >> 5), b = min(4 * kb + c, a.blocks - 1);
            const v4i x = *reinterpret_cast<const v4i *>(xrow + (int64_t)b * 16);
            const v4i w = *reinterpret_cast<const v4i *>(a.wp + ((int64_t)nb * a.kblocks + kb) * 1024 +
                                                         (16 * c + (lane & 15)) * 16);
            const int sx = srow[b];
            const int sw = a.sw[((int64_t)nb * chunks + kb / 4) * 256 + (lane & 15) * 16 + (kb & 3) * 4 + c];
            const v8i xx = {x[0], x[1], x[2], x[3], 0, 0, 0, 0}, ww = {w[0], w[1], w[2], w[3], 0, 0, 0, 0};
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(ww, xx, acc, 4, 4, 0, sw, 0, sx);
        }
    const int mo = m0 + (lane & 31);
    if (mo >= a.M)
        return;
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = n0 + 8 * q + 4 * (lane >> 5) + r;
            if (n >= a.N)
                continue;
            float v = acc[4 * q + r];
            if (OUT == kOutI32) {
                reinterpret_cast<float *>(a.out)[(int64_t)mo * a.ldo + n] = v;
                continue;
            }
            if (a.bias)
                v += OUT == kOutF16 ? quant_rule::f16_to_float(a.bias[n]) : __uint_as_float((unsigned)a.bias[n] << 16);
            const float t[4] = {v, v, v, v};
            reinterpret_cast<uint16_t *>(a.out)[(int64_t)mo * a.ldo + n] = (uint16_t)pack4<OUT == kOutF16>(t)[0];
        }
}

}  // namespace

int fp4_tile_count() { return 1; }
const char *fp4_tile_name(int) { return "64x64"; }
int fp4_tile_auto(int64_t, int64_t, int64_t) { return 0; }
bool fp4_launch_fits(int, int64_t M, int64_t N) { return mm_grid_fits(ceil_div(M, 64) * ceil_div(N, 64), 256); }

hipError_t launch_scaled_mm_fp4(const MmArgs &a, int mode, int, hipStream_t stream)
{
    auto fn = mode == kOutBF16 ? fp4_mm_kernel<kOutBF16> : mode == kOutF16 ? fp4_mm_kernel<kOutF16>
                                                                           : fp4_mm_kernel<kOutI32>;
    hipLaunchKernelGGL(fn, dim3((unsigned)(ceil_div(a.M, 64) * ceil_div(a.N, 64))), dim3(256), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w8a8
