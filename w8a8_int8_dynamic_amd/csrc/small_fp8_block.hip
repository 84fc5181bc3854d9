// Small-M block-scaled e4m3 matmul, for gfx950: a handful of token rows
// against a large weight, of a layer or of each expert that has rows.
//   acc[m,n] = sum over blocks b of 128 of
//              xs[m,b] * ws[n/128,b] * sum over k in b of e4m3(xq[m,k]) * e4m3(wq[n,k])
// The products of a block are one v_mfma_scale_f32_16x16x128_f8f6f4 with unit
// hardware scales from a zero accumulator; its fp32 sums then enter acc by one
// fused multiply-add each with the block's scale, in fp32.
//
// The weight stream bounds it (1 byte per weight), so it is spread over as
// many wavefronts as the shape gives: a workgroup owns 16*FN channels and 16
// token rows, its WK wavefronts take the blocks of K in turn, U of them at a
// time with every load issued before the first product, and the partial sums
// meet in LDS once at the end. The packed fragment is the MFMA's A operand as
// stored, the token rows its B operand, so a lane holds runs of four channels
// of one token.
// Ragged tails: token rows past the last read that one again and fragments
// past the weight its last (never stored); k-chunks past K read the row's last
// chunk, which meets zero weights.
#include <algorithm>

#include "fp8_block_device.hpp"

namespace w8a8 {
namespace {

using namespace fp8_block;

template <int FN_, int WK_, int U_>
struct Small {
    static constexpr int FN = FN_, WK = WK_, U = U_;
    static constexpr int BM = 16, BN = 16 * FN, THREADS = 64 * WK;
};

template <class S, int JOB, int OUT>
__global__ __launch_bounds__(S::THREADS) void block_mm_small_kernel(const BlockMmArgs a)
{
    __shared__ f32x4 part[S::WK - 1][S::FN][64];

    const int lane = threadIdx.x & 63;
    const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, sub = lane >> 4;
    const int tiles_n = (a.frags + S::FN - 1) / S::FN;
    // (an experts' launch holds room for more row tiles than there are)
    const int tiles_m = JOB == kJobDense ? a.tiles_m : a.tiles[a.tiles_m].rows;
    if (JOB != kJobDense && (int)blockIdx.x >= tiles_m * tiles_n)
        return;
    const int t = xcd_remap(blockIdx.x, tiles_m * tiles_n);
    const int tm = t % tiles_m, nb0 = (t / tiles_m) * S::FN;
    const BlockTile tile = JOB == kJobDense ? BlockTile{0, tm * S::BM, min(S::BM, a.M - tm * S::BM)} : a.tiles[tm];
    const uint8_t *wp = a.wp + tile.expert * a.expert_bytes;
    const float *ws = a.ws + tile.expert * a.expert_scales;

    const int row = tile.row0 + min(r16, tile.rows - 1);
    const int64_t src = JOB == kJobGateUp ? a.order[row] / a.top_k : row;
    const uint8_t *xrow = a.xq + src * a.ldq;
    const float *xsrow = a.xs + src * a.lds;
    const v4i *wsrc[S::FN];
    const float *wscale[S::FN];
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
        const int nb = min(nb0 + j, a.frags - 1);
        wsrc[j] = reinterpret_cast<const v4i *>(wp) + (int64_t)nb * a.blocks * 128 + lane;
        wscale[j] = ws + (int64_t)scale_row<JOB>(nb, a.half_scales) * a.blocks;
    }

    f32x4 acc[S::FN] = {};
    for (int b0 = wk; b0 < a.blocks; b0 += S::WK * S::U) {
        v4i w[S::U][S::FN][2], x[S::U][2];
        float xs[S::U], sw[S::U][S::FN];
#pragma unroll
        for (int u = 0; u < S::U; ++u) {
            const int b = min(b0 + u * S::WK, a.blocks - 1);
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
                w[u][j][0] = wsrc[j][(int64_t)b * 128];
                w[u][j][1] = wsrc[j][(int64_t)b * 128 + 64];
                sw[u][j] = wscale[j][b];
            }
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[u][h] = *reinterpret_cast<const v4i *>(xrow + min(b * kBlock + (4 * h + sub) * 16, a.K - 16));
            xs[u] = xsrow[b];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < S::U; ++u) {
            if (b0 + u * S::WK >= a.blocks)
                break;
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
                const f32x4 p = block_product(w[u][j], x[u]);
                const float s = xs[u] * sw[u][j];
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    acc[j][r] = __builtin_fmaf(p[r], s, acc[j][r]);
            }
        }
    }

    if (wk > 0) {
#pragma unroll
        for (int j = 0; j < S::FN; ++j)
            part[wk - 1][j][lane] = acc[j];
    }
    __syncthreads();
    if (wk != 0)
        return;
#pragma unroll
    for (int j = 0; j < S::FN; ++j)
#pragma unroll
        for (int w = 0; w < S::WK - 1; ++w)
            acc[j] += part[w][j][lane];

    // Register r of lane l is channel 4*(l/16) + r of the fragment, token l%16.
    if (r16 >= tile.rows)
        return;
    if constexpr (JOB == kJobGateUp) {
#pragma unroll
        for (int j = 0; j < S::FN; j += 2) {
            const int col = 8 * (nb0 + j) + 4 * sub;
            if (nb0 + j >= a.frags)                       // (the columns are a multiple of 16)
                continue;
            f32x4 h;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                h[r] = silu(acc[j][r]) * acc[j + 1][r];
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + (int64_t)row * a.ldo + col) = h;
        }
        return;
    }
    const int64_t orow = JOB == kJobDown ? a.order[row] : row;
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
        const int n = 16 * (nb0 + j) + 4 * sub;
        if (n >= a.N)
            continue;
        store4<OUT>(a, orow, n, acc[j]);
    }
}

template <class S>
constexpr BlockTileEntry entry(const char *name)
{
    return BlockTileEntry{name, S::BM, S::BN, S::THREADS, true,
                          {block_mm_small_kernel<S, kJobDense, kOutBF16>, block_mm_small_kernel<S, kJobDense, kOutI32>,
                           block_mm_small_kernel<S, kJobDense, kOutF16>},
                          block_mm_small_kernel<S, kJobGateUp, kOutI32>, block_mm_small_kernel<S, kJobDown, kOutI32>};
}

// 16 token rows x 16*FN channels / WK waves along K / U blocks at a time.
const BlockTileEntry kSmall[] = {
    entry<Small<2, 8, 4>>("s16x32/k8/u4"),
};

}  // namespace

int fp8_block_small_count() { return (int)(sizeof(kSmall) / sizeof(kSmall[0])); }
const BlockTileEntry &fp8_block_small(int i) { return kSmall[i]; }

}  // namespace w8a8
