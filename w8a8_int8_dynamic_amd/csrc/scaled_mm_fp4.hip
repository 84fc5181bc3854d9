// The microscaled 4-bit (MX FP4) matmul:
//   acc[m,n] = sum over blocks b of 2^(sx[m,b] + sw[n,b] - 254) *
//              sum over k in b of e2m1(xq[m,k]) * e2m1(wq[n,k])
//   out[m,n] = 16-bit float of acc [+ bias[n]], or acc itself
// on v_mfma_scale_f32_32x32x64_f8f6f4, which applies one e8m0 scale per
// operand row and 32 elements inside the instruction and adds in fp32: 64
// products of e2m1 values are exact in it, so only the sum across blocks of
// different scales rounds.
//
// The main kernel (mm_kernel.hpp) with its FP4 operands: an image byte holds
// two codes, so the loads, LDS images and MFMA count of a product over K
// elements are those of the int8 kernel over K / 2.
#include <algorithm>
#include <cmath>

#include "mm_kernel.hpp"

namespace w8a8 {
namespace {

template <class T>
struct Fp4Entry {
    static constexpr TileEntry entry(const char *name)
    {
        return TileEntry{name, T::BM, T::BN, T::THREADS, false,
                         {scaled_mm_kernel<T, kOutBF16, false, false, true>,
                          scaled_mm_kernel<T, kOutI32, false, false, true>,
                          scaled_mm_kernel<T, kOutF16, false, false, true>},
                         {nullptr, nullptr, nullptr}};
    }
};

const auto kFp4Tiles = main_table<Fp4Entry>(std::make_index_sequence<kNumMainTiles>{});

const TileEntry &fp4_entry(int tile)
{
    return tile < kNumMainTiles ? kFp4Tiles[tile] : fp4_skinny(tile - kNumMainTiles).tile;
}

}  // namespace

int fp4_tile_count() { return kNumMainTiles + fp4_skinny_count(); }
const char *fp4_tile_name(int tile) { return fp4_entry(tile).name; }

int fp4_tile_auto(int64_t M, int64_t N, int64_t K)
{
    if (M <= 16)
        return kNumMainTiles;
    const double cus = 256.0;
    const double kk = (double)round_up(K / 2, 64);
    int best = 0;
    double best_cost = 1e300;
    for (int t = 0; t < kNumMainTiles; ++t) {
        const TileEntry &e = kFp4Tiles[t];
        const int64_t tiles_m = ceil_div(M, e.bm);
        const int64_t tiles = tiles_m * ceil_div(N, e.bn);
        const double rounds = std::ceil((double)tiles / cus);
        const double t_mma = 2.0 * e.bm * e.bn * kk / 16000.0;
        const double t_l2 = (double)(e.bm + e.bn) * kk / 80.0;
        const double t_hbm = (double)e.bn * kk / (double)std::min<int64_t>(tiles_m, 4) / 22.0;
        const double cost = rounds * (std::max({t_mma, t_l2, t_hbm}) + 3000.0);
        if (cost < best_cost * 0.999) {
            best_cost = cost;
            best = t;
        }
    }
    return best;
}

bool fp4_launch_fits(int tile, int64_t M, int64_t N)
{
    const TileEntry &e = fp4_entry(tile);
    return mm_grid_fits(ceil_div(M, e.bm) * ceil_div(N, e.bn), e.threads);
}

hipError_t launch_scaled_mm_fp4(const MmArgs &a, int mode, int tile, hipStream_t stream)
{
    const TileEntry &e = fp4_entry(tile);
    const int64_t tiles = ceil_div(a.M, e.bm) * ceil_div(a.N, e.bn);
    hipLaunchKernelGGL(e.plain[mode], dim3((unsigned)tiles), dim3(e.threads), 0, stream, a);
    return hipGetLastError();
}

hipError_t launch_quant_scaled_mm_fp4(const MmArgs &a, int x_kind, int mode, int tile, hipStream_t stream)
{
    if (tile < kNumMainTiles)
        return hipErrorNotSupported;
    return launch_skinny_quant_fp4(a, x_kind, mode, tile - kNumMainTiles, stream);
}

}  // namespace w8a8
