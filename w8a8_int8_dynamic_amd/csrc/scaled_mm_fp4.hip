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
// elements are those of the int8 kernel over K / 2, and the MFMAs take half
// as long over them.
//
// What bounds it, measured on MI355X. M512 N12288 K4096 (128x192 tiles, one
// round of 256 workgroups): 20.5 us, 2.5 PFLOP/s; of it the loop 12.9 us, at
// 653-730 cycles per k-block where the MFMAs are 384: the 21.5 KB that a CU
// reads for one, at about 31 bytes a cycle. The int8 loop over the same operand
// bytes takes 10 to 20 % less: the rest is the loads of the block scales.
// Then 2.8 us of first loads and 2.2 of stores. M8192 N4096 K12288
// (256x256, two rounds): 188-204 us, 4.0-4.4 PFLOP/s; 1310-1377 cycles per
// k-block where the MFMAs are 1024, at 1.45-1.8 GHz, the clock that power
// leaves for random codes (the MFMAs alone, from registers, make 5.9-6.4
// PFLOP/s of those, 9.0 of zeros).
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

// Automatic choice: the smallest modelled time, a sum of what each tile pays
//   main:    fixed + per round of 256 workgroups (a round, and each k-block of
//            it) + per MB of weight and of 16-bit output;
//   small-M: fixed + per workgroup and k-block + per chunk of 512 elements in
//            a wave's chain, for up to 256 token rows.
// The rates (us) are fitted to the times of every tile on 643 shapes (M 8-8192,
// N 512-12288, K 512-12288, weights from HBM) on MI355X, by
// tests/probes/fp4_tile_grid.py; over them the chosen tile takes 1.3 % more than
// the best on average, 23 % at most.
struct MainCost {
    double fixed, kblock, round, weight, out;
};
constexpr MainCost kMainCost[] = {
    {3.89, 0.1045, 0.0, 0.0588, 0.2476},   {4.14, 0.1504, 0.217, 0.0578, 0.2575}, {3.04, 0.1691, 1.312, 0.0218, 0.4217},
    {3.07, 0.2347, 2.652, 0.0308, 0.2244}, {5.22, 0.2994, 2.777, 0.0080, 0.2614}, {1.93, 0.3999, 4.040, 0.0910, 0.1613},
    {4.32, 0.5250, 6.028, 0.0053, 0.1106}, {0.40, 0.5753, 8.836, 0.1214, 0.1250}};
static_assert(sizeof(kMainCost) / sizeof(kMainCost[0]) == kNumMainTiles, "a cost for every main tile");
struct SmallCost {
    double fixed, work, chain;
};
constexpr SmallCost kSmallCost[] = {{3.29, 1.773e-4, 0.692}, {3.55, 2.482e-4, 1.164}};
constexpr int64_t kSmallRows = 256;

int fp4_tile_auto(int64_t M, int64_t N, int64_t K)
{
    const double kblocks = (double)ceil_div(K, 128);
    int best = 0;
    double best_cost = 1e300;
    for (int t = 0; t < fp4_tile_count(); ++t) {
        const TileEntry &e = fp4_entry(t);
        if (e.skinny && M > kSmallRows)
            continue;
        const double tiles = (double)(ceil_div(M, e.bm) * ceil_div(N, e.bn));
        double cost;
        if (e.skinny) {
            const SmallCost &c = kSmallCost[t - kNumMainTiles];
            cost = c.fixed + c.work * tiles * kblocks + c.chain * std::ceil((double)ceil_div(K, 512) / 8.0);
        } else {
            const MainCost &c = kMainCost[t];
            cost = c.fixed + std::ceil(tiles / 256.0) * (c.kblock * kblocks + c.round) +
                   c.weight * (double)N * (double)K * 17.0 / 32e6 + c.out * (double)M * (double)N * 2e-6;
        }
        if (cost < best_cost) {
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
