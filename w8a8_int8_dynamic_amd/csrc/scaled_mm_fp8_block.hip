// The block-scaled e4m3 matmul's tiles (the main kernel's, then the small-M
// ones), their automatic choice and the launches.
#include <cmath>

#include "fp8_block.hpp"

namespace w8a8 {
namespace {

// Automatic choice: the smallest modelled time, a sum of what each tile pays
//   main:    fixed + per round of the CUs (a round, and each block of 128 along K
//            of it) + per MB of weight and of 16-bit output; a round is 256
//            workgroups, 512 of tiles that leave room for two on a CU;
//   small-M: fixed + per workgroup and block + per group of blocks in a wave's
//            chain + per MB of weight, for up to 256 token rows.
// The rates (us) are fitted to the times of every tile on 473 shapes (M 1-8192, N
// 512-12288, K 512-12288, weights from HBM) on MI355X, by
// tests/probes/fp8_block_tile_grid.py; over them the chosen tile takes 1.1 % more
// than the best on average, 28 % at most. A tile without a cost is the experts'.
struct MainCost {
    int per_round;
    double fixed, block, round, weight, out;
};
constexpr MainCost kMainCost[] = {
    {256, 1.412, 1.288, 4.905, 0.0, 0.163},        // 256x256
    {256, 2.98, 0.7625, 1.89, 0.0, 0.2407},        // 128x256
    {256, 3.84, 0.6822, 0.6553, 0.0, 0.2705},      // 128x192
    {256, 3.414, 0.5686, 0.8036, 0.0, 0.3086},     // 128x128
    {512, 3.421, 0.4418, 0.0, 0.008309, 0.4907},   // 64x128
    {512, 3.014, 0.3121, 0.0, 0.01279, 0.6865},    // 64x64
};
struct SmallCost {
    int ahead;                   // blocks of a workgroup's waves at a time
    double fixed, work, chain, weight;
};
constexpr SmallCost kSmallCost[] = {
    {32, 2.755, 5.355e-4, 1.856, 0.02085},         // s16x32/n1k8/u4
    {16, 2.462, 5.044e-4, 1.407, 0.00877},         // s16x32/n1k8/u2nt
    {0, 0, 0, 0, 0},                               // s16x128/n4k2/u4nt
};
static_assert(sizeof(kMainCost) / sizeof(MainCost) == kBlockMainTiles &&
                  sizeof(kSmallCost) / sizeof(SmallCost) == kBlockSmallTiles, "a cost per tile");
constexpr int64_t kSmallRows = 256;

double cost_of(int tile, int64_t M, int64_t N, int64_t K)
{
    const BlockTileEntry &e = fp8_block_tile(tile);
    const double tiles = (double)(ceil_div(M, e.bm) * ceil_div(N, e.bn)), blocks = (double)ceil_div(K, 128);
    const double weight = (double)N * (double)K * 1e-6;
    if (e.small) {
        const SmallCost &c = kSmallCost[tile - kBlockMainTiles];
        if (M > kSmallRows || c.ahead == 0)
            return INFINITY;
        return c.fixed + c.work * tiles * blocks + c.chain * std::ceil(blocks / c.ahead) + c.weight * weight;
    }
    const MainCost &c = kMainCost[tile];
    return c.fixed + std::ceil(tiles / c.per_round) * (c.block * blocks + c.round) + c.weight * weight +
           c.out * (double)M * (double)N * 2e-6;
}

}  // namespace

int fp8_block_tile_count() { return kBlockMainTiles + kBlockSmallTiles; }
const BlockTileEntry &fp8_block_tile(int tile)
{
    return tile < kBlockMainTiles ? fp8_block_main(tile) : fp8_block_small(tile - kBlockMainTiles);
}

int fp8_block_tile_auto(int64_t M, int64_t N, int64_t K)
{
    int best = 0;
    double least = INFINITY;
    for (int t = 0; t < fp8_block_tile_count(); ++t) {
        const double cost = cost_of(t, M, N, K);
        if (cost < least) {
            least = cost;
            best = t;
        }
    }
    return best;
}

hipError_t launch_fp8_block_quant_mm(const BlockMmArgs &a, int x_kind, int mode, int tile, hipStream_t stream)
{
    return tile < kBlockMainTiles ? hipErrorNotSupported
                                  : launch_fp8_block_small_quant(a, x_kind, mode, tile - kBlockMainTiles, stream);
}

hipError_t launch_fp8_block_mm(BlockMmArgs a, int mode, int tile, hipStream_t stream)
{
    const BlockTileEntry &e = fp8_block_tile(tile);
    a.tiles_m = (int)ceil_div(a.M, e.bm);
    const int64_t tiles = (int64_t)a.tiles_m * ceil_div(a.N, e.bn);
    hipLaunchKernelGGL(e.dense[mode], dim3((unsigned)tiles), dim3(e.threads), 0, stream, a);
    return hipGetLastError();
}

}  // namespace w8a8
