// The main kernel's tiles of the block-scaled e4m3 matmul.
#include "main_fp8_block.hpp"

namespace w8a8 {
namespace {

// The experts' kernels, for the tiles that they run on (whose inner columns are one
// block).
template <class T>
constexpr BlockMmKernel gate_up()
{
    if constexpr (T::BN == 256)
        return block_mm_kernel<T, kJobGateUp, kOutI32>;
    else
        return nullptr;
}

// The same of tiles of at most kCutRows rows, exact.
template <class T>
constexpr BlockMmKernel gate_up_cut()
{
    if constexpr (T::BN == 256 && T::BM == 128)
        return block_mm_kernel<T, kJobGateUp, kOutI32, true>;
    else
        return nullptr;
}

template <class T>
constexpr BlockMmKernel down()
{
    if constexpr (T::BN == 256)
        return block_mm_kernel<T, kJobDown, kOutF16>;
    else
        return nullptr;
}

template <class T>
constexpr BlockTileEntry entry(const char *name)
{
    return BlockTileEntry{name, T::BM, T::BN, T::THREADS, false,
                          {block_mm_kernel<T, kJobDense, kOutBF16>, block_mm_kernel<T, kJobDense, kOutI32>,
                           block_mm_kernel<T, kJobDense, kOutF16>},
                          gate_up<T>(), down<T>(), gate_up_cut<T>()};
}

// token rows x channels / wave rows and columns / LDS stages
const BlockTileEntry kMain[] = {
    entry<BlockMain<256, 256, 2, 4, 2>>("256x256/m2n4/l2"),
    entry<BlockMain<128, 256, 2, 4, 3>>("128x256/m2n4/l3"),
    entry<BlockMain<128, 192, 2, 4, 3>>("128x192/m2n4/l3"),
    entry<BlockMain<128, 128, 2, 4, 4>>("128x128/m2n4/l4"),
    entry<BlockMain<64, 128, 1, 4, 3>>("64x128/m1n4/l3"),
    entry<BlockMain<64, 64, 2, 2, 4>>("64x64/m2n2/l4"),
};
static_assert(sizeof(kMain) / sizeof(kMain[0]) == kBlockMainTiles, "tiles");

}  // namespace

const BlockTileEntry &fp8_block_main(int i) { return kMain[i]; }

}  // namespace w8a8
