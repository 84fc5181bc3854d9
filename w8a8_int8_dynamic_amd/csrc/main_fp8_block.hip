// The main kernel's tiles of the block-scaled e4m3 matmul.
#include "main_fp8_block.hpp"

namespace w8a8 {
namespace {

template <class T>
constexpr BlockTileEntry entry(const char *name)
{
    return BlockTileEntry{name, T::BM, T::BN, T::THREADS, false,
                          {block_mm_kernel<T, kJobDense, kOutBF16>, block_mm_kernel<T, kJobDense, kOutI32>,
                           block_mm_kernel<T, kJobDense, kOutF16>},
                          block_mm_kernel<T, kJobGateUp, kOutI32>, block_mm_kernel<T, kJobDown, kOutF16>};
}

// token rows x channels / wave rows and columns / LDS stages
const BlockTileEntry kMain[] = {
    entry<BlockMain<256, 256, 2, 4, 2>>("256x256/m2n4/l2"),
    entry<BlockMain<128, 256, 2, 4, 3>>("128x256/m2n4/l3"),
};

}  // namespace

int fp8_block_main_count() { return (int)(sizeof(kMain) / sizeof(kMain[0])); }
const BlockTileEntry &fp8_block_main(int i) { return kMain[i]; }

}  // namespace w8a8
