// The block-scaled e4m3 matmul's tiles and their automatic choice.
#include "fp8_block.hpp"

namespace w8a8 {

int fp8_block_tile_count() { return fp8_block_main_count() + fp8_block_small_count(); }
const BlockTileEntry &fp8_block_tile(int tile)
{
    const int n = fp8_block_main_count();
    return tile < n ? fp8_block_main(tile) : fp8_block_small(tile - n);
}

int fp8_block_tile_auto(int64_t M, int64_t N, int64_t K)
{
    return M <= 64 ? (N * K > (16 << 20) && M <= 16 ? 8 : 7) : M <= 512 ? 1 : 0;
}

hipError_t launch_fp8_block_quant_mm(const BlockMmArgs &a, int x_kind, int mode, int tile, hipStream_t stream)
{
    const int n = fp8_block_main_count();
    return tile < n ? hipErrorNotSupported : launch_fp8_block_small_quant(a, x_kind, mode, tile - n, stream);
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
