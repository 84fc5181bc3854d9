// Declarations shared by the translation units of the block-scaled 8-bit layer
// and the mixture of experts.
#pragma once

#include "internal.hpp"

namespace w8a8 {

// Packed fragments (16 channels) and scale rows (128 channels) of a weight of
// N rows; gated: N = 2I rows, each half with fragments and scale rows of its own.
inline int64_t fp8_block_frags(int64_t N, bool gated) { return gated ? 2 * ceil_div(N / 2, 16) : ceil_div(N, 16); }
inline int64_t fp8_block_scale_rows(int64_t N, bool gated)
{
    return gated ? 2 * ceil_div(N / 2, 128) : ceil_div(N, 128);
}

// ---- rows and weights (quant_fp8_block.hip) ----
// K is a multiple of 16; rows of x and out 16-byte aligned, codes 8-byte.
hipError_t launch_quant_fp8_block(const void *x, int kind, int64_t rows, int64_t K, int64_t ldx, uint8_t *q,
                                  int64_t ldq, float *s, int64_t lds, hipStream_t stream);
hipError_t launch_dequant_fp8_block(const uint8_t *q, int64_t ldq, const float *s, int64_t lds, int64_t rows,
                                    int64_t K, int kind, void *out, int64_t ldo, hipStream_t stream);
// `experts` weights [N, ldw], one behind the other. pack: codes w into the
// packed layout; otherwise back from it.
hipError_t launch_repack_fp8_block(uint8_t *w, int64_t ldw, int64_t experts, int64_t N, int64_t K, bool gated,
                                   void *packed, bool pack, hipStream_t stream);
hipError_t launch_quant_prepack_fp8_block(const void *w, bool w_f32, int64_t ldw, int64_t experts, int64_t N,
                                          int64_t K, bool gated, void *packed, float *scale, hipStream_t stream);

// ---- the product (small_fp8_block.hip) ----
// What a launch computes: a layer's product; the gated products silu(gate) * up
// of each expert's rows (rows of tokens by order / top_k, out in sorted rows:
// fp32 from the small-M kernel, codes and scales from the main kernel); or the
// down products of sorted rows, to the rows that order names (fp32 from the
// small-M kernel, fp16 under a scale per row and 128 channels from the main
// kernel).
constexpr int kJobDense = 0, kJobGateUp = 1, kJobDown = 2;

// A run of rows of one expert.
struct BlockTile {
    int expert, row0, rows;
};

struct BlockMmArgs {
    const uint8_t *xq;
    const float *xs;
    const uint8_t *wp;
    const float *ws;
    const uint16_t *bias;
    void *out;
    int64_t ldq, lds, ldo;
    int M, N, K;
    int blocks;          // ceil(K / 128)
    int frags;           // packed fragments along N
    int half_scales;     // gated: scale rows of one half
    int vec_store;       // 1 when out rows allow stores of 4 consecutive elements
    int vec16;           // 1 when out rows start on 16-byte boundaries
    int tiles_m;         // row tiles of the launch, at most
    float *out_scale;    // experts, main kernel: the scales [rows, ld_out_scale] of out
    int64_t ld_out_scale;
    // Experts:
    const BlockTile *tiles;   // then, at [tiles_m], their number as rows
    const int *order;    // slot (token * top_k + choice) of each sorted row
    int top_k, experts;
    const int *ids;      // direct: the slots' experts, without a plan
    const float *weights;
    // Rows to quantize in the same launch (direct down: fp32 inner rows).
    const void *x;
    int64_t ldx;
    int64_t expert_bytes, expert_scales;   // from one expert's weight and scales to the next's
};

// Tiles of an experts' launch that go to one XCD together: 4 row tiles by about 8
// column tiles (`across` even groups of columns); and the workgroups that the
// main kernel's launch over tiles_m x tiles_n tiles takes.
constexpr int kExpertGroupM = 4, kExpertGroupN = 8, kExpertDeal = 768;
inline int64_t expert_grid(int64_t tiles_m, int64_t tiles_n)
{
    const int64_t across = ceil_div(tiles_n, kExpertGroupN);
    if (tiles_m * tiles_n < kExpertDeal)
        return tiles_m * tiles_n;
    return round_up(ceil_div(tiles_m, kExpertGroupM) * across, kXcds) * kExpertGroupM * ceil_div(tiles_n, across);
}

typedef void (*BlockMmKernel)(const BlockMmArgs);
struct BlockTileEntry {
    const char *name;
    int bm, bn, threads;
    bool small;
    BlockMmKernel dense[kOutKinds], gate_up, down, gate_up_cut;
};
// Rows of a tile of gate_up_cut's launches, at most.
constexpr int kCutRows = 64;
constexpr int kBlockMainTiles = 6, kBlockSmallTiles = 3;
const BlockTileEntry &fp8_block_main(int i);
const BlockTileEntry &fp8_block_small(int i);
// The quant of a.x (element kind x_kind) and small-M tile i in one launch;
// hipErrorNotSupported (nothing launched) where a workgroup's rows are too many
// to be quantized by each.
hipError_t launch_fp8_block_small_quant(BlockMmArgs a, int x_kind, int mode, int i, hipStream_t stream);
// Experts of a few tokens in two launches: the gated products of every slot
// (up.M of them, rows of x quantized on the way, out fp32) and the down
// products with the sum over slots. Whether rows of those lengths fit.
bool fp8_block_direct_fits(int top_k, int64_t K, int64_t inner);
hipError_t launch_fp8_block_direct(BlockMmArgs up, BlockMmArgs down, int x_kind, int tokens, hipStream_t stream);

int fp8_block_tile_count();
const BlockTileEntry &fp8_block_tile(int tile);
int fp8_block_tile_auto(int64_t M, int64_t N, int64_t K);
// The quant of a.x and the matmul in one launch, as launch_fp8_block_small_quant.
hipError_t launch_fp8_block_quant_mm(const BlockMmArgs &a, int x_kind, int mode, int tile, hipStream_t stream);
hipError_t launch_fp8_block_mm(BlockMmArgs a, int mode, int tile, hipStream_t stream);

}  // namespace w8a8
