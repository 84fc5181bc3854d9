// The block-scaled e4m3 matmul's main kernel, for gfx950: layers of many rows
// and experts with many rows each.
//   acc[m,n] = sum over blocks b of 128 of
//              xs[m,b] * ws[n/128,b] * sum over k in b of e4m3(xq[m,k]) * e4m3(wq[n,k])
//
// Design (a dense contraction: the e4m3 MFMA roofline bounds it, with a
// multiply-add on the vector units beside every 128 products).
//   - v_mfma_scale_f32_16x16x128_f8f6f4 takes a whole block at once: from a
//     zero accumulator to a register quad, which enters the fp32 accumulators
//     by one fused multiply-add each. That product of scales is one number per
//     lane (a lane holds channels of one token), so a 16 x 16 tile costs four
//     multiply-adds, 16 cycles of the vector unit beside 32 of the matrix core.
//     They run TN MFMAs behind, beside the next tiles' MFMAs, so that they
//     neither wait for a result nor leave the matrix core idle.
//   - Eight wavefronts, two per SIMD: one's matrix instructions fill the other's
//     waits. Accumulators that vector instructions update have to be VGPRs,
//     which a wave of its own on a SIMD has no more of than a wave of two.
//     Measured on MI355X in registers alone, random codes: 3.4-3.7 PFLOP/s so,
//     1.5-1.8 with the multiply-adds right behind their MFMA, 3.7-3.9 without any.
//   - Both operands go through LDS in stages of one block, filled straight from
//     memory (buffer_load ... lds). A token image is 8 rows of 128 bytes, lane
//     8r+j loading chunk j ^ swz(r) of row r: whole lines from memory, and the
//     operand reads (row l%16, chunks l/16 and 4 + l/16) meet all banks. Weights
//     come as the packed fragments are.
//   - A wave owns TM x TN tiles: the TN weight operands of a block stay in
//     registers, the token operands come one tile ahead. Once every wave holds
//     its last token operand of a stage, one barrier frees the stage for the
//     block after next and makes the next one visible.
//   - Token scales go through LDS too, 16 bytes (four blocks) a row at a time;
//     the weight's are one or two numbers per wave and block, held by the lanes
//     of a register for 64 blocks and read from there.
// Experts: the token tiles of a run that is shorter than BM rows are not
// computed (they alternate between the two waves of a SIMD, so that what is
// left out is left out of both).
// Ragged tails: rows past the last read that one again, fragments past the
// weight its last (their results are not stored); k-chunks past K read the
// row's last chunk, which meets zero weights.
#pragma once

#include "fp8_block_device.hpp"
#include "mm_kernel.hpp"

namespace w8a8 {
namespace {

using namespace fp8_block;

template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct BlockMain {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
    static constexpr int NW = WM * WN, THREADS = NW * 64;
    static constexpr int TM = BM / 16 / WM, TN = BN / 16 / WN;   // 16 x 16 tiles per wave
    static constexpr int LX = BM / 8 / NW, LWG = BN / 8 / NW;    // 1 KB loads per wave and stage
    static constexpr int LPW = LX + LWG;
    static constexpr int TOK = BM * 128, STAGE = TOK + BN * 128; // bytes
    static constexpr int SX_UNITS = BM / 64, SX_SLOT = BM * 16;
    static constexpr int SX = NS * STAGE;                        // two slots of token scales
    static constexpr int RING = SX + 2 * SX_SLOT;
    static constexpr int PITCH = BN * 2 + 16;                    // staged 16-bit row
    static constexpr int PITCH_Q = BN / 2 + 16;                  // staged row of codes (gated)
    static constexpr int TOPS = BM * PITCH_Q;                    // then WN block maxima per row
    static constexpr int LDS = cmax(cmax(RING, BM * PITCH), TOPS + WN * BM * 4);
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0, "tile");
    static_assert(TM % 2 == 0 && BM % 64 == 0 && NW >= SX_UNITS, "token operands alternate; scales in one load");
    static_assert(LDS <= 160 * 1024, "LDS budget");
};

__device__ __forceinline__ int row_swz(int r) { return (r & 7) ^ ((r >> 3) & 1); }

template <class T, int JOB, int OUT>
__global__ __launch_bounds__(T::THREADS) void block_mm_kernel(const BlockMmArgs args)
{
    __shared__ uint4 lds[T::LDS / 16];
    char *const shared = reinterpret_cast<char *>(lds);
    constexpr int TM = T::TM, TN = T::TN;

    BlockMmArgs a = args;
    a.K = pinned(args.K);
    a.blocks = pinned(args.blocks);

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wn = wave % T::WN, wm = wave / T::WN;
    const int r16 = lane & 15, sub = lane >> 4;

    const int tiles_n = (a.frags * 16 + T::BN - 1) / T::BN;
    BlockTile tile;
    int tn;
    if constexpr (JOB == kJobDense) {
        int tm;
        tile_of(xcd_remap(blockIdx.x, a.tiles_m * tiles_n), a.tiles_m, tiles_n, tm, tn);
        tile = BlockTile{0, tm * T::BM, min(T::BM, a.M - tm * T::BM)};
    } else {
        // (the launch holds room for more row tiles than there are)
        const int tiles_m = a.tiles[a.tiles_m].rows;
        if ((int)blockIdx.x >= tiles_m * tiles_n)
            return;
        int tm;
        tile_of(xcd_remap(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
        tile = a.tiles[tm];
    }
    const int expert = __builtin_amdgcn_readfirstlane(tile.expert), row0 = __builtin_amdgcn_readfirstlane(tile.row0);
    const int rows = __builtin_amdgcn_readfirstlane(tile.rows);
    const int f0 = tn * (T::BN / 16);                     // first fragment of the tile
    const int S = a.blocks;

    // Sources. Tokens: image g = i*NW + wave, lane 8r+j row 8g + r, chunk j ^ swz.
    const uint8_t *xb = a.xq;
    const float *sxb = a.xs;
    if constexpr (JOB != kJobGateUp) {
        xb += (int64_t)row0 * a.ldq;
        sxb += (int64_t)row0 * a.lds;
    }
    auto token_row = [&](int r) __attribute__((always_inline)) {
        r = min(r, rows - 1);
        return JOB == kJobGateUp ? a.order[row0 + r] / a.top_k : r;
    };
    int xoff[T::LX];
#pragma unroll
    for (int i = 0; i < T::LX; ++i)
        xoff[i] = token_row((i * T::NW + wave) * 8 + (lane >> 3)) * (int)a.ldq;
    const int xchunk = ((lane & 7) ^ (lane >> 3) ^ (wave & 1)) * 16;   // (NW is even: image g's parity is the wave's)
    const int sunit = min(wave, T::SX_UNITS - 1);
    const int soff = token_row(sunit * 64 + lane) * (int)a.lds * 4;
    const char *wb = reinterpret_cast<const char *>(a.wp) + expert * a.expert_bytes + (int64_t)f0 * S * kFrag;
    int woff[T::LWG];
#pragma unroll
    for (int i = 0; i < T::LWG; ++i) {
        const int g = i * T::NW + wave;
        woff[i] = (min(f0 + g / 2, a.frags - 1) - f0) * S * kFrag + (g & 1) * 1024 + lane * 16;
    }
    xb = pinned_ptr(xb);
    wb = pinned_ptr(wb);
    sxb = pinned_ptr(sxb);

    // Weight scales: lanes hold 64 blocks of the (one or two) rows that this
    // wave's fragments fall in.
    constexpr bool TWO = JOB == kJobGateUp || TN % 4 != 0;
    const int wf = f0 + wn * TN;
    const float *ws = a.ws + expert * a.expert_scales;
    const int last_frag = a.frags - 1;
    const float *wsrow[2] = {ws + (int64_t)scale_row<JOB>(min(wf, last_frag), a.half_scales) * S,
                             ws + (int64_t)scale_row<JOB>(min(JOB == kJobGateUp ? wf + 1 : wf + TN - 1, last_frag),
                                                          a.half_scales) * S};
    bool second[TN];                                      // fragment j's scale is the second row's
#pragma unroll
    for (int j = 0; j < TN; ++j)
        second[j] = JOB == kJobGateUp ? (j & 1) != 0 : TWO && (wf + j) >> 3 != wf >> 3;
    float wsv[2];
    auto load_ws = [&](int b) __attribute__((always_inline)) {
        wsv[0] = wsrow[0][min(b + lane, S - 1)];
        wsv[1] = TWO ? wsrow[1][min(b + lane, S - 1)] : 0.0f;
    };

    // Block t into a stage (past the last block that one again, into a stage that
    // nothing reads any more); blocks t .. t+3's token scales, t a multiple of 4.
    auto dma_sx = [&](int t) __attribute__((always_inline)) {
        dma16(sxb, soff + min(t, (S - 1) & ~3) * 4, shared + T::SX + ((t >> 2) & 1) * T::SX_SLOT + sunit * 1024);
    };
    auto dma = [&](int t, int slot) __attribute__((always_inline)) {
        char *st = shared + slot * T::STAGE;
        t = min(t, S - 1);
        const int kc = min(t * kBlock + xchunk, a.K - 16);
#pragma unroll
        for (int i = 0; i < T::LX; ++i)
            dma16(xb, xoff[i] + kc, st + (i * T::NW + wave) * 1024);
#pragma unroll
        for (int i = 0; i < T::LWG; ++i)
            dma16(wb, woff[i] + t * kFrag, st + T::TOK + (i * T::NW + wave) * 1024);
    };

    f32x4 acc[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
            acc[i][j] = f32x4{};
    v4i w[TN][2], x[2][2];
    float sx[2];
    f32x4 p[2][TN];

    // Operands from LDS: fragment wn*TN + j, units l and 64 + l; token tile i's
    // row l%16, chunks l/16 and 4 + l/16, and its scale.
    auto read_w = [&](const char *st, int j) __attribute__((always_inline)) {
        const v4i *f = reinterpret_cast<const v4i *>(st + T::TOK) + (wn * TN + j) * 128 + lane;
        w[j][0] = f[0];
        w[j][1] = f[64];
    };
    const int xs_lane = wm * 16 + r16;
    const int xslot = xs_lane * 128, xc0 = (sub ^ row_swz(r16)) * 16, xc1 = ((4 + sub) ^ row_swz(r16)) * 16;
    auto read_x = [&](const char *st, int t, int i, v4i (&v)[2], float &s) __attribute__((always_inline)) {
        const char *r = st + xslot + i * (T::WM * 2048);
        v[0] = *reinterpret_cast<const v4i *>(r + xc0);
        v[1] = *reinterpret_cast<const v4i *>(r + xc1);
        s = *reinterpret_cast<const float *>(shared + T::SX + ((t >> 2) & 1) * T::SX_SLOT + (t & 3) * 4 +
                                             (xs_lane + i * T::WM * 16) * 16);
    };

    load_ws(0);
    dma_sx(0);
    dma(0, 0);
    if constexpr (T::NS == 3)
        dma(1, 1);
    wait_vm_lgkm0<0>();
    __builtin_amdgcn_s_barrier();
    dma(T::NS - 1, T::NS - 1);
#pragma unroll
    for (int j = 0; j < TN; ++j)
        read_w(shared, j);
    read_x(shared, 0, 0, x[0], sx[0]);

    // The K loop over the first LIVE token tiles of the wave.
    auto loop = [&](auto live_c) __attribute__((always_inline)) {
        constexpr int LIVE = decltype(live_c)::value;
        int slot = 0;
        for (int t = 0; t < S; ++t) {
            // What not every step does comes first: a branch further down would
            // part the multiply-adds from their MFMAs.
            if (((t + T::NS) & 3) == 0)
                dma_sx(t + T::NS);
            if ((t & 63) == 0 && t > 0) {
                load_ws(t);
                wait_vm_lgkm0<0>();                       // (here, not at each use in the loop)
            }
            const int next = slot + 1 == T::NS ? 0 : slot + 1;
            const char *st = shared + slot * T::STAGE, *stn = shared + next * T::STAGE;
            float sw[2];
            sw[0] = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv[0]), t & 63));
            sw[1] = TWO ? __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(wsv[1]), t & 63)) : 0.0f;
            float sc[2][2];
            // acc += p * scale for tile i's products
            auto add = [&](auto I) __attribute__((always_inline)) {
                constexpr int i = decltype(I)::value;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    const float s = TWO && second[j] ? sc[i & 1][1] : sc[i & 1][0];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        acc[i][j][r] = __builtin_fmaf(p[i & 1][j][r], s, acc[i][j][r]);
                }
            };
            static_for<LIVE>([&](auto I) __attribute__((always_inline)) {
                constexpr int i = decltype(I)::value;
                constexpr bool LAST = i == LIVE - 1;
                if constexpr (LAST) {
                    // Every token operand of this stage is in registers, and
                    // the next stage has landed.
                    wait_vm_lgkm0<T::NS == 3 ? T::LPW : 0>();
                    __builtin_amdgcn_s_barrier();
                    dma(t + T::NS, slot);
                    read_x(stn, t + 1, 0, x[0], sx[0]);
                } else {
                    read_x(st, t, i + 1, x[(i + 1) & 1], sx[(i + 1) & 1]);
                }
                sc[i & 1][0] = sx[i & 1] * sw[0];
                sc[i & 1][1] = TWO ? sx[i & 1] * sw[1] : 0.0f;
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    p[i & 1][j] = block_product(w[j], x[i & 1]);
                    if constexpr (LAST)
                        read_w(stn, j);
                }
                if constexpr (i > 0)
                    add(std::integral_constant<int, i - 1>{});
                // Behind each MFMA the previous tile's multiply-adds.
                static_for<TN>([&](auto) __attribute__((always_inline)) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);            // MFMA
                    __builtin_amdgcn_sched_group_barrier(0x100, LAST ? 2 : 1, 0); // DS read
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);            // VALU
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            add(std::integral_constant<int, LIVE - 1>{});
            slot = next;
        }
    };
    if constexpr (JOB == kJobDense) {
        loop(std::integral_constant<int, TM>{});
    } else {
        // Token tiles of this wave that hold rows: tile i is rows 16*(i*WM + wm)
        // on. Computed in whole quarters of the wave's tiles, each with a loop
        // of its own.
        constexpr int Q = TM >= 8 ? TM / 4 : 2;
        const int live = ((rows + 15) / 16 - wm + T::WM - 1) / T::WM;
        static_for<TM / Q>([&](auto I) __attribute__((always_inline)) {
            constexpr int n = decltype(I)::value;
            if (n == 0 ? live <= Q : live > n * Q && live <= (n + 1) * Q)
                loop(std::integral_constant<int, (n + 1) * Q>{});
        });
    }
    wait_vm_lgkm0<0>();                                   // (the loads past the last block)
    __builtin_amdgcn_s_barrier();

    // ---- epilogue ----
    // Register r of acc[i][j], lane l: channel 4*(l/16) + r of fragment wn*TN +
    // j, token 16*(i*WM + wm) + l%16 of the tile.
    if constexpr (JOB == kJobDown) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = 16 * (i * T::WM + wm) + r16;
            if (m >= rows)
                continue;
            const int64_t orow = a.order[row0 + m];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = 16 * (wf + j) + 4 * sub;
                if (n < a.N)
                    store4<OUT>(a, orow, n, acc[i][j]);
            }
        }
    } else if constexpr (JOB == kJobGateUp) {
        // The tile's BN / 2 = 128 columns are one block of the down product's
        // rows: silu(gate) * up, the block's maximum over the WN waves that
        // share a row, and codes and scale from here, so that the inner rows
        // are written once, in the form that they are read in.
        static_assert(T::BN == 256 && TN % 2 == 0, "one block of inner columns per tile");
        u32 *tops = reinterpret_cast<u32 *>(shared + T::TOPS);
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            u32 top = 0;
#pragma unroll
            for (int j = 0; j < TN; j += 2)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    // (fragments past the weight repeat its last, an up fragment: no part of a row)
                    const float h = wf + j < a.frags ? silu(acc[i][j][r]) * acc[i][j + 1][r] : 0.0f;
                    acc[i][j][r] = h;
                    top = max(top, __float_as_uint(h) & 0x7fffffffu);
                }
            top = max(top, (u32)__shfl_xor((int)top, 16, 64));
            top = max(top, (u32)__shfl_xor((int)top, 32, 64));
            if (sub == 0)
                tops[wn * T::BM + 16 * (i * T::WM + wm) + r16] = top;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = 16 * (i * T::WM + wm) + r16;
            u32 top = 0;
#pragma unroll
            for (int v = 0; v < T::WN; ++v)
                top = max(top, tops[v * T::BM + m]);
            float s, f;
            scale_of(top, s, f);
            if (wn == 0 && sub == 0 && m < rows)
                a.out_scale[(int64_t)(row0 + m) * a.ld_out_scale + tn] = s;
#pragma unroll
            for (int j = 0; j < TN; j += 2)
                *reinterpret_cast<u32 *>(shared + m * T::PITCH_Q + (wn * TN + j) * 8 + sub * 4) =
                    quant_rule::codes4_fp8(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], f);
        }
        __syncthreads();
        // Whole rows of 128 bytes, 8 lanes each (the columns are a multiple of 16).
        const int piece = (threadIdx.x & 7) * 16;
        uint8_t *out = static_cast<uint8_t *>(a.out) + (int64_t)row0 * a.ldo + tn * kBlock + piece;
        if (tn * kBlock + piece < a.frags * 8)
            for (int m = threadIdx.x >> 3; m < rows; m += T::THREADS / 8)
                *reinterpret_cast<uint4 *>(out + (int64_t)m * a.ldo) =
                    *reinterpret_cast<const uint4 *>(shared + m * T::PITCH_Q + piece);
    } else {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = 16 * (i * T::WM + wm) + r16;
            if (m >= rows)
                continue;
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const int n = 16 * (wf + j) + 4 * sub;
                if (n < a.N)
                    store4<OUT>(a, (int64_t)row0 + m, n, acc[i][j]);
            }
        }
    }
}

}  // namespace
}  // namespace w8a8
