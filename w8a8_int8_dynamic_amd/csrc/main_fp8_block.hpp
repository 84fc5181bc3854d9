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
//     registers, the token operands come one tile ahead. A stage is freed and
//     refilled in two parts, each at a barrier of its own: part A, the weights
//     and the first half of the token rows, once every wave has read those (half
//     way through the step); part B, the other rows, at the step's end. Each
//     then has NS - 1/2 steps to land, where refilling whole stages leaves NS -
//     1 (M8192 N4096 K12288, two stages of 64 KB, a step of 2048 matrix core
//     cycles: 367 us so, 354 now).
//   - Token scales go through LDS too, 16 bytes (four blocks) a row at a time;
//     the weight's are one or two numbers per wave and block, held by the lanes
//     of a register for 64 blocks and read from there.
// Experts: the token tiles of a run that is shorter than BM rows are not
// computed (they alternate between the two waves of a SIMD, so that what is
// left out is left out of both). Launches whose rows are cut at 64 sum gated
// products from bf16 values, for the reason in small_fp8_block.hip; that is the
// launch's choice, so that a row's result hangs neither on the rows beside it nor
// on its place among them. Outputs of bf16 are then off 64 bits by 1.67e-3 of their
// norm, of which bf16's own rounding is 1.66e-3, and 1.8-2.8e-3 from e4m3 (ten inputs
// each of 333 tokens, 3 of 24, and of 60 rows an expert). The matrix cores take twice
// the time and every wave converts both operands; what that costs a layer stands with
// the thresholds (experts.hip).
// Measured, M8192 N4096 K12288: 344 us, 2.4 PFLOP/s, the matrix cores busy 66 %
// of the cycles at 1.85 GHz: power bounds it (the same instructions from
// registers alone, on random codes, hold 1.8 GHz). A form whose workgroups stay
// on their CU, load the next tile's first stages under a tile's last steps and
// do not wait for its stores took 354-360 us there, and as long as this one for
// 32768 rows of 64 experts; so a workgroup has one tile.
// Ragged tails: rows past the last read that one again, fragments past the
// weight its last (their results are not stored); k-chunks past K read the
// row's last chunk, which meets zero weights.
#pragma once

#include "fp8_block_device.hpp"
#include "mm_kernel.hpp"

namespace w8a8 {
namespace {

using namespace fp8_block;

constexpr int cmin(int a, int b) { return a < b ? a : b; }

template <int BM_, int BN_, int WM_, int WN_, int NS_>
struct BlockMain {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NS = NS_;
    static constexpr int NW = WM * WN, THREADS = NW * 64;
    static constexpr int TM = BM / 16 / WM, TN = BN / 16 / WN;   // 16 x 16 tiles per wave
    static constexpr int LX = BM / 8 / NW, LWG = BN / 8 / NW;    // 1 KB loads per wave and stage
    static constexpr int LPW = LX + LWG, LA = LX / 2 + LWG;      // ... of the two parts, and of part A
    static constexpr int TOK = BM * 128, STAGE = TOK + BN * 128; // bytes
    static constexpr int SX_UNITS = BM / 64, SX_SLOT = BM * 16;
    static constexpr int SX = NS * STAGE;                        // two slots of token scales
    static constexpr int RING = SX + 2 * SX_SLOT;
    static constexpr int PITCH = BN * 2 + 16;                    // staged 16-bit row
    static constexpr int PITCH_Q = BN / 2 + 16;                  // staged row of codes (gated)
    static constexpr int TOPS = BM * PITCH_Q;                    // then WN block maxima per row
    static constexpr int LDS = cmax(cmax(RING, BM * PITCH), TOPS + WN * BM * 4);
    static constexpr int WAVES = (2 * LDS <= 160 * 1024 ? 2 : 1) * NW / 4;   // on a SIMD
    static_assert(BM % (16 * WM) == 0 && BN % (16 * WN) == 0 && BM % (8 * NW) == 0 && BN % (8 * NW) == 0 &&
                      NS * LPW < 64, "tile");
    static_assert(TM % 2 == 0 && LX % 2 == 0 && BM % 64 == 0 && NW >= SX_UNITS && NW % 2 == 0 && NS <= 4,
                  "token operands alternate; scales in one load, two slots of four blocks");
    static_assert(LDS <= 160 * 1024, "LDS budget");
};

// Where chunk c of row r (of 16) of a token image lies: slot 8r + (c ^
// row_swz(r)). Linear in r's bits, so that the 16 bytes of each 8 or 16 lanes
// that LDS serves together (neighbours, or 0-3, 12-15 and 20-27 with the next
// chunk) fall in different banks whichever they are: rows 0-7, 0-3 with 12-15,
// and even and odd rows, with and without the chunk's low bit, all get
// different values. (With (r ^ r/8) & 7, right for neighbours alone, a third of
// the LDS cycles were conflicts.)
__device__ __forceinline__ int row_swz(int r)
{
    return ((r & 1) * 5) ^ (r & 6) ^ ((r >> 3) * 5);
}

// Workgroup id -> row tile and column tile of an experts' launch: groups of 4 x
// 8 tiles or so, which an XCD's CUs run together (an expert's row tiles then share its
// weights in L2), dealt out to the XCDs in turn: experts are of different sizes,
// and a run of row tiles for each XCD (as layers have it) leaves some with the
// short ones. Launches of fewer tiles than kExpertDeal, a few rounds of the CUs,
// do as layers: there whole groups differ by more (4096 tokens, 1280 tiles: 332 us
// in runs, 314 dealt out; 333 tokens, 270 tiles: 14.8 and 22.5).
__device__ __forceinline__ void expert_tile_of(int pid, int tiles_n, int &tm, int &tn)
{
    const int across = (tiles_n + kExpertGroupN - 1) / kExpertGroupN, columns = (tiles_n + across - 1) / across;
    const int size = kExpertGroupM * columns, local = pid / kXcds, within = local % size;
    const int group = local / size * kXcds + pid % kXcds;
    tm = group / across * kExpertGroupM + within % kExpertGroupM;
    tn = group % across * columns + within / kExpertGroupM;
}

// WIDE: gated products from bf16 values, exact, of a launch whose tiles hold at
// most kCutRows rows.
template <class T, int JOB, int OUT, bool WIDE = false>
__global__ __launch_bounds__(T::THREADS, T::WAVES) void block_mm_kernel(const BlockMmArgs args)
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
        int tm;
        if (tiles_m * tiles_n >= kExpertDeal) {
            expert_tile_of(blockIdx.x, tiles_n, tm, tn);
        } else {
            if ((int)blockIdx.x >= tiles_m * tiles_n)
                return;
            tile_of(xcd_remap(blockIdx.x, tiles_m * tiles_n), tiles_m, tiles_n, tm, tn);
        }
        if (tm >= tiles_m || tn >= tiles_n)
            return;
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
    const int xchunk = ((lane & 7) ^ row_swz((wave & 1) * 8 + (lane >> 3))) * 16;   // (NW is even: so is g - wave)
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
    // Loads N0 .. N1-1 of part A (the first half's token images, then the weights)
    // and of part B (the other token images).
    auto dma_a = [&](int t, int slot, auto n0_c, auto n1_c) __attribute__((always_inline)) {
        char *st = shared + slot * T::STAGE;
        t = min(t, S - 1);
        const int kc = min(t * kBlock + xchunk, a.K - 16);
        static_for<decltype(n1_c)::value - decltype(n0_c)::value>([&](auto U) __attribute__((always_inline)) {
            constexpr int n = decltype(n0_c)::value + decltype(U)::value;
            if constexpr (n < T::LX / 2)
                dma16(xb, xoff[n] + kc, st + (n * T::NW + wave) * 1024);
            else
                dma16(wb, woff[n - T::LX / 2] + t * kFrag, st + T::TOK + ((n - T::LX / 2) * T::NW + wave) * 1024);
        });
    };
    auto dma_b = [&](int t, int slot) __attribute__((always_inline)) {
        char *st = shared + slot * T::STAGE;
        const int kc = min(min(t, S - 1) * kBlock + xchunk, a.K - 16);
#pragma unroll
        for (int i = T::LX / 2; i < T::LX; ++i)
            dma16(xb, xoff[i] + kc, st + (i * T::NW + wave) * 1024);
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
    // Down: the sums of a token's scales, to bound its results by.
    static_assert(JOB != kJobDown || 8 % TN == 0, "a wave's channels share a block");
    float bound[JOB == kJobDown ? TM : 1];
#pragma unroll
    for (int i = 0; i < (JOB == kJobDown ? TM : 1); ++i)
        bound[i] = 0.0f;

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
    static_for<T::NS>([&](auto U) __attribute__((always_inline)) {
        dma_a(decltype(U)::value, decltype(U)::value, std::integral_constant<int, 0>{},
              std::integral_constant<int, T::LA>{});
        dma_b(decltype(U)::value, decltype(U)::value);
    });
    wait_vm_lgkm0<T::LX - T::LX / 2 + (T::NS - 1) * T::LPW>();   // part A of stage 0
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int j = 0; j < TN; ++j)
        read_w(shared, j);
    read_x(shared, 0, 0, x[0], sx[0]);

    // The K loop over the first LIVE token tiles of the wave.
    auto loop = [&](auto live_c) __attribute__((always_inline)) {
        constexpr int LIVE = decltype(live_c)::value;
        static_assert(LIVE % 2 == 0, "products and scales alternate across steps too");
        v8bf wide[WIDE ? TN : 1][4];
        float sc[2][2] = {};                              // scales of the products in p
#pragma unroll
        for (int j = 0; j < TN; ++j)
            p[1][j] = f32x4{};
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
            static_for<LIVE>([&](auto I) __attribute__((always_inline)) {
                constexpr int i = decltype(I)::value;
                constexpr bool LAST = i == LIVE - 1;
                // Half way: every wave has its weights and the first half's
                // tokens in registers, and this stage's part B has landed.
                constexpr int MID = LIVE > TM / 2 ? TM / 2 - 1 : LIVE - 1;
                if constexpr (i == MID) {
                    wait_vm_lgkm0<(T::NS - 1) * T::LPW>();
                    __builtin_amdgcn_s_barrier();
                }
                // Part A's loads are spread over the tiles up to the end.
                constexpr int OVER = LIVE - 1 - MID;
                constexpr int A0 = OVER == 0 ? 0 : cmin(i - MID, OVER) * T::LA / cmax(OVER, 1);
                constexpr int A1 = OVER == 0 ? T::LA : cmin(i + 1 - MID, OVER) * T::LA / cmax(OVER, 1);
                constexpr int LOADS = i < MID ? 0 : A1 - A0;
                if constexpr (LOADS > 0)
                    dma_a(t + T::NS, slot, std::integral_constant<int, A0>{}, std::integral_constant<int, A1>{});
                if constexpr (LAST) {
                    // The end: every token operand of this stage is in
                    // registers, and the next stage's part A has landed.
                    wait_vm_lgkm0<(T::NS - 1) * T::LPW>();
                    __builtin_amdgcn_s_barrier();
                    dma_b(t + T::NS, slot);
                    read_x(stn, t + 1, 0, x[0], sx[0]);
                } else {
                    read_x(st, t, i + 1, x[(i + 1) & 1], sx[(i + 1) & 1]);
                }
                sc[i & 1][0] = sx[i & 1] * sw[0];
                sc[i & 1][1] = TWO ? sx[i & 1] * sw[1] : 0.0f;
                if constexpr (JOB == kJobDown)
                    bound[i] += __builtin_fabsf(sc[i & 1][0]);
                if constexpr (WIDE) {
                    if constexpr (i == 0)
#pragma unroll
                        for (int j = 0; j < TN; ++j)
#pragma unroll
                            for (int g = 0; g < 4; ++g)
                                wide[j][g] = widen(w[j], g);
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const v8bf xw = widen(x[i & 1], g);
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            p[i & 1][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                wide[j][g], xw, g == 0 ? f32x4{} : p[i & 1][j], 0, 0, 0);
                    }
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    if constexpr (!WIDE)
                        p[i & 1][j] = block_product(w[j], x[i & 1]);
                    if constexpr (LAST)
                        read_w(stn, j);
                }
                constexpr int PER = (LOADS + (LAST ? T::LX - T::LX / 2 : 0) + TN - 1) / TN;
                // Behind each MFMA the previous tile's multiply-adds (the first
                // tile's: the last one's of the step before).
                add(std::integral_constant<int, i == 0 ? LIVE - 1 : i - 1>{});
                static_for<WIDE ? 0 : TN>([&](auto) __attribute__((always_inline)) {
                    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);            // MFMA
                    __builtin_amdgcn_sched_group_barrier(0x020, PER, 0);          // VMEM read
                    __builtin_amdgcn_sched_group_barrier(0x100, LAST ? 2 : 1, 0); // DS read
                    __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);            // VALU
                });
                __builtin_amdgcn_sched_barrier(0);
            });
            slot = next;
        }
        add(std::integral_constant<int, LIVE - 1>{});
    };
    if constexpr (JOB == kJobDense) {
        loop(std::integral_constant<int, TM>{});
    } else {
        // Token tiles of this wave that hold rows: tile i is rows 16*(i*WM + wm)
        // on. Computed in whole quarters of the wave's tiles, each with a loop
        // of its own.
        constexpr int Q = TM >= 8 ? TM / 4 : 2;
        static_assert(!WIDE || (JOB == kJobGateUp && kCutRows == 16 * T::WM * Q), "a cut tile's rows are one loop's");
        const int live = ((rows + 15) / 16 - wm + T::WM - 1) / T::WM;
        static_for<WIDE ? 1 : TM / Q>([&](auto I) __attribute__((always_inline)) {
            constexpr int n = decltype(I)::value;
            if (n == 0 ? WIDE || live <= Q : live > n * Q && live <= (n + 1) * Q)
                loop(std::integral_constant<int, (n + 1) * Q>{});
        });
    }
    wait_vm_lgkm0<0>();                                   // (the loads past the last block)
    __builtin_amdgcn_s_barrier();

    // ---- epilogue ----
    // Register r of acc[i][j], lane l: channel 4*(l/16) + r of fragment wn*TN +
    // j, token 16*(i*WM + wm) + l%16 of the tile.
    if constexpr (JOB == kJobGateUp) {
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
    } else if constexpr (OUT == kOutI32) {
        // Raw sums, straight from registers.
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
    } else {
        // 16-bit rows, staged in LDS and written whole, 16 bytes a lane (M4096
        // N4096: 9 us of 8-byte stores from registers, 3.4 so). Down: fp16 under a
        // power of two per row and block of channels, so that a slot's row
        // costs half of fp32's bytes and an eighth of the 2^-8 that bf16 would
        // lose: |acc| <= 448 * 448 * 128 * the sum of its scales < 2^25 times that,
        // brought below 2^15; values below about 2^-28 of that leave fp16's normal
        // range.
        constexpr bool F16 = OUT == kOutF16;
        // Down: the slots of the wave's rows, then of the thread's pieces, are read
        // ahead of the stores, which the compiler would else keep them behind (M
        // 32768 rows of 64 experts, K 1024, N 4096: 234 us behind them, 214 now).
        int slot_of[JOB == kJobDown ? TM : 1];
        if constexpr (JOB == kJobDown) {
#pragma unroll
            for (int i = 0; i < TM; ++i)
                slot_of[i] = a.order[row0 + min(16 * (i * T::WM + wm) + r16, rows - 1)];
        }
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int m = 16 * (i * T::WM + wm) + r16;
            float down = 1.0f;
            if constexpr (JOB == kJobDown) {
                // bound < 2^(e - 10), or else |acc| < 2^128 (and what is not finite stays so)
                const int e = min((int)((__float_as_uint(bound[i]) >> 23) & 255u) - 126 + 10, 113);
                down = __uint_as_float((u32)(127 - e) << 23);
                if (sub == 0 && (wn * TN) % 8 == 0 && m < rows && wf < a.frags)
                    a.out_scale[(int64_t)slot_of[i] * a.ld_out_scale + (wf >> 3)] =
                        __uint_as_float((u32)(127 + e) << 23);
            }
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                f32x4 v = acc[i][j];
                if constexpr (JOB == kJobDown) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        v[r] *= down;
                } else if (a.bias) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const unsigned b = a.bias[min(16 * (wf + j) + 4 * sub + r, a.N - 1)];
                        v[r] += F16 ? quant_rule::f16_to_float(b) : __uint_as_float(b << 16);
                    }
                }
                *reinterpret_cast<uint2 *>(shared + m * T::PITCH + (wn * TN + j) * 32 + sub * 8) =
                    make_uint2(pack2<F16>(v[0], v[1]), pack2<F16>(v[2], v[3]));
            }
        }
        constexpr int P16 = T::BN / 8, RPP = T::THREADS / P16;   // pieces per row, rows per pass
        const int c = threadIdx.x % P16, first = threadIdx.x / P16, n = f0 * 16 + c * 8;
        constexpr int PASSES = (T::BM + RPP - 1) / RPP;
        int row_of[JOB == kJobDown ? PASSES : 1];
        if constexpr (JOB == kJobDown) {
#pragma unroll
            for (int q = 0; q < PASSES; ++q)
                row_of[q] = a.order[row0 + min(first + q * RPP, rows - 1)];
        }
        __syncthreads();
        uint16_t *out = static_cast<uint16_t *>(a.out) + n;
        if (n >= a.N)
            return;
        const bool whole = a.vec16 && n + 8 <= a.N;
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int m = first + q * RPP;
            if (m >= rows)
                break;
            const int64_t orow = JOB == kJobDown ? row_of[q] : row0 + m;
            uint16_t *o = out + orow * a.ldo;
            const v4u v = *reinterpret_cast<const v4u *>(shared + m * T::PITCH + c * 16);
            if (whole) {
                __builtin_nontemporal_store(v, reinterpret_cast<v4u *>(o));
            } else {
#pragma unroll
                for (int r = 0; r < 8; ++r)
                    if (n + r < a.N)
                        o[r] = (uint16_t)(v[r >> 1] >> (16 * (r & 1)));
            }
        }
    }
}

}  // namespace
}  // namespace w8a8
