// Small-M block-scaled e4m3 matmul, for gfx950: a handful of token rows
// against a large weight, of a layer or of each expert that has rows, with the
// quantization of the rows in the same launch where they are few.
//   acc[m,n] = sum over blocks b of 128 of
//              xs[m,b] * ws[n/128,b] * sum over k in b of e4m3(xq[m,k]) * e4m3(wq[n,k])
// The products of a block are one v_mfma_scale_f32_16x16x128_f8f6f4 with unit
// hardware scales from a zero accumulator; its fp32 sums then enter acc by one
// fused multiply-add each with the block's scale, in fp32.
//
// The weight stream bounds it (1 byte per weight), so it is spread over as
// many wavefronts as the shape gives, each with U blocks of weights in flight
// before its first product: a workgroup owns 16 token rows and 16*FN*WN
// channels, its WK wavefronts along K take the blocks in turn, and the partial
// sums meet in LDS once at the end. The packed fragment is the MFMA's A operand
// as stored, the token rows its B operand, so a lane holds runs of four
// channels of one token.
//   - WK = 8 for a layer, whose column tiles alone are few; WK = 2 beside WN = 4 for
//     experts, whose tiles are many: a wave with a block or two waits for those
//     and then for its neighbours (48 tokens, 8 of 64 experts each, N 4096, K
//     1024: 90 us with WK = 8, 46 so; whole layer, K 4096, inner 1024, 4 of 64: 4
//     tokens 51.6 and 48.9, 256 234 and 218).
//   - NT: weights that one row tile reads pass the caches by (M1 N12288 K4096:
//     11.7 us without, 10.3 so, 4.9 TB/s; below 16 MB, which the caches may
//     hold, 4.6 without and 5.0 so). Experts' tiles always do: an expert with several
//     row tiles has them side by side on one XCD, which read its weights together
//     (64 experts, K 4096, inner 1024, 160 tokens of 4: 166 us spread, 95 all to four).
//     Experts, 48 tokens to 8 of 64, K 4096, inner 1024: gated products 84 us, 6.4
//     TB/s, down 44 us, 6.1.
//   - Gated products are summed from bf16 values, without the e4m3 instruction's
//     error: an inner element near the border of two codes falls to either side by
//     it, a step of 2^-3. The matrix cores wait for the weights anyway (48 tokens
//     as above 144 us from e4m3, 146 so; outputs 1.6-2.8e-3 of their norm from the
//     elementwise form's, and 4e-4 so). The main kernel does so
//     in launches of few rows an expert, and keeps e4m3 in the others (experts.hip).
//   - QK: the rows come as floats. Every workgroup quantizes them into LDS
//     while its first weights are on their way, 8 elements a thread at a time
//     (they are few and sit in L2); the workgroups of the first channels write
//     codes and scales out. Up to kSlots such steps (as in the 4-bit layer's).
// Ragged tails: token rows past the last read that one again and fragments
// past the weight its last (never stored); k-chunks past K read the row's last
// chunk, which meets zero weights.
#include <algorithm>

#include "fp8_block_device.hpp"

namespace w8a8 {
namespace {

using namespace fp8_block;

template <int FN_, int WN_, int WK_, int U_, bool NT_>
struct Small {
    static constexpr int FN = FN_, WN = WN_, WK = WK_, U = U_;
    static constexpr bool NT = NT_;
    static constexpr int BM = 16, BF = FN * WN, BN = 16 * BF, THREADS = 64 * WN * WK;
};

constexpr int cmin(int a, int b) { return a < b ? a : b; }
constexpr int kCodes = -1;       // QK: codes and scales made before
constexpr int kSlots = 4;        // units of 8 elements that a thread quantizes, at most

// Bytes of LDS behind one quantized row: the codes of whole blocks, then the scales.
__host__ __device__ constexpr int row_bytes(int blocks) { return blocks * 128 + (blocks * 4 + 15) / 16 * 16; }

// `rows` rows of x (row r at source(r)) quantized by the workgroup into LDS, row
// r at r * row_bytes, and with `writer` to xq and xs. The rows' units of 8
// elements, in whole blocks, are one list, dealt out THREADS at a time; a
// block's 16 are neighbouring lanes'.
template <int THREADS, int E, class Source>
__device__ __forceinline__ void quantize_rows(const BlockMmArgs &a, Source &&source, int rows, bool writer, int row0,
                                              char *tok)
{
    constexpr int XB = quant_rule::Elem<E>::BYTES;
    const int per_row = a.blocks * 16, total = rows * per_row;
    uint4 lo[kSlots], hi[kSlots];
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        const int at = s * THREADS + (int)threadIdx.x, r = at / per_row, u = at - r * per_row;
        lo[s] = hi[s] = make_uint4(0, 0, 0, 0);
        if (at < total && u * 8 < a.K) {
            const uint4 *src = reinterpret_cast<const uint4 *>(source(r) + (int64_t)u * 8 * XB);
            lo[s] = src[0];
            if (E == kF32)
                hi[s] = src[1];
        }
    }
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
        if (s * THREADS >= total)
            break;
        const int at = s * THREADS + (int)threadIdx.x, r = at / per_row, u = at - r * per_row;
        float sc, f;
        scale_of(row16_max(absmax8<E>(lo[s], hi[s])), sc, f);
        const uint2 c = codes8<E>(lo[s], hi[s], f);
        if (at >= total)
            continue;
        char *row = tok + r * row_bytes(a.blocks);
        *reinterpret_cast<uint2 *>(row + u * 8) = c;
        if ((u & 15) == 0)
            *reinterpret_cast<float *>(row + a.blocks * 128 + (u >> 4) * 4) = sc;
        if (writer && u * 8 < a.K) {
            *reinterpret_cast<uint2 *>(const_cast<uint8_t *>(a.xq) + (int64_t)(row0 + r) * a.ldq + u * 8) = c;
            if ((u & 15) == 0)
                const_cast<float *>(a.xs)[(int64_t)(row0 + r) * a.lds + (u >> 4)] = sc;
        }
    }
}

// (four waves to a SIMD where the registers' limit would else leave three)
template <class S, int JOB, int OUT, int QK>
__global__ __launch_bounds__(S::THREADS, JOB == kJobGateUp || S::WN == 4 ? 4 : 1) void
block_mm_small_kernel(const BlockMmArgs a)
{
    __shared__ f32x4 part[S::WN][S::WK - 1][S::FN][64];
    extern __shared__ __attribute__((aligned(16))) char tok[];   // QK: the quantized rows

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wk = wave % S::WK, wn = wave / S::WK;
    const int r16 = lane & 15, sub = lane >> 4;
    const int tiles_n = (a.frags + S::BF - 1) / S::BF;
    BlockTile tile;
    int tn;
    if constexpr (JOB == kJobGateUp && QK != kCodes) {
        // A slot is a tile of its own: its expert by its id.
        const int t = xcd_remap(blockIdx.x, a.M * tiles_n), slot = t % a.M;
        tn = t / a.M;
        tile = BlockTile{a.ids[slot], slot, 1};
        if (tile.expert < 0 || tile.expert >= a.experts)
            return;
    } else {
        // (an experts' launch holds room for more row tiles than there are)
        const int tiles_m = JOB == kJobDense ? a.tiles_m : a.tiles[a.tiles_m].rows;
        if (JOB != kJobDense && (int)blockIdx.x >= tiles_m * tiles_n)
            return;
        const int t = xcd_remap(blockIdx.x, tiles_m * tiles_n);
        const int tm = t % tiles_m;
        tn = t / tiles_m;
        tile = JOB == kJobDense ? BlockTile{0, tm * S::BM, min(S::BM, a.M - tm * S::BM)} : a.tiles[tm];
    }
    tile = BlockTile{__builtin_amdgcn_readfirstlane(tile.expert), __builtin_amdgcn_readfirstlane(tile.row0),
                     __builtin_amdgcn_readfirstlane(tile.rows)};
    const int nb0 = tn * S::BF + wn * S::FN;
    const uint8_t *wp = a.wp + tile.expert * a.expert_bytes;
    const float *ws = a.ws + tile.expert * a.expert_scales;

    const int r = min(r16, tile.rows - 1);
    const char *xrow, *xsrow;                              // this lane's row of codes and scales
    if constexpr (QK == kCodes) {
        const int64_t src = JOB == kJobGateUp ? a.order[tile.row0 + r] / a.top_k : tile.row0 + r;
        xrow = reinterpret_cast<const char *>(a.xq) + src * a.ldq;
        xsrow = reinterpret_cast<const char *>(a.xs + src * a.lds);
    } else {
        xrow = tok + r * row_bytes(a.blocks);
        xsrow = xrow + a.blocks * 128;
    }
    // (LDS rows hold whole blocks)
    const int last_chunk = QK == kCodes ? a.K - 16 : a.blocks * kBlock - 16;
    const v4i *wsrc[S::FN];
    const float *wscale[S::FN];
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
        const int nb = min(nb0 + j, a.frags - 1);
        wsrc[j] = reinterpret_cast<const v4i *>(wp) + (int64_t)nb * a.blocks * 128 + lane;
        wscale[j] = ws + (int64_t)scale_row<JOB>(nb, a.half_scales) * a.blocks;
    }

    f32x4 acc[S::FN] = {};
    v4i w[S::U][S::FN][2];
    float sw[S::U][S::FN];
    // (blocks past the last read that one; their products are skipped)
    auto weights = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < S::U; ++u) {
            const int b = min(b0 + u * S::WK, a.blocks - 1);
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const v4i *p = wsrc[j] + (int64_t)b * 128 + h * 64;
                    w[u][j][h] = S::NT ? __builtin_nontemporal_load(p) : *p;
                }
                sw[u][j] = wscale[j][b];
            }
        }
    };
    // Token operands: of all U blocks at a time, or where bf16 operands need the
    // registers of two.
    constexpr int AT = JOB == kJobGateUp ? cmin(S::U, 2) : S::U;
    auto products = [&](int b0) __attribute__((always_inline)) {
        v4i x[AT][2];
        float xs[AT];
        auto tokens = [&](int u) __attribute__((always_inline)) {
            const int b = min(b0 + u * S::WK, a.blocks - 1);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                x[u % AT][h] = *reinterpret_cast<const v4i *>(xrow + min(b * kBlock + (4 * h + sub) * 16, last_chunk));
            xs[u % AT] = *reinterpret_cast<const float *>(xsrow + b * 4);
        };
#pragma unroll
        for (int u = 0; u < AT; ++u)
            tokens(u);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < S::U; ++u) {
            if (b0 + u * S::WK >= a.blocks)
                break;
            f32x4 p[S::FN];
            if constexpr (JOB == kJobGateUp)
                wide_products(w[u], x[u % AT], p);
#pragma unroll
            for (int j = 0; j < S::FN; ++j) {
                if constexpr (JOB != kJobGateUp)
                    p[j] = block_product(w[u][j], x[u]);
                const float s = xs[u % AT] * sw[u][j];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[j][k] = __builtin_fmaf(p[j][k], s, acc[j][k]);
            }
            if constexpr (JOB == kJobGateUp) {
                __builtin_amdgcn_sched_barrier(0);        // (one block's bf16 operands at a time)
                if (u + AT < S::U)
                    tokens(u + AT);
            }
        }
    };
    int b0 = wk;
    if constexpr (QK != kCodes) {
        // (of every wave, clamped into the weight: no wave skips the barrier)
        weights(b0);
        quantize_rows<S::THREADS, QK>(
            a,
            [&](int row) __attribute__((always_inline)) {
                const int64_t src = JOB == kJobGateUp ? (tile.row0 + row) / a.top_k : tile.row0 + row;
                return static_cast<const char *>(a.x) + src * a.ldx * quant_rule::Elem<QK>::BYTES;
            },
            tile.rows, JOB == kJobDense && tn == 0, tile.row0, tok);
        __syncthreads();
        products(b0);
        b0 += S::WK * S::U;
    }
    for (; b0 < a.blocks; b0 += S::WK * S::U) {
        weights(b0);
        products(b0);
    }

    // The partial sums along K meet in LDS: unit u of the fragments (a gate and
    // its up fragment are one) is finished by wave u % WK of those that share
    // the channels, which adds all their sums in the waves' order.
    constexpr int STEP = JOB == kJobGateUp ? 2 : 1, UNITS = S::FN / STEP;
    auto slot = [](int w, int unit) { return w - (w > unit % S::WK); };
#pragma unroll
    for (int q = 0; q < S::FN; ++q)
        if (wk != q / STEP % S::WK)
            part[wn][slot(wk, q / STEP)][q][lane] = acc[q];
    __syncthreads();
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
        if (wk != u % S::WK)
            continue;
        f32x4 v[STEP];
#pragma unroll
        for (int e = 0; e < STEP; ++e) {
            const int q = u * STEP + e;
#pragma unroll
            for (int o = 0; o < S::WK; ++o) {
                const f32x4 one = o == u % S::WK ? acc[q] : part[wn][slot(o, u)][q][lane];
                v[e] = o == 0 ? one : v[e] + one;
            }
        }
        // Register k of lane l is channel 4*(l/16) + k of the fragment, token l%16.
        const int nb = nb0 + u * STEP;
        if (r16 >= tile.rows || nb >= a.frags)
            continue;
        if constexpr (JOB == kJobGateUp) {
            f32x4 h;
#pragma unroll
            for (int k = 0; k < 4; ++k)
                h[k] = silu(v[0][k]) * v[1][k];
            *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + (int64_t)(tile.row0 + r16) * a.ldo + 8 * nb +
                                       4 * sub) = h;
        } else {
            const int64_t orow = JOB == kJobDown ? a.order[tile.row0 + r16] : tile.row0 + r16;
            if (16 * nb + 4 * sub < a.N)
                store4<OUT>(a, orow, 16 * nb + 4 * sub, v[0]);
        }
    }
}

// The down products of a token's slots and their weighted sum in one launch,
// for a few tokens: a workgroup takes 16 channels of a token's output, its
// waves the (slot, part of K) pairs in turn, so that the sum over slots is the
// one over waves. Its slots' inner rows (fp32) are quantized first, as above.
constexpr int kDirectWaves = 8, kDirectAhead = 8;
template <int E>
__global__ __launch_bounds__(64 * kDirectWaves) void down_direct_kernel(const BlockMmArgs a)
{
    __shared__ f32x4 part[kDirectWaves - 1][64];
    extern __shared__ __attribute__((aligned(16))) char tok[];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sub = lane >> 4;
    const int t = xcd_remap(blockIdx.x, a.M * a.frags);
    const int token = t % a.M, nb = t / a.M, slot0 = token * a.top_k;
    // Pairs: each slot's blocks in `parts` runs.
    const int parts = max(1, kDirectWaves / a.top_k), run = (a.blocks + parts - 1) / parts;
    const int pairs = a.top_k * parts;

    v4i w[kDirectAhead][2];
    float sw[kDirectAhead], weight = 0.0f;
    int first = 0, end = 0;
    const v4i *wsrc = nullptr;
    const float *wscale = nullptr;
    // The pair's weights (none for a slot without an expert).
    auto begin = [&](int pair) __attribute__((always_inline)) {
        const int j = pair / parts, id = pair < pairs ? a.ids[slot0 + j] : -1;
        first = pair % parts * run;
        end = id >= 0 && id < a.experts ? min(first + run, a.blocks) : 0;
        if (first >= end)
            return;
        weight = a.weights[slot0 + j];
        wsrc = reinterpret_cast<const v4i *>(a.wp + id * a.expert_bytes) + (int64_t)nb * a.blocks * 128 + lane;
        wscale = a.ws + id * a.expert_scales + (int64_t)(nb >> 3) * a.blocks;
    };
    auto weights = [&](int b0) __attribute__((always_inline)) {
#pragma unroll
        for (int u = 0; u < kDirectAhead; ++u) {
            const int b = min(b0 + u, end - 1);
            w[u][0] = __builtin_nontemporal_load(wsrc + (int64_t)b * 128);
            w[u][1] = __builtin_nontemporal_load(wsrc + (int64_t)b * 128 + 64);
            sw[u] = wscale[b];
        }
    };
    begin(wave);
    if (first < end)
        weights(first);
    quantize_rows<64 * kDirectWaves, kF32>(
        a,
        [&](int row) __attribute__((always_inline)) {
            return static_cast<const char *>(a.x) + (int64_t)(slot0 + row) * a.ldx * 4;
        },
        a.top_k, false, 0, tok);
    __syncthreads();
    f32x4 total = {};
    for (int pair = wave; pair < pairs; pair += kDirectWaves) {
        if (pair != wave)
            begin(pair);
        if (first >= end)
            continue;
        const char *row = tok + pair / parts * row_bytes(a.blocks);
        f32x4 acc = {};
        for (int b0 = first; b0 < end; b0 += kDirectAhead) {
            if (pair != wave || b0 != first)
                weights(b0);
#pragma unroll
            for (int u = 0; u < kDirectAhead; ++u) {
                if (b0 + u >= end)
                    break;
                v4i x[2];
                x[0] = *reinterpret_cast<const v4i *>(row + (b0 + u) * kBlock + sub * 16);
                x[1] = *reinterpret_cast<const v4i *>(row + (b0 + u) * kBlock + 64 + sub * 16);
                const f32x4 p = block_product(w[u], x);
                const float s = *reinterpret_cast<const float *>(row + a.blocks * 128 + (b0 + u) * 4) * sw[u];
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    acc[k] = __builtin_fmaf(p[k], s, acc[k]);
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            total[k] = __builtin_fmaf(weight, acc[k], total[k]);
    }
    if (wave > 0)
        part[wave - 1][lane] = total;
    __syncthreads();
    if (wave != 0 || (lane & 15) != 0)
        return;                                            // (all 16 columns of the product are the one token)
#pragma unroll
    for (int v = 0; v < kDirectWaves - 1; ++v)
        total += part[v][lane];
    const int64_t at = (int64_t)token * a.ldo + 16 * nb + 4 * sub;
    if constexpr (E == kF32)
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at) = total;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
            make_uint2(pack2<E == kF16>(total[0], total[1]), pack2<E == kF16>(total[2], total[3]));
}

template <class S>
constexpr BlockTileEntry entry(const char *name)
{
    // (the experts run on the last two tiles)
    BlockMmKernel up = nullptr, down = nullptr;
    if constexpr (S::NT) {
        up = block_mm_small_kernel<S, kJobGateUp, kOutI32, kCodes>;
        down = block_mm_small_kernel<S, kJobDown, kOutI32, kCodes>;
    }
    return BlockTileEntry{
        name, S::BM, S::BN, S::THREADS, true,
        {block_mm_small_kernel<S, kJobDense, kOutBF16, kCodes>, block_mm_small_kernel<S, kJobDense, kOutI32, kCodes>,
         block_mm_small_kernel<S, kJobDense, kOutF16, kCodes>},
        up, down};
}

// 16 token rows x 16*FN*WN channels / WN x WK waves / U blocks at a time.
const BlockTileEntry kSmall[] = {
    entry<Small<2, 1, 8, 4, false>>("s16x32/n1k8/u4"),
    entry<Small<2, 1, 8, 2, true>>("s16x32/n1k8/u2nt"),
    entry<Small<2, 4, 2, 4, true>>("s16x128/n4k2/u4nt"),
};
static_assert(sizeof(kSmall) / sizeof(kSmall[0]) == kBlockSmallTiles, "tiles");

// The quant in the same launch: of a layer's rows, and of slots' tokens.
template <class S, int E>
constexpr BlockMmKernel quant_kernel(int mode)
{
    return mode == kOutBF16  ? block_mm_small_kernel<S, kJobDense, kOutBF16, E>
           : mode == kOutI32 ? block_mm_small_kernel<S, kJobDense, kOutI32, E>
                             : block_mm_small_kernel<S, kJobDense, kOutF16, E>;
}
template <class S>
BlockMmKernel quant_pick(int kind, int mode)
{
    return kind == kElemF32 ? quant_kernel<S, kF32>(mode) : kind == kElemF16 ? quant_kernel<S, kF16>(mode)
                                                                             : quant_kernel<S, kBF16>(mode);
}
using Plain = Small<2, 1, 8, 4, false>;
using Stream = Small<2, 1, 8, 2, true>;

}  // namespace

const BlockTileEntry &fp8_block_small(int i) { return kSmall[i]; }

hipError_t launch_fp8_block_small_quant(BlockMmArgs a, int x_kind, int mode, int i, hipStream_t stream)
{
    const BlockTileEntry &e = kSmall[i];
    const int64_t rows = std::min<int64_t>(a.M, e.bm);
    if (i > 1 || ceil_div(rows * a.blocks * 16, e.threads) > kSlots)
        return hipErrorNotSupported;
    a.tiles_m = (int)ceil_div(a.M, e.bm);
    const int64_t tiles = a.tiles_m * ceil_div(a.frags, e.bn / 16);
    hipLaunchKernelGGL(i == 0 ? quant_pick<Plain>(x_kind, mode) : quant_pick<Stream>(x_kind, mode),
                       dim3((unsigned)tiles), dim3(e.threads), (size_t)(rows * row_bytes(a.blocks)), stream, a);
    return hipGetLastError();
}

bool fp8_block_direct_fits(int top_k, int64_t K, int64_t inner)
{
    return ceil_div(K, kBlock) * 16 <= kSlots * Stream::THREADS &&
           top_k * ceil_div(inner, kBlock) * 16 <= kSlots * 64 * kDirectWaves;
}

hipError_t launch_fp8_block_direct(BlockMmArgs up, BlockMmArgs down, int x_kind, int tokens, hipStream_t stream)
{
    auto fn = x_kind == kElemF32   ? block_mm_small_kernel<Stream, kJobGateUp, kOutI32, kF32>
              : x_kind == kElemF16 ? block_mm_small_kernel<Stream, kJobGateUp, kOutI32, kF16>
                                   : block_mm_small_kernel<Stream, kJobGateUp, kOutI32, kBF16>;
    hipLaunchKernelGGL(fn, dim3((unsigned)(up.M * ceil_div(up.frags, Stream::BF))), dim3(Stream::THREADS),
                       (size_t)row_bytes(up.blocks), stream, up);
    hipError_t err = hipGetLastError();
    if (err != hipSuccess)
        return err;
    down.M = tokens;
    auto last = x_kind == kElemF32   ? down_direct_kernel<kF32>
                : x_kind == kElemF16 ? down_direct_kernel<kF16> : down_direct_kernel<kBF16>;
    hipLaunchKernelGGL(last, dim3((unsigned)(tokens * down.frags)), dim3(64 * kDirectWaves),
                       (size_t)(down.top_k * row_bytes(down.blocks)), stream, down);
    return hipGetLastError();
}

}  // namespace w8a8
