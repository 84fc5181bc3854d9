// The mixture of experts: for each token t with chosen experts e_j and weights
// w_j (an id outside [0, experts) stands for no expert)
//   h_j = silu(gate_e x) * (up_e x)                     fp32
//   out_t = sum over j of w_j * down_e q(h_j)           fp32, rounded once
// with x and h as block-scaled e4m3 rows (fp8_block_rule.hpp) and the experts'
// weights block-scaled e4m3 matrices.
//
// The plan sets the slots (token, choice) out by expert, so that each expert's
// rows are one run, cut into row tiles; the products then run over all
// experts' tiles in one launch each, the first gathering its rows by token,
// the second scattering them back to slots. The sum over a token's slots comes
// last, in the slots' order, so that no result depends on an order of atomics.
#include <algorithm>

#include "experts.hpp"
#include "fp8_block_device.hpp"

namespace w8a8 {
namespace {

using namespace fp8_block;

constexpr int kPlanThreads = 1024;

// One workgroup per expert: where its rows begin (the slots of lower experts
// come first), its slots in ascending order, and its row tiles. Every
// workgroup counts all experts by itself (LDS counters: their sums do not
// depend on the order), so that none waits for another.
__global__ __launch_bounds__(kPlanThreads) void plan_kernel(const int *__restrict__ ids, int slots, int experts,
                                                            int bm, int *__restrict__ order,
                                                            BlockTile *__restrict__ tiles, int tiles_m)
{
    __shared__ int count[kMaxExperts];
    __shared__ int sums[2];
    __shared__ int in_wave[kPlanThreads / 64];
    const int t = threadIdx.x, e = blockIdx.x, wave = t >> 6;
    if (t < experts)
        count[t] = 0;
    if (t < 2)
        sums[t] = 0;
    __syncthreads();
    for (int i = t; i < slots; i += kPlanThreads) {
        const int id = ids[i];
        if (id >= 0 && id < experts)
            atomicAdd(&count[id], 1);
    }
    __syncthreads();
    if (t < e) {
        atomicAdd(&sums[0], count[t]);
        atomicAdd(&sums[1], (count[t] + bm - 1) / bm);
    }
    __syncthreads();
    const int first = sums[0], tile0 = sums[1], rows = count[e], mine = (rows + bm - 1) / bm;
    for (int i = t; i < mine; i += kPlanThreads)
        tiles[tile0 + i] = BlockTile{e, first + i * bm, min(bm, rows - i * bm)};
    if (e == experts - 1 && t == 0)
        tiles[tiles_m] = BlockTile{-1, 0, tile0 + mine};
    if (rows == 0)
        return;
    int at = first;
    for (int i0 = 0; i0 < slots; i0 += kPlanThreads) {
        const int i = i0 + t;
        const bool hit = i < slots && ids[i] == e;
        const unsigned long long mask = __ballot(hit);
        if ((t & 63) == 0)
            in_wave[wave] = __popcll(mask);
        __syncthreads();
        int before = 0, all = 0;
#pragma unroll
        for (int w = 0; w < kPlanThreads / 64; ++w) {
            before += w < wave ? in_wave[w] : 0;
            all += in_wave[w];
        }
        if (hit)
            order[at + before + __popcll(mask & ((1ull << (t & 63)) - 1))] = i;
        at += all;
        __syncthreads();
    }
}

// out[t] = sum over the token's slots of weight * y[slot], y fp32 rows or fp16
// rows under a scale per 128 columns: eight columns a thread. A slot without an
// expert has no row.
template <int E, bool Y16>
__global__ __launch_bounds__(256) void combine_kernel(const void *__restrict__ y, const float *__restrict__ y_scale,
                                                      int ld_scale, const int *__restrict__ ids,
                                                      const float *__restrict__ weights, int top_k, int experts,
                                                      int K, void *__restrict__ out, int64_t ldo, int segs)
{
    const int64_t token = blockIdx.x / segs;
    const int col = ((int)(blockIdx.x - token * segs) * 256 + (int)threadIdx.x) * 8;
    if (col >= K)
        return;
    float acc[8] = {};
    for (int j = 0; j < top_k; ++j) {
        const int64_t slot = token * top_k + j;
        const int id = ids[slot];
        if (id < 0 || id >= experts)
            continue;
        float w = weights[slot], v[8];
        if constexpr (Y16) {
            w *= y_scale[slot * ld_scale + col / kBlock];
            const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(y) + slot * K + col);
            const u32 d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int r = 0; r < 8; ++r)
                v[r] = quant_rule::f16_to_float(d[r >> 1] >> (16 * (r & 1)));
        } else {
            const f32x4 *q = reinterpret_cast<const f32x4 *>(static_cast<const float *>(y) + slot * K + col);
            const f32x4 lo = q[0], hi = q[1];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                v[r] = lo[r];
                v[4 + r] = hi[r];
            }
        }
#pragma unroll
        for (int r = 0; r < 8; ++r)
            acc[r] = __builtin_fmaf(w, v[r], acc[r]);
    }
    if constexpr (E == kF32) {
        f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(out) + token * ldo + col);
        o[0] = f32x4{acc[0], acc[1], acc[2], acc[3]};
        o[1] = f32x4{acc[4], acc[5], acc[6], acc[7]};
    } else {
        constexpr bool H = E == kF16;
        *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(out) + token * ldo + col) =
            make_uint4(pack2<H>(acc[0], acc[1]), pack2<H>(acc[2], acc[3]), pack2<H>(acc[4], acc[5]),
                       pack2<H>(acc[6], acc[7]));
    }
}

template <int E>
auto combine_pick(bool y16)
{
    return y16 ? combine_kernel<E, true> : combine_kernel<E, false>;
}

// Tokens of one pass: what bounds the workspace and keeps every row offset of
// the codes within 31 bits.
int64_t tokens_at_once(int64_t tokens, int top_k, int64_t K)
{
    const int64_t most = std::max<int64_t>(1, std::min<int64_t>(65536 / top_k, (int64_t(1) << 30) / K));
    return std::min(tokens, most);
}

// Scales per row of codes, in whole 16 bytes.
int64_t scale_pitch(int64_t K) { return round_up(ceil_div(K, kBlock), 4); }

struct Layout {
    size_t xq, xs, order, tiles, hq, hs, h, y, ys, end;
    int64_t tiles_m;
};

Layout layout_of(int64_t tokens, int top_k, int experts, int64_t K, int64_t inner, const BlockTileEntry &e)
{
    Layout l;
    const int bm = e.bm;
    const bool small = e.small;
    const int64_t slots = tokens * top_k;
    l.tiles_m = slots / bm + std::min<int64_t>(experts, slots);
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t p = at;
        at += (size_t)round_up(bytes, 256);
        return p;
    };
    l.xq = take(tokens * K);
    l.xs = take(tokens * scale_pitch(K) * 4);
    l.order = take(slots * 4);
    l.tiles = take((l.tiles_m + 1) * (int64_t)sizeof(BlockTile));
    l.hq = take(slots * inner);
    l.hs = take(slots * scale_pitch(inner) * 4);
    l.h = take(small ? slots * inner * 4 : 0);
    l.y = take(slots * K * (small ? 4 : 2));
    l.ys = take(small ? 0 : slots * ceil_div(K, kBlock) * 4);
    l.end = at;
    return l;
}

const BlockTileEntry &tile_of_call(int64_t tokens, int top_k, int experts)
{
    const int64_t rows = tokens * top_k / experts;       // of an expert, on average
    return rows > 128 ? fp8_block_main(0) : rows > 32 ? fp8_block_main(1) : fp8_block_small(0);
}

}  // namespace

size_t experts_workspace_bytes(int64_t tokens, int top_k, int experts, int64_t K, int64_t inner)
{
    const int64_t step = tokens_at_once(tokens, top_k, K);
    return layout_of(step, top_k, experts, K, inner, tile_of_call(step, top_k, experts)).end;
}

bool experts_fit(int64_t tokens, int top_k, int experts, int64_t K, int64_t inner)
{
    const int64_t step = tokens_at_once(tokens, top_k, K);
    const BlockTileEntry &e = tile_of_call(step, top_k, experts);
    const int64_t tiles_m = step * top_k / e.bm + std::min<int64_t>(experts, step * top_k);
    return mm_grid_fits(tiles_m * ceil_div(std::max(2 * inner, K), e.bn), e.threads);
}

hipError_t launch_experts(const ExpertsArgs &args, void *workspace, hipStream_t stream)
{
    const int64_t step = tokens_at_once(args.tokens, args.top_k, args.K);
    const BlockTileEntry &e = tile_of_call(step, args.top_k, args.experts);
    const Layout l = layout_of(step, args.top_k, args.experts, args.K, args.inner, e);
    char *work = static_cast<char *>(workspace);
    const int x_bytes = args.kind == kElemF32 ? 4 : 2;
    const int blocks = (int)ceil_div(args.K, kBlock), inner_blocks = (int)ceil_div(args.inner, kBlock);
    uint8_t *xq = reinterpret_cast<uint8_t *>(work + l.xq), *hq = reinterpret_cast<uint8_t *>(work + l.hq);
    float *xs = reinterpret_cast<float *>(work + l.xs), *hs = reinterpret_cast<float *>(work + l.hs);
    float *h = reinterpret_cast<float *>(work + l.h), *ys = reinterpret_cast<float *>(work + l.ys);
    void *y = work + l.y;
    int *order = reinterpret_cast<int *>(work + l.order);
    BlockTile *tiles = reinterpret_cast<BlockTile *>(work + l.tiles);

    for (int64_t t0 = 0; t0 < args.tokens; t0 += step) {
        const int64_t tokens = std::min(args.tokens - t0, step);
        const int slots = (int)(tokens * args.top_k);
        const int *ids = args.ids + t0 * args.top_k;
        hipError_t err = launch_quant_fp8_block(static_cast<const char *>(args.x) + t0 * args.ldx * x_bytes, args.kind,
                                                tokens, args.K, args.ldx, xq, args.K, xs, scale_pitch(args.K),
                                                stream);
        if (err != hipSuccess)
            return err;
        const int tiles_m = (int)(slots / e.bm + std::min(args.experts, slots));
        hipLaunchKernelGGL(plan_kernel, dim3(args.experts), dim3(kPlanThreads), 0, stream, ids, slots, args.experts,
                           e.bm, order, tiles, tiles_m);

        BlockMmArgs m{};
        m.tiles = tiles;
        m.tiles_m = tiles_m;
        m.order = order;
        m.top_k = args.top_k;
        m.vec_store = 1;
        m.xq = xq;
        m.xs = xs;
        m.ldq = args.K;
        m.lds = scale_pitch(args.K);
        m.wp = args.gate_up;
        m.ws = args.gate_up_scale;
        m.out = e.small ? static_cast<void *>(h) : hq;
        m.ldo = args.inner;
        m.out_scale = hs;
        m.ld_out_scale = scale_pitch(args.inner);
        m.M = slots;
        m.N = (int)(2 * args.inner);
        m.K = (int)args.K;
        m.blocks = blocks;
        m.frags = (int)fp8_block_frags(m.N, true);
        m.half_scales = inner_blocks;
        m.expert_bytes = (int64_t)m.frags * blocks * kFrag;
        m.expert_scales = (int64_t)2 * inner_blocks * blocks;
        hipLaunchKernelGGL(e.gate_up, dim3((unsigned)(tiles_m * ceil_div(m.frags, e.bn / 16))), dim3(e.threads), 0,
                           stream, m);
        if (e.small) {
            err = launch_quant_fp8_block(h, kElemF32, slots, args.inner, args.inner, hq, args.inner, hs,
                                         scale_pitch(args.inner), stream);
            if (err != hipSuccess)
                return err;
        }
        m.xq = hq;
        m.xs = hs;
        m.ldq = args.inner;
        m.lds = scale_pitch(args.inner);
        m.wp = args.down;
        m.ws = args.down_scale;
        m.out = y;
        m.ldo = args.K;
        m.vec16 = 1;
        m.out_scale = ys;
        m.ld_out_scale = blocks;
        m.N = (int)args.K;
        m.K = (int)args.inner;
        m.blocks = inner_blocks;
        m.frags = (int)fp8_block_frags(m.N, false);
        m.half_scales = 0;
        m.expert_bytes = (int64_t)m.frags * inner_blocks * kFrag;
        m.expert_scales = fp8_block_scale_rows(m.N, false) * inner_blocks;
        hipLaunchKernelGGL(e.down, dim3((unsigned)(tiles_m * ceil_div(m.frags, e.bn / 16))), dim3(e.threads), 0,
                           stream, m);

        const int segs = (int)ceil_div(args.K, 2048);
        auto combine = args.kind == kElemF32 ? combine_pick<kF32>(!e.small)
                     : args.kind == kElemF16 ? combine_pick<kF16>(!e.small) : combine_pick<kBF16>(!e.small);
        hipLaunchKernelGGL(combine, dim3((unsigned)(tokens * segs)), dim3(256), 0, stream, y, ys, blocks, ids,
                           args.weights + t0 * args.top_k, args.top_k, args.experts, (int)args.K,
                           static_cast<char *>(args.out) + t0 * args.ldo * x_bytes, args.ldo, segs);
        err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace w8a8
