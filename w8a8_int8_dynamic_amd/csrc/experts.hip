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
#include "quant_fp8_block.hpp"

namespace w8a8 {
namespace {

using namespace fp8_block;

// Threads of a workgroup and ids that each holds at a time: more where there are
// many slots to go through. The ids of a run of kThreads * AHEAD slots are loaded
// at once and stay in registers for both looks at them: beside the quantization's
// loads a load takes microseconds (32768 slots, 64 experts: 28 us with 1024 x 4,
// 17 with 1024 x 32).
constexpr int kFewSlots = 4096, kFewThreads = 256, kFewAhead = 4, kManyThreads = 1024, kManyAhead = 32;

// The plan of expert e by one workgroup: where its rows begin (the slots of
// lower experts come first), its slots in ascending order, and its row tiles of
// bm rows. Every workgroup counts all experts by itself (LDS counters: their
// sums do not depend on the order), so that none waits for another. The last
// one writes the number of row tiles behind them.
template <int kThreads, int AHEAD>
__device__ __forceinline__ void plan_expert(int e, const int *__restrict__ ids, int slots, int experts, int bm,
                                            int *__restrict__ order, BlockTile *__restrict__ tiles, int tiles_m)
{
    constexpr int WAVES = kThreads / 64, RUN = kThreads * AHEAD;
    __shared__ int count[kMaxExperts];
    __shared__ int sums[2];
    __shared__ int in_wave[WAVES];
    const int t = threadIdx.x, wave = t >> 6, lane = t & 63;
    for (int i = t; i < experts; i += kThreads)
        count[i] = 0;
    if (t < 2)
        sums[t] = 0;
    __syncthreads();
    // Of a run, wave w has the ids from w * 64 * AHEAD on, in rows of 64.
    const int mine0 = wave * 64 * AHEAD + lane;
    int id[AHEAD];
    auto load = [&](int i0) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const int i = i0 + mine0 + q * 64;
            id[q] = i < slots ? ids[i] : -1;
        }
    };
    for (int i0 = 0; i0 < slots; i0 += RUN) {
        load(i0);
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
            if (id[q] >= 0 && id[q] < experts)
                atomicAdd(&count[id[q]], 1);
    }
    __syncthreads();
    int before = 0, before_tiles = 0;
    for (int i = t; i < e; i += kThreads) {
        before += count[i];
        before_tiles += (count[i] + bm - 1) / bm;
    }
    if (t < e) {
        atomicAdd(&sums[0], before);
        atomicAdd(&sums[1], before_tiles);
    }
    __syncthreads();
    const int first = sums[0], tile0 = sums[1], rows = count[e], mine = (rows + bm - 1) / bm;
    for (int i = t; i < mine; i += kThreads)
        tiles[tile0 + i] = BlockTile{e, first + i * bm, min(bm, rows - i * bm)};
    if (e == experts - 1 && t == 0)
        tiles[tiles_m] = BlockTile{-1, 0, tile0 + mine};
    if (rows == 0)
        return;
    int at = first;
    for (int i0 = 0; i0 < slots; i0 += RUN) {
        if (slots > RUN)                                  // (a single run is still in registers)
            load(i0);
        int hits = 0;
#pragma unroll
        for (int q = 0; q < AHEAD; ++q)
            hits += __popcll(__ballot(id[q] == e));
        if (lane == 0)
            in_wave[wave] = hits;
        __syncthreads();
        int all = 0, place = at;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const int n = in_wave[w];
            all += n;
            place += w < wave ? n : 0;
        }
#pragma unroll
        for (int q = 0; q < AHEAD; ++q) {
            const unsigned long long mask = __ballot(id[q] == e);
            if (id[q] == e)
                order[place + __popcll(mask & ((1ull << lane) - 1))] = i0 + mine0 + q * 64;
            place += __popcll(mask);
        }
        at += all;
        __syncthreads();
    }
}

// The plan, one workgroup per expert, and beside it the quantization of the
// tokens' rows: neither waits for the other.
template <int E, int U, int kThreads, int AHEAD>
__global__ __launch_bounds__(kThreads) void prepare_kernel(const int *__restrict__ ids, int slots, int experts, int bm,
                                                           int *__restrict__ order, BlockTile *__restrict__ tiles,
                                                           int tiles_m, const char *__restrict__ x, int64_t rows,
                                                           int units, int padded, int64_t ldx, uint8_t *__restrict__ q,
                                                           int64_t ldq, float *__restrict__ s, int64_t lds, int segs,
                                                           int rpb)
{
    if ((int)blockIdx.x < experts)
        plan_expert<kThreads, AHEAD>(blockIdx.x, ids, slots, experts, bm, order, tiles, tiles_m);
    else
        quant_block_rows<E, U>((int64_t)(blockIdx.x - experts) * (kThreads / 256) + threadIdx.x / 256,
                               threadIdx.x % 256, x, rows, units, padded, ldx, q, ldq, s, lds, segs, rpb);
}

template <int E, int N, int A>
auto prepare_pick(int u)
{
    return u == 1 ? prepare_kernel<E, 1, N, A> : u == 2 ? prepare_kernel<E, 2, N, A>
         : u == 3 ? prepare_kernel<E, 3, N, A> : prepare_kernel<E, 4, N, A>;
}
template <int E>
auto prepare_pick(int u, bool many)
{
    return many ? prepare_pick<E, kManyThreads, kManyAhead>(u) : prepare_pick<E, kFewThreads, kFewAhead>(u);
}

// out[t] = sum over the token's slots of weight * y[slot], y fp32 rows or fp16
// rows under a scale per 128 columns: eight columns a thread. A slot without an
// expert has no row. HBM-bound: 4096 tokens of 8 slots, K 4096 53 us, 5.7 TB/s.
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
        const float w = weights[slot];
        float v[8];
        if constexpr (Y16) {
            const float s = y_scale[slot * ld_scale + col / kBlock];
            const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(y) + slot * K + col);
            const u32 d[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
            for (int r = 0; r < 8; ++r)
                v[r] = quant_rule::f16_to_float(d[r >> 1] >> (16 * (r & 1))) * s;   // (exact)
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
};

// How a pass runs: slots alone in two launches, or by a plan, on tiles of the
// main kernel or of the small-M one (those of the up and the down products).
struct Path {
    bool direct;
    int bm;                      // rows of a tile, at most
    const BlockTileEntry *up, *down;
    BlockMmKernel gate_up;
    bool small() const { return up->small; }
};

// The choice, by what each side took (us, the whole layer; A: 64 experts, K 4096,
// inner 1024, 4 a token; B: 24, 2064, 720, 3; C: 8, 4096, 2048):
//   small-M tiles up to 10 rows an expert, on average, then the main kernel's:
//     A at 8 rows 155 against 183, at 16 rows 218 against 186; B 41 : 45, 49 : 49.
//     Of those 16 x 128, but 16 x 32 where K is long and column tiles are few: A at
//     4 slots 8 tokens 70 against 74, at 64 slots 104 : 101, B 41 : 47;
//   its 128 x 256 tile up to 104 rows, then 256 x 256:
//     A at 64 rows 192 : 200, at 96 210 : 221, at 112 243 : 228, at 256 404 : 376;
//     B at 96 59 : 64, at 128 72 : 67 (64 x 256 tiles gained 2 % at most, below 32);
//     of it, kCutRows rows at a time and with exact gated products (main_fp8_block.hpp) up to
//     32 rows. Against whole tiles of e4m3 products that costs, at 24 rows of uneven
//     shares, B 50 : 47, A 222 : 184, C 69 : 62; exact whole tiles would at 41 rows, B 58
//     : 51, A 252 : 215, C 84 : 65, and at 64, B 65 : 56, A 278 : 225, C 86 : 67;
//   slots alone, without a plan, each with its expert's weights to itself, for up
//   to four tokens and 24 slots, no more than there are experts (more would read
//   weights twice): A, one token of 8 25.6 : 39.0, three of 8 56 : 63, eight of 1
//   42.8 : 35.4; C, two of 8 58 : 48.
constexpr int kSmallRows = 10, kExactRows = 32, kHalfRows = 104, kDirectTokens = 4, kDirectSlots = 24;

Path path_of(int64_t tokens, int top_k, int experts, int64_t K, int64_t inner)
{
    const int64_t slots = tokens * top_k, rows = slots / experts;   // rows of an expert, on average
    Path p{};
    if (rows > kSmallRows) {
        p.up = p.down = &fp8_block_main(rows > kHalfRows ? 0 : 1);
        const bool cut = rows <= kExactRows;
        p.bm = cut ? kCutRows : p.up->bm;
        p.gate_up = cut ? p.up->gate_up_cut : p.up->gate_up;
        return p;
    }
    p.direct = tokens <= kDirectTokens && slots <= std::min(kDirectSlots, experts) &&
               fp8_block_direct_fits(top_k, K, inner);
    // (of K, frags / 8 column tiles of an expert)
    auto small = [&](int64_t k, int64_t frags) {
        return &fp8_block_small(k > 1024 && std::min<int64_t>(slots, experts) * ceil_div(frags, 8) <= 512 ? 1 : 2);
    };
    p.up = small(K, fp8_block_frags(2 * inner, true));
    p.down = small(inner, fp8_block_frags(K, false));
    p.bm = p.up->bm;
    p.gate_up = p.up->gate_up;
    return p;
}

// Row tiles of a launch, at most.
int64_t most_tiles(int64_t slots, int experts, int bm) { return slots / bm + std::min<int64_t>(experts, slots); }

// Workgroups of a product's launch: 3.5 million of 512 threads at most (a pass has
// up to 65536 slots; 10 rows an expert on 16 x 128 tiles of 131056 rows of weights),
// so that threads are counted in 32 bits.
int64_t grid_of(const BlockTileEntry &e, int64_t tiles_m, int64_t frags)
{
    const int64_t tiles_n = ceil_div(frags, e.bn / 16);
    return e.small ? tiles_m * tiles_n : expert_grid(tiles_m, tiles_n);
}

Layout layout_of(int64_t tokens, int top_k, int experts, int64_t K, int64_t inner, const Path &p)
{
    Layout l;
    const int64_t slots = tokens * top_k;
    const bool small = p.small();
    size_t at = 0;
    auto take = [&](int64_t bytes) {
        const size_t o = at;
        at += (size_t)round_up(bytes, 256);
        return o;
    };
    l.h = take(small ? slots * inner * 4 : 0);
    if (p.direct) {
        l.end = at;
        return l;
    }
    l.xq = take(tokens * K);
    l.xs = take(tokens * scale_pitch(K) * 4);
    l.order = take(slots * 4);
    l.tiles = take((most_tiles(slots, experts, p.bm) + 1) * (int64_t)sizeof(BlockTile));
    l.hq = take(slots * inner);
    l.hs = take(slots * scale_pitch(inner) * 4);
    l.y = take(slots * K * (small ? 4 : 2));
    l.ys = take(small ? 0 : slots * ceil_div(K, kBlock) * 4);
    l.end = at;
    return l;
}

}  // namespace

size_t experts_workspace_bytes(int64_t tokens, int top_k, int experts, int64_t K, int64_t inner)
{
    const int64_t step = tokens_at_once(tokens, top_k, K);
    return layout_of(step, top_k, experts, K, inner, path_of(step, top_k, experts, K, inner)).end;
}

hipError_t launch_experts(const ExpertsArgs &args, void *workspace, hipStream_t stream)
{
    const int64_t step = tokens_at_once(args.tokens, args.top_k, args.K);
    // (the last pass, if shorter, runs as the others do)
    const Path p = path_of(step, args.top_k, args.experts, args.K, args.inner);
    const Layout l = layout_of(step, args.top_k, args.experts, args.K, args.inner, p);
    char *work = static_cast<char *>(workspace);
    const int x_bytes = args.kind == kElemF32 ? 4 : 2;
    const int blocks = (int)ceil_div(args.K, kBlock), inner_blocks = (int)ceil_div(args.inner, kBlock);

    for (int64_t t0 = 0; t0 < args.tokens; t0 += step) {
        const int64_t tokens = std::min(args.tokens - t0, step);
        const int slots = (int)(tokens * args.top_k);
        const int *ids = args.ids + t0 * args.top_k;
        const float *weights = args.weights + t0 * args.top_k;
        const char *x = static_cast<const char *>(args.x) + t0 * args.ldx * x_bytes;
        char *out = static_cast<char *>(args.out) + t0 * args.ldo * x_bytes;

        BlockMmArgs up{}, down{};
        up.top_k = down.top_k = args.top_k;
        up.experts = down.experts = args.experts;
        up.vec_store = down.vec_store = down.vec16 = 1;
        up.M = down.M = slots;
        up.wp = args.gate_up;
        up.ws = args.gate_up_scale;
        up.N = (int)(2 * args.inner);
        up.K = (int)args.K;
        up.blocks = blocks;
        up.frags = (int)fp8_block_frags(up.N, true);
        up.half_scales = inner_blocks;
        up.expert_bytes = (int64_t)up.frags * blocks * kFrag;
        up.expert_scales = (int64_t)2 * inner_blocks * blocks;
        up.ldo = args.inner;
        down.wp = args.down;
        down.ws = args.down_scale;
        down.N = (int)args.K;
        down.K = (int)args.inner;
        down.blocks = inner_blocks;
        down.frags = (int)fp8_block_frags(down.N, false);
        down.expert_bytes = (int64_t)down.frags * inner_blocks * kFrag;
        down.expert_scales = fp8_block_scale_rows(down.N, false) * inner_blocks;

        hipError_t err;
        if (p.direct) {
            up.ids = down.ids = ids;
            up.x = x;
            up.ldx = args.ldx;
            up.out = work + l.h;
            down.weights = weights;
            down.x = work + l.h;
            down.ldx = args.inner;
            down.out = out;
            down.ldo = args.ldo;
            err = launch_fp8_block_direct(up, down, args.kind, (int)tokens, stream);
            if (err != hipSuccess)
                return err;
            continue;
        }

        uint8_t *xq = reinterpret_cast<uint8_t *>(work + l.xq), *hq = reinterpret_cast<uint8_t *>(work + l.hq);
        float *xs = reinterpret_cast<float *>(work + l.xs), *hs = reinterpret_cast<float *>(work + l.hs);
        float *ys = reinterpret_cast<float *>(work + l.ys);
        int *order = reinterpret_cast<int *>(work + l.order);
        BlockTile *tiles = reinterpret_cast<BlockTile *>(work + l.tiles);
        const int bm = p.bm, tiles_m = (int)most_tiles(slots, args.experts, bm);
        const int units = (int)(args.K / 8), padded = blocks * 16;
        const Cut c = cut_of(tokens, padded);
        const bool many = slots > kFewSlots;
        const int threads = many ? kManyThreads : kFewThreads;
        auto prepare = args.kind == kElemF32 ? prepare_pick<kF32>(c.u, many)
                     : args.kind == kElemF16 ? prepare_pick<kF16>(c.u, many) : prepare_pick<kBF16>(c.u, many);
        hipLaunchKernelGGL(prepare, dim3((unsigned)(args.experts + ceil_div(c.blocks, threads / 256))), dim3(threads),
                           0, stream, ids, slots, args.experts, bm, order, tiles, tiles_m, x, tokens, units, padded,
                           args.ldx, xq, args.K, xs, scale_pitch(args.K), c.segs, c.rpb);

        up.tiles = down.tiles = tiles;
        up.tiles_m = down.tiles_m = tiles_m;
        up.order = down.order = order;
        up.xq = xq;
        up.xs = xs;
        up.ldq = args.K;
        up.lds = scale_pitch(args.K);
        up.out = p.small() ? static_cast<void *>(work + l.h) : hq;
        up.out_scale = hs;
        up.ld_out_scale = scale_pitch(args.inner);
        hipLaunchKernelGGL(p.gate_up, dim3((unsigned)grid_of(*p.up, tiles_m, up.frags)), dim3(p.up->threads), 0,
                           stream, up);
        if (p.small()) {
            err = launch_quant_fp8_block(work + l.h, kElemF32, slots, args.inner, args.inner, hq, args.inner, hs,
                                         scale_pitch(args.inner), stream);
            if (err != hipSuccess)
                return err;
        }
        down.xq = hq;
        down.xs = hs;
        down.ldq = args.inner;
        down.lds = scale_pitch(args.inner);
        down.out = work + l.y;
        down.ldo = args.K;
        down.out_scale = ys;
        down.ld_out_scale = blocks;
        hipLaunchKernelGGL(p.down->down, dim3((unsigned)grid_of(*p.down, tiles_m, down.frags)), dim3(p.down->threads),
                           0, stream, down);

        const int segs = (int)ceil_div(args.K, 2048);
        auto combine = args.kind == kElemF32 ? combine_pick<kF32>(!p.small())
                     : args.kind == kElemF16 ? combine_pick<kF16>(!p.small()) : combine_pick<kBF16>(!p.small());
        hipLaunchKernelGGL(combine, dim3((unsigned)(tokens * segs)), dim3(256), 0, stream, work + l.y, ys, blocks, ids,
                           weights, args.top_k, args.experts, (int)args.K, out, args.ldo, segs);
        err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace w8a8
