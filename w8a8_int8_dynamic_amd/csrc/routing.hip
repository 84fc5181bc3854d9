// Routing of tokens to experts, on gfx950.
//   score_e  = softmax(logits)_e or 1 / (1 + e^-logit_e)
//   choice_e = score_e + bias_e
//   groups: the experts in G equal groups; a group's worth is the sum of its
//   group_top (1 or 2) largest choices; the top_groups best groups stay.
//   ids: the top_k experts of the groups that stayed, by choice, the best first
//   weights: their scores, over their sum (renormalize), times scale
// Ties go to the lowest index. An expert whose logit is NaN or -infinity (or
// whose bias is) is left out; where fewer than top_k are left, the rest of the
// row is id -1 with weight 0.
//
// Scores are computed in 64 bits: which expert comes first hangs on the last
// bits of a sum of a score and a bias, and whole experts' outputs on that.
//
// What bounds it is the vector unit where there are many tokens (at 256 experts
// a token costs four wavefront instructions for every step of its 64-bit
// exponential and division, and the selection's steps come on top) and the
// chain of a token's steps where there are few. So exchanges between lanes stay
// in registers (DPP and row swaps), a lane sorts out its three best choices once
// and a step of the selection compares only the lanes' best, and the scores of
// the chosen are computed again at the end, one lane each, instead of being
// carried along. 256 experts in 8 groups, 8 chosen: 8192 tokens 14.9 us, one
// token 5.6 (with exchanges through LDS, all of a lane's choices compared at
// every step and the library's exponential: 31 and 10 us).
#include "experts.hpp"
#include "quant_rule.hpp"

namespace w8a8 {
namespace {

using quant_rule::kBF16;
using quant_rule::kF16;
using quant_rule::kF32;

constexpr int kWaves = 4;        // wavefronts per workgroup
constexpr int kBest = 3;         // choices that a lane sorts out at a time
constexpr double kOut = -__builtin_huge_val();   // the choice of an expert that is left out

// e^x: x = n ln 2 + r, |r| <= ln(2)/2, by the Taylor polynomial of degree 13
// (its remainder is below 2^-57 there). Beyond +-750 it is infinite or zero.
__device__ __forceinline__ double exp64(double x)
{
    x = fmin(fmax(x, -750.0), 750.0);
    const double n = __builtin_rint(x * 1.4426950408889634);
    double r = __builtin_fma(n, -0.6931471803691238, x);       // ln 2 in two parts, the first with zeros behind
    r = __builtin_fma(n, -1.9082149292705877e-10, r);
    double p = 1.0 / 6227020800.0;
    constexpr double c[13] = {1.0 / 479001600.0, 1.0 / 39916800.0, 1.0 / 3628800.0, 1.0 / 362880.0, 1.0 / 40320.0,
                              1.0 / 5040.0, 1.0 / 720.0, 1.0 / 120.0, 1.0 / 24.0, 1.0 / 6.0, 0.5, 1.0, 1.0};
#pragma unroll
    for (int i = 0; i < 13; ++i)
        p = __builtin_fma(p, r, c[i]);
    return __builtin_ldexp(p, (int)n);
}

// v from another lane of the row of 16, as DPP control CTRL says.
template <int CTRL>
__device__ __forceinline__ int dpp(int v)
{
    return __builtin_amdgcn_update_dpp(v, v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ double dpp(double v)
{
    const uint2 b = __builtin_bit_cast(uint2, v);
    return __builtin_bit_cast(double, make_uint2((unsigned)dpp<CTRL>((int)b.x), (unsigned)dpp<CTRL>((int)b.y)));
}
constexpr int kRor8 = 0x128, kRor4 = 0x124, kRor2 = 0x122, kRor1 = 0x121;   // row rotations

// op over each row of 16 lanes and the one beside it (SPAN 16), or each half of
// the wavefront and the other (SPAN 32): gfx950's swap of rows between two
// registers, of two copies of v, leaves each lane its own side's and the other's.
template <int SPAN, class Op>
__device__ __forceinline__ int across(int v, Op &&op)
{
    const auto s = SPAN == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                              : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    return op((int)s[0], (int)s[1]);
}
template <int SPAN, class Op>
__device__ __forceinline__ double across(double v, Op &&op)
{
    const uint2 b = __builtin_bit_cast(uint2, v);
    const auto x = SPAN == 16 ? __builtin_amdgcn_permlane16_swap(b.x, b.x, false, false)
                              : __builtin_amdgcn_permlane32_swap(b.x, b.x, false, false);
    const auto y = SPAN == 16 ? __builtin_amdgcn_permlane16_swap(b.y, b.y, false, false)
                              : __builtin_amdgcn_permlane32_swap(b.y, b.y, false, false);
    return op(__builtin_bit_cast(double, make_uint2(x[0], y[0])), __builtin_bit_cast(double, make_uint2(x[1], y[1])));
}

// op over the LANES (32 or 64) lanes of a token, the result in all of them.
template <int LANES, class V, class Op>
__device__ __forceinline__ V all(V v, Op &&op)
{
    v = op(v, dpp<kRor8>(v));
    v = op(v, dpp<kRor4>(v));
    v = op(v, dpp<kRor2>(v));
    v = op(v, dpp<kRor1>(v));
    v = across<16>(v, op);
    if constexpr (LANES == 64)
        v = across<32>(v, op);
    return v;
}
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }
__device__ __forceinline__ double sum_of(double a, double b) { return a + b; }
__device__ __forceinline__ int smaller(int a, int b) { return min(a, b); }

template <int E>
__device__ __forceinline__ double load_logit(const void *p, int64_t i)
{
    if constexpr (E == kF32)
        return static_cast<const float *>(p)[i];
    const unsigned v = static_cast<const uint16_t *>(p)[i];
    return E == kF16 ? quant_rule::f16_to_float(v) : __uint_as_float(v << 16);
}

// The two largest of both pairs (a1 >= a2, b1 >= b2).
__device__ __forceinline__ void two_largest(double &a1, double &a2, double b1, double b2)
{
    a2 = fmax(fmin(a1, b1), fmax(a2, b2));
    a1 = fmax(a1, b1);
}

// LANES lanes a token, V experts a lane: expert v * LANES + lane.
template <int E, int LANES, int V>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const RouteArgs a)
{
    constexpr int TOKENS = 64 / LANES;                    // tokens of a wavefront
    extern __shared__ __attribute__((aligned(16))) double shared[];   // groups: choices, then the groups' worths
    const int lane = threadIdx.x & (LANES - 1), mine = threadIdx.x / LANES;
    const int64_t token = (int64_t)blockIdx.x * (kWaves * TOKENS) + mine;
    const bool live = token < a.tokens;                   // (every wave meets the barriers)

    double choice[V], top = kOut;
    float bias[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * LANES + lane;
        const double x = live && e < a.experts ? load_logit<E>(a.logits, token * a.ld + e) : kOut;
        bias[v] = a.bias && e < a.experts ? a.bias[e] : 0.0f;
        choice[v] = x != x ? kOut : x;
        top = fmax(top, choice[v]);
    }
    // Scores of logits that are not left out; softmax: infinite ones share
    // the weight between them.
    const bool softmax = a.score == kScoreSoftmax;
    double sum = 1.0;
    auto part = [&](double x) __attribute__((always_inline)) { return x == top ? 1.0 : exp64(x - top); };
    auto sigmoid = [](double x) __attribute__((always_inline)) { return 1.0 / (1.0 + exp64(-x)); };
    if (softmax) {
        top = all<LANES>(top, larger);
        sum = 0.0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double p = part(choice[v]);
            sum += choice[v] == kOut ? 0.0 : p;
            choice[v] = choice[v] == kOut ? kOut : p;
        }
        sum = all<LANES>(sum, sum_of);
#pragma unroll
        for (int v = 0; v < V; ++v)
            choice[v] = choice[v] == kOut ? kOut : choice[v] / sum;
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double p = sigmoid(choice[v]);
            choice[v] = choice[v] == kOut ? kOut : p;
        }
    }
    if (a.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const double b = bias[v];
            choice[v] = choice[v] == kOut || b != b ? kOut : choice[v] + b;
        }
    }

    if (a.groups > 1) {
        // A group's lanes look at its choices in turn, then exchange their two
        // largest; every lane then counts the groups before its own.
        const int size = a.experts / a.groups, share = a.group_lanes;
        double *choices = shared + mine * a.experts, *worths = shared + kWaves * TOKENS * a.experts + mine * a.groups;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * LANES + lane < a.experts)
                choices[v * LANES + lane] = choice[v];
        __syncthreads();
        const int group = lane / share;
        double first = kOut, second = kOut;
        if (group < a.groups)
            for (int i = lane % share; i < size; i += share) {
                const double c = choices[group * size + i];
                second = fmax(second, fmin(first, c));
                first = fmax(first, c);
            }
        if (share > 1)
            two_largest(first, second, dpp<0xB1>(first), dpp<0xB1>(second));     // lane ^ 1
        if (share > 2)
            two_largest(first, second, dpp<0x4E>(first), dpp<0x4E>(second));     // lane ^ 2
        if (share > 4)
            two_largest(first, second, dpp<0x141>(first), dpp<0x141>(second));   // the row's halves mirrored
        if (share > 8)
            two_largest(first, second, dpp<0x140>(first), dpp<0x140>(second));   // the row mirrored
        // (a group with one expert left is worth that one)
        const double worth = a.group_top == 2 && second != kOut ? first + second : first;
        if (group < a.groups && lane % share == 0)
            worths[group] = worth;
        __syncthreads();
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double w = worths[g];
            before += w > worth || (w == worth && g < group);
        }
        const unsigned long long ballot = __ballot(group < a.groups && before < a.top_groups);
        const unsigned long long kept = LANES == 64 ? ballot : ballot >> (threadIdx.x & (64 - LANES));
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int g = (int)(((unsigned)(v * LANES + lane) * a.size_inverse) >> 20);   // expert / size
            if (!((kept >> min(g * share, 63)) & 1))
                choice[v] = kOut;
        }
    }

    // A lane's best choices not taken yet, the best first (of equal ones the
    // lowest expert: they come in order).
    double best[kBest];
    int id[kBest], left = 0;
    unsigned taken = 0;
    auto sort_out = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int b = 0; b < kBest; ++b) {
            best[b] = kOut;
            id[b] = 1 << 30;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            double c = (taken >> v) & 1 ? kOut : choice[v];
            int e = v * LANES + lane;
#pragma unroll
            for (int b = 0; b < kBest; ++b) {
                const bool up = c > best[b];
                const double c2 = up ? best[b] : c;
                const int e2 = up ? id[b] : e;
                best[b] = up ? c : best[b];
                id[b] = up ? e : id[b];
                c = c2;
                e = e2;
            }
        }
        left = kBest;
    };
    sort_out();

    // Lane j keeps the j-th choice.
    int my_id = -1;
    for (int j = 0; j < a.top_k; ++j) {
        if (V > kBest && __ballot(left == 0) != 0) {
            if (left == 0)
                sort_out();
        }
        const double most = all<LANES>(best[0], larger);
        const int winner = all<LANES>(best[0] == most ? id[0] : 1 << 30, smaller);
        const bool none = most == kOut;
        if (lane == j && !none)
            my_id = winner;
        if (!none && id[0] == winner) {
            taken |= 1u << (winner / LANES);
            left -= 1;
#pragma unroll
            for (int b = 0; b + 1 < kBest; ++b) {
                best[b] = best[b + 1];
                id[b] = id[b + 1];
            }
            best[kBest - 1] = kOut;
            id[kBest - 1] = 1 << 30;
        }
    }

    double score = 0.0;
    if (live && my_id >= 0) {
        const double x = load_logit<E>(a.logits, token * a.ld + my_id);
        score = softmax ? part(x) / sum : sigmoid(x);
    }
    if (a.renormalize) {
        const double total = all<LANES>(score, sum_of);
        score = total > 0.0 ? score / total : 0.0;
    }
    if (live && lane < a.top_k) {
        a.ids[token * a.top_k + lane] = my_id;
        a.weights[token * a.top_k + lane] = (float)(score * (double)a.scale);
    }
}

struct Variant {
    void (*kernel)(const RouteArgs);
    int lanes;
};
template <int E, int LANES>
Variant of_lanes(const RouteArgs &a)
{
    const int v = (a.experts + LANES - 1) / LANES;
    return {v <= 2   ? route_kernel<E, LANES, 2>
            : v <= 4 ? route_kernel<E, LANES, 4>
            : v <= 8 ? route_kernel<E, LANES, 8> : route_kernel<E, LANES, 16>,
            LANES};
}
// Lanes of a token: half a wavefront's, so that two tokens share its
// instructions, unless a lane's share of the experts is long and the tokens few:
// then the chain of a token's own steps counts. us of 64 and of 32 lanes, 8
// chosen: 256 experts 2048 tokens 8.1 and 8.5, 4096 11.6 and 10.5, 8192 18.7 and
// 14.9; one token 6.0 and 7.3; 64 experts, one token, 4.1 and 4.0.
template <int E>
Variant pick(const RouteArgs &a)
{
    if ((a.experts <= 128 || a.tokens > 2048) && a.experts <= 512 && a.top_k <= 32 && a.groups <= 32)
        return of_lanes<E, 32>(a);
    return of_lanes<E, 64>(a);
}

}  // namespace

hipError_t launch_route(const RouteArgs &args, hipStream_t stream)
{
    RouteArgs a = args;
    const Variant k = a.kind == kElemF32 ? pick<kF32>(a) : a.kind == kElemF16 ? pick<kF16>(a) : pick<kBF16>(a);
    const int tokens = kWaves * 64 / k.lanes, bytes = a.kind == kElemF32 ? 4 : 2;
    // Lanes of a group: a power of two, at most a row of 16, and all groups' within the token's.
    for (a.group_lanes = 16; a.group_lanes * a.groups > k.lanes; a.group_lanes /= 2)
        ;
    // expert / size for experts below 1024: size_inverse is less than 1 above 2^20 / size, so the quotient is
    // less than expert / 2^20 too large, which is below 1 / size (expert * size < 2^20): it reaches no next whole.
    const int size = a.experts / a.groups;
    a.size_inverse = ((1u << 20) + size - 1) / size;
    const size_t lds = a.groups > 1 ? (size_t)tokens * (a.experts + a.groups) * 8 : 0;
    const int64_t step = kMaxBlocksPerLaunch * tokens;
    for (int64_t t0 = 0; t0 < args.tokens; t0 += step) {
        a.logits = static_cast<const char *>(args.logits) + t0 * args.ld * bytes;
        a.ids = args.ids + t0 * args.top_k;
        a.weights = args.weights + t0 * args.top_k;
        a.tokens = args.tokens - t0 < step ? args.tokens - t0 : step;
        hipLaunchKernelGGL(k.kernel, dim3((unsigned)ceil_div(a.tokens, tokens)), dim3(64 * kWaves), lds, stream, a);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace w8a8
