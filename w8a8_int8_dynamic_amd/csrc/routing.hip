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
// One wavefront takes a token, its lanes V logits each.
#include "experts.hpp"
#include "quant_rule.hpp"

namespace w8a8 {
namespace {

using quant_rule::kBF16;
using quant_rule::kF16;
using quant_rule::kF32;

constexpr int kWaves = 4;        // tokens per workgroup

__device__ __forceinline__ double shfl_xor(double v, int m) { return __shfl_xor(v, m, 64); }

__device__ __forceinline__ double wave_sum(double v)
{
    for (int m = 1; m < 64; m *= 2)
        v += shfl_xor(v, m);
    return v;
}
__device__ __forceinline__ double wave_max(double v)
{
    for (int m = 1; m < 64; m *= 2)
        v = fmax(v, shfl_xor(v, m));
    return v;
}

template <int E>
__device__ __forceinline__ float load_logit(const void *p, int64_t i)
{
    if constexpr (E == kF32)
        return static_cast<const float *>(p)[i];
    const unsigned v = static_cast<const uint16_t *>(p)[i];
    return E == kF16 ? quant_rule::f16_to_float(v) : __uint_as_float(v << 16);
}

template <int E, int V>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(const RouteArgs a)
{
    __shared__ double choices[kWaves][64 * V];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t token = (int64_t)blockIdx.x * kWaves + wave;
    const bool live = token < a.tokens;                   // (every wave meets the barrier)
    constexpr double kOut = -__builtin_huge_val();

    // Expert v*64 + lane.
    double score[V], choice[V];
    double top = kOut;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        const int e = v * 64 + lane;
        const float x = live && e < a.experts ? load_logit<E>(a.logits, token * a.ld + e) : (float)kOut;
        score[v] = x != x ? kOut : (double)x;
        top = fmax(top, score[v]);
    }
    if (a.score == kScoreSoftmax) {
        top = wave_max(top);
        double sum = 0;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            choice[v] = score[v];
            // (infinite logits share the weight between them)
            score[v] = score[v] == top ? 1.0 : score[v] == kOut ? 0.0 : exp(score[v] - top);
            if (choice[v] == kOut)
                score[v] = 0.0;
            sum += score[v];
        }
        sum = wave_sum(sum);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            score[v] = sum > 0 ? score[v] / sum : 0.0;
            choice[v] = choice[v] == kOut ? kOut : score[v];
        }
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            choice[v] = score[v];
            score[v] = 1.0 / (1.0 + exp(-score[v]));
            choice[v] = choice[v] == kOut ? kOut : score[v];
        }
    }
    if (a.bias) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            const double b = e < a.experts ? (double)a.bias[e] : 0.0;
            choice[v] = choice[v] == kOut || b != b ? kOut : choice[v] + b;
        }
    }

    if (a.groups > 1) {
        const int size = a.experts / a.groups;
#pragma unroll
        for (int v = 0; v < V; ++v)
            choices[wave][v * 64 + lane] = choice[v];
        __syncthreads();
        // Lane g: the worth of group g.
        double first = kOut, second = kOut;
        if (lane < a.groups)
            for (int i = 0; i < size; ++i) {
                const double c = choices[wave][lane * size + i];
                second = fmax(second, fmin(first, c));
                first = fmax(first, c);
            }
        // (a group with one expert left is worth that one)
        const double worth = a.group_top == 2 && second != kOut ? first + second : first;
        int before = 0;
        for (int g = 0; g < a.groups; ++g) {
            const double w = __shfl(worth, g, 64);
            before += w > worth || (w == worth && g < lane);
        }
        const unsigned long long kept = __ballot(lane < a.groups && before < a.top_groups);
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int e = v * 64 + lane;
            if (e >= a.experts || !((kept >> (e / size)) & 1))
                choice[v] = kOut;
        }
    }

    // Lane j keeps the j-th choice.
    int my_id = -1;
    double my_score = 0.0, total = 0.0;
    for (int j = 0; j < a.top_k; ++j) {
        double best = kOut, s = 0.0;
        int id = 1 << 30;
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (choice[v] > best) {
                best = choice[v];
                id = v * 64 + lane;
                s = score[v];
            }
        for (int m = 1; m < 64; m *= 2) {
            const double b = shfl_xor(best, m), t = shfl_xor(s, m);
            const int i = __shfl_xor(id, m, 64);
            if (b > best || (b == best && i < id)) {
                best = b;
                id = i;
                s = t;
            }
        }
        if (best == kOut)
            break;
        total += s;
        if (lane == j) {
            my_id = id;
            my_score = s;
        }
#pragma unroll
        for (int v = 0; v < V; ++v)
            if (v * 64 + lane == id)
                choice[v] = kOut;
    }
    if (live && lane < a.top_k) {
        double w = my_score;
        if (a.renormalize)
            w = total > 0 ? w / total : 0.0;
        a.ids[token * a.top_k + lane] = my_id;
        a.weights[token * a.top_k + lane] = (float)(w * (double)a.scale);
    }
}

template <int E>
auto pick(int v)
{
    return v <= 1 ? route_kernel<E, 1> : v <= 2 ? route_kernel<E, 2> : v <= 4 ? route_kernel<E, 4>
         : v <= 8 ? route_kernel<E, 8> : route_kernel<E, 16>;
}

}  // namespace

hipError_t launch_route(const RouteArgs &args, hipStream_t stream)
{
    const int v = (int)ceil_div(args.experts, 64);
    auto fn = args.kind == kElemF32 ? pick<kF32>(v) : args.kind == kElemF16 ? pick<kF16>(v) : pick<kBF16>(v);
    const int bytes = args.kind == kElemF32 ? 4 : 2;
    const int64_t step = kMaxBlocksPerLaunch * kWaves;
    for (int64_t t0 = 0; t0 < args.tokens; t0 += step) {
        RouteArgs a = args;
        a.logits = static_cast<const char *>(args.logits) + t0 * args.ld * bytes;
        a.ids = args.ids + t0 * args.top_k;
        a.weights = args.weights + t0 * args.top_k;
        a.tokens = args.tokens - t0 < step ? args.tokens - t0 : step;
        hipLaunchKernelGGL(fn, dim3((unsigned)ceil_div(a.tokens, kWaves)), dim3(64 * kWaves), 0, stream, a);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace w8a8
