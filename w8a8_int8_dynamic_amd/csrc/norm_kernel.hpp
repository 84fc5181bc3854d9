// Norms around a quantized layer, on gfx950: the modulated norm in front of a
// block, and the gate, residual scale and norm behind it with the next block's
// norm in the same pass (NormRowsArgs in internal.hpp):
//   rms:   n(v) = v * rsqrt(mean(v^2) + eps)
//   layer: n(v) = (v - mean(v)) * rsqrt(mean((v - mean(v))^2) + eps)
//   next(v) = (n(v) * weight + bias) * (1 + scale) + shift
// All in fp32, with the variance taken around the mean in a second pass over
// the values; each output is rounded once, and the codes come from the fp32
// values by the rule of int8_quant_per_token / fp8_quant_per_token.
//
// What bounds it: the bytes of x, y, r and out; the arithmetic (some 20
// operations per element) and the vectors, which every row reads from L2,
// come next. norm_rows_kernel reads each row once and holds it in registers
// (8 * CH elements per thread) while its sums meet; TPR threads share a row.
// Rows too long for that take norm_rows_looped_kernel, one workgroup a row,
// which reads the row again (from L2) for each of its passes. Neither writes
// an element before it has read it for the last time, so r may be x itself.
// Measured on MI355X, bf16, from rotating buffers (median and range of a trace;
// a copy kernel makes 6.05 TB/s over 0.5 GB): M8192 K4096 layer norm with scale
// and shift 25.7 us (24.7-27.7; 5.2 TB/s); M8192 K12288 rms to e4m3 codes 58.3 us
// (56.0-61.7; 5.2); M8192 K4096 gated residual with post norm and next norm 44.4
// us (43.8-47.0; 6.0); M999 K5001 fp16 into an fp32 stream 15.1 us (13.2-15.8;
// 3.3: four rows to a workgroup); one row of 4096 to int8 codes 3.1 us.
#pragma once

#include <algorithm>

#include "norm_rows.hpp"

namespace w8a8 {
namespace {

using namespace norm_rule;

// ---- rows held in registers ----

// Sum of v over the WAVES wavefronts of a row, the same in each of them.
// `part` holds WAVES words twice, for one exchange and the next in turn: a
// wavefront can reach the next exchange's write only past this one's barrier,
// and the one after that only when every wavefront has read this one's words.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float *part, int &turn)
{
    v = wave_sum(v);
    if constexpr (WAVES == 1)
        return v;
    float *p = part + turn * WAVES;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
        p[threadIdx.x >> 6] = v;
    __syncthreads();
    float s[WAVES];
#pragma unroll
    for (int i = 0; i < WAVES; ++i)
        s[i] = p[i];
#pragma unroll
    for (int n = WAVES; n > 1; n = (n + 1) / 2)
#pragma unroll
        for (int i = 0; i < n / 2; ++i)
            s[i] += s[i + (n + 1) / 2];
    return s[0];
}

// The same for the largest of bit patterns.
template <int WAVES>
__device__ __forceinline__ u32 row_max(u32 m, float *part, int &turn)
{
    m = quant_rule::wave_max(m);
    if constexpr (WAVES == 1)
        return m;
    u32 *p = reinterpret_cast<u32 *>(part) + turn * WAVES;
    turn ^= 1;
    if ((threadIdx.x & 63) == 0)
        p[threadIdx.x >> 6] = m;
    __syncthreads();
    m = p[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i)
        m = max(m, p[i]);
    return m;
}

// A thread's piece of a row: 8 elements from `at` on, of which those from
// `skip` on are its own. Pieces begin at multiples of 8 and the row's last one
// ends with the row, so a ragged row's last piece reads over the piece before
// it; 8 or more: nothing is this thread's, and it reads what another does.
struct Piece {
    int at, skip;
    int own;                                           // bit j: element j is this thread's
};

// v where it is this thread's, else 0. (A bit of a register per element: eight
// comparisons a chunk would be held in more scalar registers than there are.)
template <bool WHOLE>
__device__ __forceinline__ float own_or_zero(const Piece &p, int j, float v)
{
    return WHOLE ? v : __int_as_float(__float_as_int(v) & __builtin_amdgcn_sbfe(p.own, j, 1));
}

// One 16-byte word of 16-bit elements, or two of fp32, still in their bits.
template <int E>
struct Raw {
    uint4 w[E == kF32 ? 2 : 1];
};
// Rows are read once: nontemporal loads keep them out of the caches' way
// (measured on MI355X: M8192 K8192 bf16, gated residual 82 -> 66 us).
__device__ __forceinline__ uint4 load16(const void *p)
{
    const v4u_any a = __builtin_nontemporal_load(static_cast<const v4u_any *>(p));
    return make_uint4(a[0], a[1], a[2], a[3]);
}
template <int E>
__device__ __forceinline__ Raw<E> raw_load(const char *row, int at)
{
    Raw<E> r;
    r.w[0] = load16(row + (int64_t)at * (E == kF32 ? 4 : 2));
    if constexpr (E == kF32)
        r.w[1] = load16(row + (int64_t)at * 4 + 16);
    return r;
}
template <int E>
__device__ __forceinline__ void raw_values(const uint4 &lo, const uint4 &hi, float (&v)[8])
{
    const u32 a[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = E == kF32 ? __uint_as_float(a[j])
             : E == kF16 ? quant_rule::f16_to_float(j & 1 ? a[j / 2] >> 16 : a[j / 2])
                         : __uint_as_float(j & 1 ? a[j / 2] & 0xffff0000u : a[j / 2] << 16);
}
template <int E>
__device__ __forceinline__ void raw_values(const Raw<E> &r, float (&v)[8])
{
    raw_values<E>(r.w[0], r.w[E == kF32 ? 1 : 0], v);
}

// One chunk of a vector of a norm or gate: its raw words, read without
// waiting, whatever its kind (uniform over the launch; a 16-bit vector's one
// word is read twice, and where there is no vector the row's own words are,
// unused). vec_values gives `none` where there is no vector.
struct RawVec {
    v4u_any lo, hi;
};
__device__ __forceinline__ RawVec vec_load(const void *p, int kind, int64_t offset, int at, const char *otherwise)
{
    const int size = kind == kF32 ? 4 : 2;
    const char *s = p ? static_cast<const char *>(p) + (offset + at) * size : otherwise;
    RawVec r;
    r.lo = *reinterpret_cast<const v4u_any *>(s);
    r.hi = *reinterpret_cast<const v4u_any *>(s + (p && kind == kF32 ? 16 : 0));
    return r;
}
__device__ __forceinline__ void vec_values(const void *p, int kind, const RawVec &r, float none, float (&v)[8])
{
    const uint4 lo = make_uint4(r.lo[0], r.lo[1], r.lo[2], r.lo[3]);
    const uint4 hi = make_uint4(r.hi[0], r.hi[1], r.hi[2], r.hi[3]);
    if (p == nullptr) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = none;
    } else if (kind == kF32) {
        raw_values<kF32>(lo, hi, v);
    } else if (kind == kF16) {
        raw_values<kF16>(lo, hi, v);
    } else {
        raw_values<kBF16>(lo, hi, v);
    }
}

// v = n(v) for the row's values held as v[CH][8]; elements that are not this
// thread's are left out of the sums.
template <int CH, int WAVES, bool WHOLE>
__device__ __forceinline__ void normalize(float (&v)[CH][8], const Piece (&p)[CH], float k_inv, int kind, float eps,
                                          float *part, int &turn)
{
    if (kind == kNormLayer) {
        float s = 0.0f;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += own_or_zero<WHOLE>(p[c], j, v[c][j]);
        const float mean = row_sum<WAVES>(s, part, turn) * k_inv;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                v[c][j] -= mean;
    }
    float q = 0.0f;
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = own_or_zero<WHOLE>(p[c], j, v[c][j]);
            q = fmaf(d, d, q);
        }
    const float inv = rsqrt_of(row_sum<WAVES>(q, part, turn) * k_inv + eps);
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[c][j] *= inv;
}

// A piece of a row to memory: whole, or its own elements one by one.
// A norm's own output needs no such care: pieces that share elements hold the
// same values there, bit for bit, so each is stored whole (NormRowsArgs.r may be
// x, where a piece may have read its neighbour's result). Stores that no
// branch skips can be counted, and the next row's elements waited for alone.
template <int E, bool WHOLE>
__device__ __forceinline__ void piece_store(char *row, const Piece &p, const float (&v)[8])
{
    if (WHOLE || p.skip == 0) {
        store8<E>(row, p.at, p.at + 8, v);
        return;
    }
#pragma unroll
    for (int j = 1; j < 8; ++j)
        if (j >= p.skip) {
            if constexpr (E == kF32)
                reinterpret_cast<float *>(row)[p.at + j] = v[j];
            else
                reinterpret_cast<uint16_t *>(row)[p.at + j] = (uint16_t)pack2<E>(v[j], v[j]);
        }
}

// TPR threads (whole wavefronts) per row, R rows at a time per workgroup, which
// takes a run of `per_block` rows. The vectors are read once for all of a
// run's rows in one group and held as the two factors of each norm:
//   r = residual_scale * x + n(y) * g1 + g0,  g1 = branch_scale * gate * weight
//   h = n(r) * h1 + h0,  h1 = weight * (1 + scale), h0 = bias * (1 + scale) + shift
// and the next row's elements are on their way while a row's sums meet.
// WHOLE: K is exactly the TPR * CH pieces of 8. OUT: what becomes of h (kOut*),
// a template argument so that the loop's loads and stores are the same in every
// pass: the wait for the next row's elements then leaves this row's stores in
// flight.
constexpr int kOutNone = 0, kOutFloat = 1, kOutCodes = 2;
// HOLD: the factors stay in registers for the run; otherwise each row makes
// them again, chunk by chunk.
template <int XE, int AE, bool RES, int OUT, int CH, int TPR, int R, bool WHOLE, bool HOLD>
__global__ __launch_bounds__(TPR * R) void norm_rows_kernel(const NormRowsArgs a, int64_t per_block)
{
    constexpr int WAVES = TPR / 64;
    static_assert(R == 1 || WAVES == 1, "rows that share a workgroup do not share barriers");
    constexpr int XB = XE == kF32 ? 4 : 2;
    __shared__ float part[2 * WAVES];
    const int t = (int)threadIdx.x % TPR;
    const int K = (int)a.K;
    const float k_inv = 1.0f / (float)K;
    Piece p[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        const int begin = (c * TPR + t) * 8;
        p[c].at = min(begin, K - 8);
        p[c].skip = begin - p[c].at;
        p[c].own = p[c].skip < 8 ? 0xff & (0xff << p[c].skip) : 0;
    }
    const int64_t first = (int64_t)blockIdx.x * per_block +
                          (R > 1 ? __builtin_amdgcn_readfirstlane((int)threadIdx.x / TPR) : 0);
    const int64_t end = min(a.rows, ((int64_t)blockIdx.x + 1) * per_block);
    if (first >= end)
        return;                                        // whole wavefronts that share no barrier (R > 1), or none
    constexpr bool next = OUT != kOutNone;

    Raw<XE> xr[CH];                                    // the next row
    Raw<AE> yr[RES ? CH : 1];
    auto fetch = [&](int64_t row) __attribute__((always_inline)) {
        const char *x = static_cast<const char *>(a.x) + row * a.ldx * XB;
#pragma unroll
        for (int c = 0; c < CH; ++c)
            xr[c] = raw_load<XE>(x, p[c].at);
        if constexpr (RES) {
            const char *y = static_cast<const char *>(a.y) + row * a.ldy * 2;
#pragma unroll
            for (int c = 0; c < CH; ++c)
                yr[c] = raw_load<AE>(y, p[c].at);
        }
    };
    fetch(first);

    float g1[HOLD ? CH : 1][8], g0[HOLD ? CH : 1][8], h1[HOLD ? CH : 1][8], h0[HOLD ? CH : 1][8];
    int64_t gg = 0, ng = 0;                            // the row's groups of the gate and of the next norm
    int turn = 0;
    int64_t row = first, stop = first;                 // the rows before `stop` share the vectors held
    const int64_t last = first + (end - 1 - first) / R * R;
    // Chunk C's factors of the residual (G) and of the next norm (N), all loads
    // before the first wait.
    const void *pw = RES && a.post.kind != kNormNone ? a.post.weight : nullptr;
    const void *pb = RES && a.post.kind != kNormNone ? a.post.bias : nullptr;
    auto factors = [&](auto G, auto N, auto C, float (&c1)[8], float (&c0)[8], float (&d1)[8], float (&d0)[8])
                       __attribute__((always_inline)) {
        constexpr bool gate = RES && decltype(G)::value, norm = next && decltype(N)::value;
        const int at = p[decltype(C)::value].at;
        const char *x = static_cast<const char *>(a.x) + row * a.ldx * XB + (int64_t)at * XB;
        RawVec vg, vpw, vpb, vw, vb, vs, vt;
        if constexpr (gate) {
            vg = vec_load(a.gate, a.gate_kind, gg * a.ld_gate, at, x);
            vpw = vec_load(pw, a.post.vec_kind, 0, at, x);
            vpb = vec_load(pb, a.post.vec_kind, 0, at, x);
        }
        if constexpr (norm) {
            vw = vec_load(a.next.weight, a.next.vec_kind, 0, at, x);
            vb = vec_load(a.next.bias, a.next.vec_kind, 0, at, x);
            vs = vec_load(a.next.scale, a.next.mod_kind, ng * a.next.ld_scale, at, x);
            vt = vec_load(a.next.shift, a.next.mod_kind, ng * a.next.ld_shift, at, x);
        }
        if constexpr (gate) {
            float w[8], b[8];
            vec_values(a.gate, a.gate_kind, vg, 1.0f, c1);
            vec_values(pw, a.post.vec_kind, vpw, 1.0f, w);
            vec_values(pb, a.post.vec_kind, vpb, 0.0f, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float g = a.branch_scale * c1[j];
                c1[j] = g * w[j];
                c0[j] = g * b[j];
            }
        }
        if constexpr (norm) {
            float sc[8], sh[8];
            vec_values(a.next.weight, a.next.vec_kind, vw, 1.0f, d1);
            vec_values(a.next.bias, a.next.vec_kind, vb, 0.0f, d0);
            vec_values(a.next.scale, a.next.mod_kind, vs, 0.0f, sc);
            vec_values(a.next.shift, a.next.mod_kind, vt, 0.0f, sh);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                d1[j] = d1[j] * (1.0f + sc[j]);
                d0[j] = fmaf(d0[j], 1.0f + sc[j], sh[j]);
            }
        }
    };
    using Yes = std::integral_constant<bool, true>;
    using No = std::integral_constant<bool, false>;
    auto vectors = [&]() __attribute__((always_inline)) {
        stop = end;
        if (RES && a.gate) {
            gg = (uint32_t)row / (uint32_t)a.gate_rows;
            stop = min(stop, (gg + 1) * a.gate_rows);
        }
        if (next && (a.next.scale || a.next.shift)) {
            ng = (uint32_t)row / (uint32_t)a.next.group_rows;
            stop = min(stop, (ng + 1) * a.next.group_rows);
        }
        if constexpr (HOLD)
            static_for<CH>([&](auto C) __attribute__((always_inline)) {
                constexpr int c = decltype(C)::value;
                factors(Yes{}, Yes{}, C, g1[c], g0[c], h1[c], h0[c]);
            });
    };
    auto one_row = [&]() __attribute__((always_inline)) {
        float v[CH][8], b[RES ? CH : 1][8];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            raw_values<XE>(xr[c], v[c]);
            if constexpr (RES)
                raw_values<AE>(yr[c], b[c]);
        }
        // The next row into the registers that this one's words leave (the last
        // row once more at the end of the run: a load that nothing waits for).
        __builtin_amdgcn_sched_barrier(0);
        fetch(min(row + R, last));
        if constexpr (RES) {
            if (a.post.kind != kNormNone)
                normalize<CH, WAVES, WHOLE>(b, p, k_inv, a.post.kind, a.post.eps, part, turn);
            static_for<CH>([&](auto C) __attribute__((always_inline)) {
                constexpr int c = decltype(C)::value, k = HOLD ? c : 0;
                if constexpr (!HOLD)
                    factors(Yes{}, No{}, C, g1[0], g0[0], h1[0], h0[0]);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[c][j] = fmaf(b[c][j], g1[k][j], fmaf(a.residual_scale, v[c][j], g0[k][j]));
                if (WHOLE || p[c].skip < 8)
                    piece_store<XE, WHOLE>(static_cast<char *>(a.r) + row * a.ldr * XB, p[c], v[c]);
            });
            if constexpr (!next)
                return;
        }
        normalize<CH, WAVES, WHOLE>(v, p, k_inv, a.next.kind, a.next.eps, part, turn);
        u32 m = 0;
        static_for<CH>([&](auto C) __attribute__((always_inline)) {
            constexpr int c = decltype(C)::value, k = HOLD ? c : 0;
            if constexpr (!HOLD)
                factors(No{}, Yes{}, C, g1[0], g0[0], h1[0], h0[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[c][j] = fmaf(v[c][j], h1[k][j], h0[k][j]);
                if constexpr (OUT == kOutCodes)
                    m = max(m, __float_as_uint(own_or_zero<WHOLE>(p[c], j, v[c][j])) & 0x7fffffffu);
            }
            if constexpr (OUT == kOutFloat && !RES)
                store8<AE>(static_cast<char *>(a.out) + row * a.ldo * 2, p[c].at, p[c].at + 8, v[c]);
            else if (OUT == kOutFloat && (WHOLE || p[c].skip < 8))
                piece_store<AE, WHOLE>(static_cast<char *>(a.out) + row * a.ldo * 2, p[c], v[c]);
        });
        if constexpr (OUT != kOutCodes)
            return;
        float sc, inv;
        quant_rule::scale_of(row_max<WAVES>(m, part, turn), kF32, sc, inv, a.out_kind == kNormOutFp8);
        if (t == 0)
            a.out_scale[row] = sc;
        uint8_t *q = static_cast<uint8_t *>(a.out) + row * a.ldo;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            u32 lo, hi;
            if (a.out_kind == kNormOutFp8) {
                lo = quant_rule::codes4_fp8(v[c][0], v[c][1], v[c][2], v[c][3], inv);
                hi = quant_rule::codes4_fp8(v[c][4], v[c][5], v[c][6], v[c][7], inv);
            } else {
                lo = quant_rule::codes4_i8(v[c][0], v[c][1], v[c][2], v[c][3], inv);
                hi = quant_rule::codes4_i8(v[c][4], v[c][5], v[c][6], v[c][7], inv);
            }
            if constexpr (!RES && !WHOLE) {
                *reinterpret_cast<v2u_any *>(q + p[c].at) = v2u_any{lo, hi};
            } else if (WHOLE || p[c].skip == 0) {
                *reinterpret_cast<uint2 *>(q + p[c].at) = make_uint2(lo, hi);
            } else {
#pragma unroll
                for (int j = 1; j < 8; ++j)
                    if (j >= p[c].skip)
                        q[p[c].at + j] = (uint8_t)((j < 4 ? lo >> (8 * j) : hi >> (8 * (j - 4))) & 0xffu);
            }
        }
    };
    while (row < end) {
        vectors();
        do {
            one_row();
            row += R;
        } while (row < stop);
    }
}

// ---- rows of any length, read again for each pass ----

__device__ __forceinline__ float block_sum(float v, float *part)
{
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0)
        part[threadIdx.x >> 6] = v;
    __syncthreads();
    return (part[0] + part[1]) + (part[2] + part[3]);
}

// Mean (0 for rms) and reciprocal deviation of the K values that `value`
// yields, 8 at a time.
template <class F>
__device__ __forceinline__ void stats(F &&value, int64_t K, int kind, float eps, float *part, float &mean, float &inv)
{
    mean = 0.0f;
    if (kind == kNormLayer) {
        float s = 0.0f;
        for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
            float v[8];
            value(e, v);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                s += e + j < K ? v[j] : 0.0f;
        }
        mean = block_sum(s, part) / (float)K;
    }
    float q = 0.0f;
    for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
        float v[8];
        value(e, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float d = e + j < K ? v[j] - mean : 0.0f;
            q += d * d;
        }
    }
    inv = 1.0f / sqrtf(block_sum(q, part) / (float)K + eps);
}

// (v - mean) * inv * weight + bias, then * (1 + scale) + shift.
__device__ __forceinline__ void apply(const NormVectors &n, int64_t row, int64_t e, int64_t K, float mean, float inv,
                                      float (&v)[8])
{
    float t[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        v[j] = (v[j] - mean) * inv;
    if (n.weight) {
        load8(n.weight, n.vec_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= t[j];
    }
    if (n.bias) {
        load8(n.bias, n.vec_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] += t[j];
    }
    const int64_t g = n.scale || n.shift ? row / n.group_rows : 0;
    const int bytes = n.mod_kind == kF32 ? 4 : 2;
    if (n.scale) {
        load8(static_cast<const char *>(n.scale) + g * n.ld_scale * bytes, n.mod_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] *= 1.0f + t[j];
    }
    if (n.shift) {
        load8(static_cast<const char *>(n.shift) + g * n.ld_shift * bytes, n.mod_kind, e, K, t);
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] += t[j];
    }
}

template <int XE, int AE, bool RES>
__global__ __launch_bounds__(256) void norm_rows_looped_kernel(const NormRowsArgs a)
{
    __shared__ float part[4];
    __shared__ u32 most;
    const int64_t K = a.K;
    constexpr int XB = XE == kF32 ? 4 : 2;
    for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
        const char *x = static_cast<const char *>(a.x) + row * a.ldx * XB;
        const char *y = RES ? static_cast<const char *>(a.y) + row * a.ldy * 2 : nullptr;
        const char *gate = nullptr;
        if (RES && a.gate)
            gate = static_cast<const char *>(a.gate) + row / a.gate_rows * a.ld_gate * (a.gate_kind == kF32 ? 4 : 2);
        float pmean = 0.0f, pinv = 1.0f;
        if (RES && a.post.kind != kNormNone)
            stats([&](int64_t e, float (&v)[8]) { load8<AE>(y, e, K, v); }, K, a.post.kind, a.post.eps, part, pmean,
                  pinv);
        auto value = [&](int64_t e, float (&v)[8]) {
            load8<XE>(x, e, K, v);
            if constexpr (RES) {
                float b[8];
                load8<AE>(y, e, K, b);
                if (a.post.kind != kNormNone)
                    apply(a.post, row, e, K, pmean, pinv, b);
                if (gate) {
                    float t[8];
                    load8(gate, a.gate_kind, e, K, t);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        b[j] *= t[j];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[j] = a.residual_scale * v[j] + a.branch_scale * b[j];
            }
        };
        float mean = 0.0f, inv = 1.0f;
        const bool next = a.next.kind != kNormNone;
        if (next)
            stats(value, K, a.next.kind, a.next.eps, part, mean, inv);
        // Largest |h| as its bit pattern (which orders NaN above infinity).
        float sc = 0.0f, cinv = 0.0f;
        if (next && a.out_kind != kNormOut16) {
            u32 m = 0;
            for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
                float v[8];
                value(e, v);
                apply(a.next, row, e, K, mean, inv, v);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    m = max(m, e + j < K ? __float_as_uint(v[j]) & 0x7fffffffu : 0u);
            }
            m = quant_rule::wave_max(m);
            if (threadIdx.x == 0)
                most = 0;
            __syncthreads();
            if ((threadIdx.x & 63) == 0)
                atomicMax(&most, m);
            __syncthreads();
            m = most;
            quant_rule::scale_of(m, kF32, sc, cinv, a.out_kind == kNormOutFp8);
            if (threadIdx.x == 0)
                a.out_scale[row] = sc;
        }
        for (int64_t e = (int64_t)threadIdx.x * 8; e < K; e += 256 * 8) {
            float v[8];
            value(e, v);
            if (RES)
                store8<XE>(static_cast<char *>(a.r) + row * a.ldr * XB, e, K, v);
            if (!next)
                continue;
            apply(a.next, row, e, K, mean, inv, v);
            if (a.out_kind == kNormOut16) {
                store8<AE>(static_cast<char *>(a.out) + row * a.ldo * 2, e, K, v);
            } else {
                u32 lo, hi;
                if (a.out_kind == kNormOutFp8) {
                    lo = quant_rule::codes4_fp8(v[0], v[1], v[2], v[3], cinv);
                    hi = quant_rule::codes4_fp8(v[4], v[5], v[6], v[7], cinv);
                } else {
                    lo = quant_rule::codes4_i8(v[0], v[1], v[2], v[3], cinv);
                    hi = quant_rule::codes4_i8(v[4], v[5], v[6], v[7], cinv);
                }
                quant_rule::store_codes<kBF16, false>(static_cast<int8_t *>(a.out) + row * a.ldo, e, (int)K, lo, hi);
            }
        }
        __syncthreads();                               // part and most are free again
    }
}

typedef void (*RowsFn)(const NormRowsArgs, int64_t);
struct Shape {
    RowsFn fn;
    int threads, rows;                                 // per workgroup; rows at a time
    int per_cu;                                        // workgroups a CU holds
};

// The row shapes of norm_rows_kernel: threads per row and chunks per thread,
// up to 16384 elements (beyond, a row and its vectors no longer fit the
// registers of one workgroup; M4096 K16000 in passes takes 1.4 to 1.8 times as
// long).
constexpr int64_t kHeldElements = 16384;
template <int XE, int AE, bool RES, int OUT, int CH, int TPR, int R, bool HOLD = true>
Shape shape(int64_t K)
{
    static_assert(TPR * R <= (CH > 2 ? 512 : 1024), "a workgroup fits its share of a CU");
    return {K == CH * TPR * 8 ? norm_rows_kernel<XE, AE, RES, OUT, CH, TPR, R, true, HOLD>
                              : norm_rows_kernel<XE, AE, RES, OUT, CH, TPR, R, false, HOLD>, TPR * R, R,
            (CH > 2 ? 512 : 1024) / (TPR * R)};
}
// One chunk per thread as far as 1024 threads reach, where a thread has the
// words of two tensors and the vectors of two norms to hold, or where rows are
// few and their latency counts; two otherwise, for more rows in flight. In
// between, the thread counts leave at most a third of the threads without
// elements.
// Measured on MI355X, bf16: two chunks against one, M8192 K4096, gated residual
// with post norm and next norm 48.9 against 45.1 us, norm to int8 codes 24.0
// against 28.9 us, the same of one row 3.5 against 3.2 us; M4096 K6000, the
// gated residual on 768 threads 37.1, on 1024 44.5 us.
constexpr int64_t kFewRows = 512;
// Both norms of a row of two chunks on 1024 threads do not fit the registers:
// many rows are faster with some of the factors spilled, few with all of them
// read again (measured on MI355X, K16384 bf16, read again against held: 64 rows
// 10.8 against 18.1 us, 256 rows 13.2 against 33.4, 999 rows 47.0 against 48.7,
// 2000 rows 86.5 against 68.8).
constexpr int64_t kReadAgainRows = 1024;
template <int XE, int AE, bool RES, int OUT>
Shape pick(int64_t rows, int64_t K)
{
    const int64_t chunks = ceil_div(K, 8);
    if (chunks <= 64)
        return shape<XE, AE, RES, OUT, 1, 64, 4>(K);
    if (chunks <= 128)
        return shape<XE, AE, RES, OUT, 1, 128, 1>(K);
    if (chunks <= 192)
        return shape<XE, AE, RES, OUT, 1, 192, 1>(K);
    if (chunks <= 256)
        return shape<XE, AE, RES, OUT, 1, 256, 1>(K);
    if (RES || rows <= kFewRows) {
        if (chunks <= 384)
            return shape<XE, AE, RES, OUT, 1, 384, 1>(K);
        if (chunks <= 512)
            return shape<XE, AE, RES, OUT, 1, 512, 1>(K);
        if (chunks <= 640)
            return shape<XE, AE, RES, OUT, 1, 640, 1>(K);
        if (chunks <= 768)
            return shape<XE, AE, RES, OUT, 1, 768, 1>(K);
        if (chunks <= 1024)
            return shape<XE, AE, RES, OUT, 1, 1024, 1>(K);
    } else {
        if (chunks <= 384)
            return shape<XE, AE, false, OUT, 2, 192, 1>(K);
        if (chunks <= 512)
            return shape<XE, AE, false, OUT, 2, 256, 1>(K);
        if (chunks <= 768)
            return shape<XE, AE, false, OUT, 2, 384, 1>(K);
        if (chunks <= 1024)
            return shape<XE, AE, false, OUT, 2, 512, 1>(K);
    }
    if (chunks <= 1280)
        return shape<XE, AE, RES, OUT, 2, 640, 1>(K);
    if (chunks <= 1536)
        return shape<XE, AE, RES, OUT, 3, 512, 1>(K);
    if constexpr (RES && OUT != kOutNone)
        if (rows <= kReadAgainRows)
            return shape<XE, AE, RES, OUT, 2, 1024, 1, false>(K);
    return shape<XE, AE, RES, OUT, 2, 1024, 1>(K);
}

template <int XE, int AE>
hipError_t launch(const NormRowsArgs &a, hipStream_t stream)
{
    const bool res = a.y != nullptr;
    if (a.K < 8 || a.K > kHeldElements) {
        const int64_t blocks = std::min(a.rows, kMaxBlocksPerLaunch);
        auto fn = res ? norm_rows_looped_kernel<XE, AE, true> : norm_rows_looped_kernel<XE, AE, false>;
        hipLaunchKernelGGL(fn, dim3((unsigned)blocks), dim3(256), 0, stream, a);
        return hipGetLastError();
    }
    const bool codes = a.out_kind != kNormOut16;
    const Shape s = !res ? (codes ? pick<XE, AE, false, kOutCodes>(a.rows, a.K) : pick<XE, AE, false, kOutFloat>(a.rows, a.K))
                  : a.next.kind == kNormNone ? pick<XE, AE, true, kOutNone>(a.rows, a.K)
                  : codes ? pick<XE, AE, true, kOutCodes>(a.rows, a.K) : pick<XE, AE, true, kOutFloat>(a.rows, a.K);
    // A run of rows per workgroup, as long as every CU has its workgroups: each
    // run pays for its vectors once (measured on MI355X, twice as many
    // workgroups cost 5 to 30 % from 600 rows on).
    const int64_t want = 256 * s.per_cu;
    const int64_t per_block = round_up(ceil_div(a.rows, want), s.rows);
    hipLaunchKernelGGL(s.fn, dim3((unsigned)ceil_div(a.rows, per_block)), dim3(s.threads), 0, stream, a, per_block);
    return hipGetLastError();
}

}  // namespace
}  // namespace w8a8
