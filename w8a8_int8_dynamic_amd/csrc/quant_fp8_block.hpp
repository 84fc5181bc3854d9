// Block-scaled quantization of rows: the work of one workgroup, and how rows are
// cut over workgroups (quant_fp8_block.hip; experts.hip runs it beside the plan
// of the experts' rows).
#pragma once

#include "fp8_block.hpp"
#include "fp8_block_rule.hpp"

namespace w8a8 {
namespace fp8_block {

// The row and first unit (8 elements; units of whole blocks) of this thread.
struct Place {
    int64_t row;
    int unit0;
    bool valid;
};
__device__ __forceinline__ Place place_of(int64_t b, int t, int64_t rows, int padded, int segs, int rpb, int per_block)
{
    Place p;
    if (rpb == 1) {
        p.row = b / segs;
        p.unit0 = (int)(b - p.row * segs) * per_block + t;
        p.valid = p.row < rows;
    } else {
        const int r = t / padded;
        p.row = b * rpb + r;
        p.unit0 = t - r * padded;
        p.valid = r < rpb && p.row < rows;
    }
    return p;
}

// Thread t of workgroup b of 256 threads, U units (8 elements) each.
template <int E, int U>
__device__ __forceinline__ void quant_block_rows(int64_t b, int t, const char *__restrict__ x, int64_t rows, int units,
                                                 int padded, int64_t ldx, uint8_t *__restrict__ q, int64_t ldq,
                                                 float *__restrict__ s, int64_t lds, int segs, int rpb)
{
    const Place p = place_of(b, t, rows, padded, segs, rpb, 256 * U);
    constexpr int BYTES = quant_rule::Elem<E>::BYTES;
    uint4 lo[U], hi[U];
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = p.unit0 + i * 256;
        lo[i] = hi[i] = make_uint4(0, 0, 0, 0);
        if (p.valid && u < units) {
            const uint4 *src = reinterpret_cast<const uint4 *>(x + (p.row * ldx + (int64_t)u * 8) * BYTES);
            if (E == kF32) {
                lo[i] = src[0];
                hi[i] = src[1];
            } else {
                const quant_rule::v4u v = __builtin_nontemporal_load(reinterpret_cast<const quant_rule::v4u *>(src));
                lo[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = p.unit0 + i * 256;
        float sc, inv;
        scale_of(row16_max(absmax8<E>(lo[i], hi[i])), sc, inv);
        if (p.valid && u < units) {
            *reinterpret_cast<uint2 *>(q + p.row * ldq + (int64_t)u * 8) = codes8<E>(lo[i], hi[i], inv);
            if ((u & 15) == 0)
                s[p.row * lds + (u >> 4)] = sc;
        }
    }
}

// How rows of `units` units (`padded` with those of the last block) are cut
// over workgroups of 256 threads with up to four units each: enough
// workgroups first (one unit a thread below about 1024 of them), then as few
// idle threads as four or three units leave.
struct Cut {
    int u, segs, rpb;
    int64_t blocks;
};
inline Cut cut_of(int64_t rows, int padded)
{
    Cut c;
    const int n = (int)ceil_div(padded, 256);
    if (padded <= 128) {
        c.u = 1;
        c.segs = 1;
        c.rpb = 256 / padded;
        c.blocks = ceil_div(rows, c.rpb);
        return c;
    }
    c.u = n <= 4 ? n : (round_up(n, 3) < round_up(n, 4) ? 3 : 4);
    if (rows * ceil_div(n, c.u) < 1024)
        c.u = 1;
    c.segs = (int)ceil_div(n, c.u);
    c.rpb = 1;
    c.blocks = rows * c.segs;
    return c;
}

}  // namespace fp8_block
}  // namespace w8a8
