// Microscaled 4-bit (MX FP4) quantization, its inverse and the weight repack,
// on gfx950. The rule is fp4_rule.hpp's; nothing here reduces over more than
// 32 elements, so every step streams.
//
// quant_blocks_kernel (HBM-bound: 2 bytes read and 17/32 written per 16-bit
// element): four neighbouring lanes share a block of 32, 8 elements each, so
// a wavefront's loads are contiguous (16 bytes a lane), two quad exchanges
// give the block's maximum, and its 4-byte code words and 16 scale bytes are
// contiguous too. A workgroup takes U x 256 such units of one row, or
// several whole rows where a row is shorter than that. 16-bit rows pass the
// caches by (nontemporal; an fp32 lane's two words share lines, where that
// costs 5 %); the codes stay in them for the matmul. Measured on MI355X,
// M8192 K12288 bf16 from rotating buffers: 40.6 us, 6.3 TB/s; back to bf16
// 37.4 us, 6.8 TB/s; fp32 109.8 us, 4.1 TB/s, and back to fp32 110.7 us.
#include <algorithm>

#include "fp4_rule.hpp"
#include "internal.hpp"

namespace w8a8 {
namespace {

using namespace fp4_rule;

__device__ __forceinline__ u32 quad_max(u32 v)
{
    v = max(v, (u32)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false));
    return max(v, (u32)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, false));
}

// The rows and units (8 elements) that this thread takes: unit0, unit0 + 256,
// ... (U of them) of row. Rows of at least 256 units are cut into segs
// segments; of shorter ones a workgroup takes rpb whole rows.
struct Place {
    int64_t row;
    int unit0;
    bool valid;
};
__device__ __forceinline__ Place place_of(int64_t b, int64_t rows, int units, int segs, int rpb, int per_block)
{
    Place p;
    if (rpb == 1) {
        p.row = b / segs;
        p.unit0 = (int)(b - p.row * segs) * per_block + (int)threadIdx.x;
        p.valid = p.row < rows;
    } else {
        const int r = (int)threadIdx.x / units;
        p.row = b * rpb + r;
        p.unit0 = (int)threadIdx.x - r * units;
        p.valid = r < rpb && p.row < rows;
    }
    return p;
}

template <int E, int U>
__global__ __launch_bounds__(256) void quant_blocks_kernel(const char *__restrict__ x, int64_t rows, int units,
                                                           int64_t ldx, uint8_t *__restrict__ q, int64_t ldq,
                                                           uint8_t *__restrict__ s, int64_t lds, int segs,
                                                           int rpb)
{
    const Place p = place_of(blockIdx.x, rows, units, segs, rpb, 256 * U);
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
                const quant_rule::v4u t = __builtin_nontemporal_load(reinterpret_cast<const quant_rule::v4u *>(src));
                lo[i] = make_uint4(t[0], t[1], t[2], t[3]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = p.unit0 + i * 256;
        // units is a multiple of 4 and unit0's quad is whole, so the four
        // lanes of a block are all valid or all idle.
        const u32 byte = scale_byte(quad_max(absmax8<E>(lo[i], hi[i])));
        if (p.valid && u < units) {
            *reinterpret_cast<u32 *>(q + p.row * ldq + (int64_t)u * 4) = codes8<E>(lo[i], hi[i], byte);
            if ((u & 3) == 0)
                s[p.row * lds + (u >> 2)] = (uint8_t)byte;
        }
    }
}

// 8 codes a thread back to their values, rounded to the output's type.
template <int E, int U>
__global__ __launch_bounds__(256) void dequant_blocks_kernel(const uint8_t *__restrict__ q, int64_t ldq,
                                                             const uint8_t *__restrict__ s, int64_t lds,
                                                             int64_t rows, int units, char *__restrict__ out,
                                                             int64_t ldo, int segs, int rpb)
{
    const Place p = place_of(blockIdx.x, rows, units, segs, rpb, 256 * U);
    constexpr int BYTES = quant_rule::Elem<E>::BYTES;
    if (!p.valid)
        return;
#pragma unroll
    for (int i = 0; i < U; ++i) {
        const int u = p.unit0 + i * 256;
        if (u >= units)
            break;
        const u32 w = *reinterpret_cast<const u32 *>(q + p.row * ldq + (int64_t)u * 4);
        const u32 byte = s[p.row * lds + (u >> 2)];
        const float sc = byte == 255u ? __uint_as_float(0x7fc00000u) : scale_value(byte);
        float v[8];
#pragma unroll
        for (int j = 0; j < 8; ++j)
            v[j] = code_value(w >> (4 * j), sc);
        uint4 *dst = reinterpret_cast<uint4 *>(out + (p.row * ldo + (int64_t)u * 8) * BYTES);
        if constexpr (E == kF32) {
            dst[0] = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]),
                                __float_as_uint(v[3]));
            dst[1] = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]),
                                __float_as_uint(v[7]));
        } else {
            u32 o[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                typedef float f32x2 __attribute__((ext_vector_type(2)));
                const f32x2 pair = {v[2 * j], v[2 * j + 1]};
                if constexpr (E == kF16)
                    o[j] = __builtin_bit_cast(u32, __builtin_convertvector(pair, f16x2));
                else
                    o[j] = __builtin_bit_cast(u32, __builtin_convertvector(pair, bf16x2));
            }
            __builtin_nontemporal_store(quant_rule::v4u{o[0], o[1], o[2], o[3]},
                                        reinterpret_cast<quant_rule::v4u *>(dst));
        }
    }
}

// Weight repack: one 16-byte unit (32 codes, one block) of a fragment per
// thread. Fragment F[nb][kb] is int8_prepack_weight's over the code bytes:
// byte 16*l + j is byte 64*kb + 16*(l/16) + j of channel 16*nb + l%16, which
// is block 4*kb + l/16. Scales: byte 256*(nb*chunks + c) + 16*r + j is block
// 16*c + j of channel 16*nb + r. Outside the weight: codes 0, scale byte 127.
// SRC: -1 codes and scale bytes made before, else the element kind to
// quantize from.
template <int SRC>
__global__ __launch_bounds__(256) void prepack_fp4_kernel(const char *__restrict__ w, int64_t ldw,
                                                          const uint8_t *__restrict__ ws, int64_t lds, int N,
                                                          int blocks, int kblocks, uint4 *__restrict__ packed,
                                                          uint8_t *__restrict__ spacked, int64_t units, int64_t u0)
{
    const int64_t u = u0 + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= units)
        return;
    const int lane = (int)(u & 63);
    const int64_t frag = u >> 6;
    const int64_t nb = frag / kblocks;
    const int kb = (int)(frag - nb * kblocks);
    const int64_t n = nb * 16 + (lane & 15);
    const int b = kb * 4 + (lane >> 4);
    uint4 c = make_uint4(0, 0, 0, 0);
    u32 byte = 127;
    if (n < N && b < blocks) {
        if constexpr (SRC < 0) {
            const uint8_t *src = reinterpret_cast<const uint8_t *>(w) + n * ldw + (int64_t)b * 16;
            u32 o[4] = {0, 0, 0, 0};
            for (int j = 0; j < 16; ++j)
                o[j >> 2] |= (u32)src[j] << (8 * (j & 3));
            c = make_uint4(o[0], o[1], o[2], o[3]);
            byte = ws[n * lds + b];
        } else {
            constexpr int PER = SRC == kF32 ? 2 : 1;         // 16-byte words per 8 elements
            const uint4 *src = reinterpret_cast<const uint4 *>(
                w + (n * ldw + (int64_t)b * kBlock) * quant_rule::Elem<SRC>::BYTES);
            uint4 v[4 * PER];
            u32 m = 0;
#pragma unroll
            for (int i = 0; i < 4 * PER; ++i)
                v[i] = src[i];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                m = max(m, absmax8<SRC>(v[i * PER], v[i * PER + PER - 1]));
            byte = scale_byte(m);
            c.x = codes8<SRC>(v[0], v[PER - 1], byte);
            c.y = codes8<SRC>(v[PER], v[2 * PER - 1], byte);
            c.z = codes8<SRC>(v[2 * PER], v[3 * PER - 1], byte);
            c.w = codes8<SRC>(v[3 * PER], v[4 * PER - 1], byte);
        }
    }
    packed[u] = c;
    const int chunks = (kblocks + 3) / 4;
    const int64_t at = (nb * chunks + kb / 4) * 256 + (lane & 15) * 16;
    spacked[at + (kb & 3) * 4 + (lane >> 4)] = (uint8_t)byte;
    if (kb == kblocks - 1)                                   // the rest of the last chunk
        for (int k = (kb & 3) + 1; k < 4; ++k)
            spacked[at + k * 4 + (lane >> 4)] = 127;
}

__global__ __launch_bounds__(256) void unpack_fp4_kernel(const uint4 *__restrict__ packed,
                                                         const uint8_t *__restrict__ spacked, int N, int blocks,
                                                         int kblocks, uint8_t *__restrict__ wq, int64_t ldw,
                                                         uint8_t *__restrict__ ws, int64_t lds, int64_t units,
                                                         int64_t u0)
{
    const int64_t u = u0 + (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (u >= units)
        return;
    const int lane = (int)(u & 63);
    const int64_t frag = u >> 6;
    const int64_t nb = frag / kblocks;
    const int kb = (int)(frag - nb * kblocks);
    const int64_t n = nb * 16 + (lane & 15);
    const int b = kb * 4 + (lane >> 4);
    if (n >= N || b >= blocks)
        return;
    const uint4 v = packed[u];
    const u32 o[4] = {v.x, v.y, v.z, v.w};
    uint8_t *dst = wq + n * ldw + (int64_t)b * 16;
    for (int j = 0; j < 16; ++j)
        dst[j] = (uint8_t)(o[j >> 2] >> (8 * (j & 3)));
    const int chunks = (kblocks + 3) / 4;
    ws[n * lds + b] = spacked[(nb * chunks + kb / 4) * 256 + (lane & 15) * 16 + (kb & 3) * 4 + (lane >> 4)];
}

// How rows of `units` units are cut over workgroups of 256 threads with up to
// four units each: enough workgroups first (one unit a thread below about
// 1024 of them), then as few idle threads as four or three units leave.
struct Cut {
    int u, segs, rpb;
    int64_t blocks;
};
Cut cut_of(int64_t rows, int units)
{
    Cut c;
    const int n = (int)ceil_div(units, 256);
    if (units < 256) {
        c.u = 1;
        c.segs = 1;
        c.rpb = 256 / units;
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

template <int E>
auto quant_pick(int u)
{
    return u == 1 ? quant_blocks_kernel<E, 1> : u == 2 ? quant_blocks_kernel<E, 2>
         : u == 3 ? quant_blocks_kernel<E, 3> : quant_blocks_kernel<E, 4>;
}
template <int E>
auto dequant_pick(int u)
{
    return u == 1 ? dequant_blocks_kernel<E, 1> : u == 2 ? dequant_blocks_kernel<E, 2>
         : u == 3 ? dequant_blocks_kernel<E, 3> : dequant_blocks_kernel<E, 4>;
}

// launch(first row, rows, cut) over slices of rows whose workgroups fit one
// launch.
template <class F>
hipError_t in_row_slices(int64_t rows, int units, F &&launch)
{
    const Cut whole = cut_of(rows, units);
    const int64_t step = std::max<int64_t>(1, kMaxBlocksPerLaunch / whole.segs) * whole.rpb;
    for (int64_t r0 = 0; r0 < rows; r0 += step) {
        Cut c = whole;
        const int64_t n = std::min(rows - r0, step);
        c.blocks = whole.rpb == 1 ? n * c.segs : ceil_div(n, c.rpb);
        launch(r0, n, c);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace

hipError_t launch_quant_fp4(const void *x, int kind, int64_t rows, int64_t K, int64_t ldx, uint8_t *q, int64_t ldq,
                            uint8_t *s, int64_t lds, hipStream_t stream)
{
    const int units = (int)(K / 8), bytes = kind == kElemF32 ? 4 : 2;
    return in_row_slices(rows, units, [&](int64_t r0, int64_t n, const Cut &c) {
        auto fn = kind == kElemF32 ? quant_pick<kF32>(c.u) : kind == kElemF16 ? quant_pick<kF16>(c.u)
                                                                              : quant_pick<kBF16>(c.u);
        hipLaunchKernelGGL(fn, dim3((unsigned)c.blocks), dim3(256), 0, stream,
                           static_cast<const char *>(x) + r0 * ldx * bytes, n, units, ldx, q + r0 * ldq, ldq,
                           s + r0 * lds, lds, c.segs, c.rpb);
    });
}

hipError_t launch_dequant_fp4(const uint8_t *q, int64_t ldq, const uint8_t *s, int64_t lds, int64_t rows, int64_t K,
                              int kind, void *out, int64_t ldo, hipStream_t stream)
{
    const int units = (int)(K / 8), bytes = kind == kElemF32 ? 4 : 2;
    return in_row_slices(rows, units, [&](int64_t r0, int64_t n, const Cut &c) {
        auto fn = kind == kElemF32 ? dequant_pick<kF32>(c.u) : kind == kElemF16 ? dequant_pick<kF16>(c.u)
                                                                                : dequant_pick<kBF16>(c.u);
        hipLaunchKernelGGL(fn, dim3((unsigned)c.blocks), dim3(256), 0, stream, q + r0 * ldq, ldq, s + r0 * lds, lds,
                           n, units, static_cast<char *>(out) + r0 * ldo * bytes, ldo, c.segs, c.rpb);
    });
}

hipError_t launch_prepack_fp4(const void *w, int kind, const uint8_t *ws, int64_t N, int64_t K, int64_t ldw,
                              int64_t lds, void *packed, void *spacked, hipStream_t stream)
{
    const int blocks = (int)(K / kBlock), kblocks = (int)ceil_div(K, 128);
    const int64_t units = ceil_div(N, 16) * kblocks * 64;
    auto fn = kind < 0 ? prepack_fp4_kernel<-1> : kind == kElemF32 ? prepack_fp4_kernel<kF32>
                                                                   : prepack_fp4_kernel<kBF16>;
    for (int64_t u0 = 0; u0 < units; u0 += kMaxBlocksPerLaunch * 256) {
        const int64_t n = std::min(ceil_div(units - u0, 256), kMaxBlocksPerLaunch);
        hipLaunchKernelGGL(fn, dim3((unsigned)n), dim3(256), 0, stream, static_cast<const char *>(w), ldw, ws, lds,
                           (int)N, blocks, kblocks, static_cast<uint4 *>(packed), static_cast<uint8_t *>(spacked),
                           units, u0);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

hipError_t launch_unpack_fp4(const void *packed, const void *spacked, int64_t N, int64_t K, uint8_t *wq, int64_t ldw,
                             uint8_t *ws, int64_t lds, hipStream_t stream)
{
    const int blocks = (int)(K / kBlock), kblocks = (int)ceil_div(K, 128);
    const int64_t units = ceil_div(N, 16) * kblocks * 64;
    for (int64_t u0 = 0; u0 < units; u0 += kMaxBlocksPerLaunch * 256) {
        const int64_t n = std::min(ceil_div(units - u0, 256), kMaxBlocksPerLaunch);
        hipLaunchKernelGGL(unpack_fp4_kernel, dim3((unsigned)n), dim3(256), 0, stream,
                           static_cast<const uint4 *>(packed), static_cast<const uint8_t *>(spacked), (int)N, blocks,
                           kblocks, wq, ldw, ws, lds, units, u0);
        hipError_t err = hipGetLastError();
        if (err != hipSuccess)
            return err;
    }
    return hipSuccess;
}

}  // namespace w8a8
