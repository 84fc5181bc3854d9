// Small-M microscaled 4-bit matmul, for gfx950: a handful of token rows
// against a large weight, with the quantization of the rows in the same launch
// where they come as floats. Same products as the main kernel's
// (scaled_mm_fp4.hip); the fp32 sums across blocks are added in another order.
//
// The weight stream bounds it (17/32 bytes per weight), so it is spread over
// as many wavefronts as the shape gives, and nothing but the last sums passes
// through LDS:
//   - A workgroup owns 16*FN channels and 16*FM token rows; its WK wavefronts
//     take chunks of 512 elements in turn (4 k-blocks, the 16 bytes of scales
//     that a row keeps together). All loads of a chunk are issued before its
//     first product waits for any of them.
//   - A k-block is one v_mfma_scale_f32_16x16x128_f8f6f4 per fragment pair.
//     The packed 1 KB weight fragment is its A operand as stored (lane l: the
//     32 codes of channel l%16, block l/16), the token rows its B operand.
//   - With float rows (QK) every workgroup quantizes its rows into LDS while
//     its first weights are on their way, 8 elements a thread at a time (the
//     rows are few and sit in L2), and takes its token operands from there;
//     the workgroups of the first channels write the codes and scales out.
//     Up to kSlots such steps: measured on MI355X, N 1111, two launches against
//     this, M 16 K 512 (two steps) 4.7 against 3.5 us, M 8 K 2048 (four) 5.3
//     against 4.3, M 16 K 2048 (eight) 5.4 against 5.9. One row, N 12288, K
//     4096: a row quantized by each lane in place of its own operand takes 10.6
//     us, this 6.5 to 8.0 (7.3 in the median of a trace, 3.7 TB/s of weights),
//     two launches 8.7.
// Ragged tails: token rows past M read row M-1 and channels past N the last
// image (never stored); blocks past the row's last read the last one again, as
// 1.0-scaled operands of zero weights.
#include <algorithm>

#include "fp4_rule.hpp"
#include "internal.hpp"

namespace w8a8 {
namespace {

using namespace fp4_rule;

typedef int v4i __attribute__((ext_vector_type(4)));
typedef int v8i __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

template <int FM_, int FN_, int WK_>
struct Skinny4 {
    static constexpr int FM = FM_, FN = FN_, WK = WK_;
    static constexpr int BM = 16 * FM, BN = 16 * FN, THREADS = 64 * WK;
};

constexpr int kCodes = -1;       // QK: codes and scale bytes made before
constexpr int kSlots = 4;        // units of 8 elements that a thread quantizes, at most

// Bytes of LDS behind one quantized row of K = 16 * blocks code bytes: the
// codes, then the scale bytes of whole chunks.
__host__ __device__ constexpr int row_bytes(int blocks) { return blocks * 16 + (blocks + 15) / 16 * 16; }

// Rows m0 .. m0+rows-1 of x quantized by the workgroup into LDS, row r at
// r * row_bytes, and with `writer` to xq and sx. The rows' units of 8 elements
// are one list, dealt out THREADS at a time, of which a thread reads AHEAD
// before it quantizes the first; a block's four are neighbouring lanes'.
template <int THREADS, int E, int AHEAD>
__device__ __forceinline__ void quantize_rows(const MmArgs &a, int m0, int rows, bool writer, char *tok)
{
    constexpr int XB = E == kF32 ? 4 : 2;
    const int units = a.blocks * 4;
    const int row_step = THREADS / units, unit_step = THREADS % units;
    auto next = [&](int &row, int &unit) __attribute__((always_inline)) {
        row += row_step;
        unit += unit_step;
        if (unit >= units) {
            unit -= units;
            ++row;
        }
    };
    int r = (int)threadIdx.x / units, u = (int)threadIdx.x - r * units;
    for (int s0 = 0; s0 < rows * units; s0 += AHEAD * THREADS) {
        uint4 lo[AHEAD], hi[AHEAD];
        int rr = r, uu = u;
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            // (past the last row: the first unit again, not kept)
            const bool in = rr < rows;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                reinterpret_cast<const char *>(a.x) + ((int64_t)(m0 + (in ? rr : 0)) * a.ldx + (in ? uu : 0) * 8) * XB);
            lo[s] = src[0];
            hi[s] = E == kF32 ? src[1] : lo[s];
            next(rr, uu);
        }
#pragma unroll
        for (int s = 0; s < AHEAD; ++s) {
            // The four lanes of a block are all inside the rows or all past them.
            u32 m = absmax8<E>(lo[s], hi[s]);
            m = max(m, (u32)__builtin_amdgcn_update_dpp((int)m, (int)m, 0xB1, 0xF, 0xF, false));
            m = max(m, (u32)__builtin_amdgcn_update_dpp((int)m, (int)m, 0x4E, 0xF, 0xF, false));
            const u32 byte = scale_byte(m);
            if (r < rows) {
                const u32 c = codes8<E>(lo[s], hi[s], byte);
                char *row = tok + r * row_bytes(a.blocks);
                *reinterpret_cast<u32 *>(row + u * 4) = c;
                if ((u & 3) == 0)
                    row[a.blocks * 16 + (u >> 2)] = (char)byte;
                if (writer) {
                    *reinterpret_cast<u32 *>(const_cast<int8_t *>(a.xq) + (int64_t)(m0 + r) * a.ldq + u * 4) = c;
                    if ((u & 3) == 0)
                        const_cast<uint8_t *>(a.sx)[(int64_t)(m0 + r) * a.lds + (u >> 2)] = (uint8_t)byte;
                }
            }
            next(r, u);
        }
    }
}

template <class S, int OUT, int QK>
__global__ __launch_bounds__(S::THREADS) void skinny_fp4_kernel(const MmArgs a)
{
    constexpr bool RAW = OUT == kOutI32, OUT_F16 = OUT == kOutF16;
    __shared__ f32x4 part[S::WK - 1][S::FM * S::FN][64];
    extern __shared__ __attribute__((aligned(16))) char tok[];   // QK: the quantized rows

    const int lane = threadIdx.x & 63;
    const int wk = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int r16 = lane & 15, sub = lane >> 4;
    const int tiles_m = (a.M + S::BM - 1) / S::BM;
    const int tiles_n = (a.nblocks + S::FN - 1) / S::FN;
    const int t = xcd_remap(blockIdx.x, tiles_m * tiles_n);
    const int m0 = (t % tiles_m) * S::BM, nb0 = (t / tiles_m) * S::FN;
    const int KB = a.kblocks, chunks = (KB + 3) / 4;

    const v4i *wsrc[S::FN];
    const v4i *ssrc[S::FN];
#pragma unroll
    for (int j = 0; j < S::FN; ++j) {
        const int64_t nb = min(nb0 + j, a.nblocks - 1);
        wsrc[j] = reinterpret_cast<const v4i *>(a.wp) + nb * KB * 64 + lane;
        ssrc[j] = reinterpret_cast<const v4i *>(a.sw) + nb * chunks * 16 + r16;
    }
    const char *xsrc[S::FM], *sxsrc[S::FM];            // this lane's rows of codes and scale bytes
#pragma unroll
    for (int f = 0; f < S::FM; ++f) {
        const int r = min(16 * f + r16, a.M - 1 - m0);
        xsrc[f] = QK == kCodes ? reinterpret_cast<const char *>(a.xq) + (int64_t)(m0 + r) * a.ldq
                               : tok + r * row_bytes(a.blocks);
        sxsrc[f] = QK == kCodes ? reinterpret_cast<const char *>(a.sx) + (int64_t)(m0 + r) * a.lds
                                : xsrc[f] + a.blocks * 16;
    }

    f32x4 acc[S::FM][S::FN] = {};
    // Fragments past the weight's last k-block read the last one; their products
    // are skipped.
    auto weights = [&](int c, v4i (&w)[4][S::FN], v4i (&ws)[S::FN]) __attribute__((always_inline)) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                w[q][j] = __builtin_nontemporal_load(wsrc[j] + (int64_t)min(4 * c + q, KB - 1) * 64);
#pragma unroll
        for (int j = 0; j < S::FN; ++j)
            ws[j] = ssrc[j][(int64_t)min(c, chunks - 1) * 16];
    };
    auto products = [&](int c, const v4i (&w)[4][S::FN], const v4i (&ws)[S::FN]) __attribute__((always_inline)) {
        v4i x[4][S::FM], xs[S::FM];
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int f = 0; f < S::FM; ++f)
                x[q][f] = *reinterpret_cast<const v4i *>(xsrc[f] + (int64_t)min(16 * c + 4 * q + sub, a.blocks - 1) * 16);
#pragma unroll
        for (int f = 0; f < S::FM; ++f)
            xs[f] = *reinterpret_cast<const v4i *>(sxsrc[f] + c * 16);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            if (4 * c + q >= KB)
                break;
            const bool inside = 16 * c + 4 * q + sub < a.blocks;
#pragma unroll
            for (int f = 0; f < S::FM; ++f) {
                const u32 sx = inside ? (u32)xs[f][q] >> (8 * sub) : 127u;
#pragma unroll
                for (int j = 0; j < S::FN; ++j)
                    acc[f][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                        v8i{w[q][j][0], w[q][j][1], w[q][j][2], w[q][j][3]},
                        v8i{x[q][f][0], x[q][f][1], x[q][f][2], x[q][f][3]}, acc[f][j], 4, 4, 0,
                        (int)((u32)ws[j][q] >> (8 * sub)), 0, (int)sx);
            }
        }
    };
    v4i w[4][S::FN], ws[S::FN];
    if constexpr (QK != kCodes) {
        // (of every wave, clamped into the weight: no wave skips the barrier)
        weights(wk, w, ws);
        const int rows = min(S::BM, a.M - m0);
        if (rows * a.blocks * 4 <= S::THREADS)
            quantize_rows<S::THREADS, QK, 1>(a, m0, rows, nb0 == 0, tok);
        else if (rows * a.blocks * 4 <= 2 * S::THREADS)
            quantize_rows<S::THREADS, QK, 2>(a, m0, rows, nb0 == 0, tok);
        else
            quantize_rows<S::THREADS, QK, 4>(a, m0, rows, nb0 == 0, tok);
        __syncthreads();
        if (wk < chunks)
            products(wk, w, ws);
    }
    for (int c = QK != kCodes ? wk + S::WK : wk; c < chunks; c += S::WK) {
        weights(c, w, ws);
        products(c, w, ws);
    }

    if (wk > 0) {
#pragma unroll
        for (int f = 0; f < S::FM; ++f)
#pragma unroll
            for (int j = 0; j < S::FN; ++j)
                part[wk - 1][f * S::FN + j][lane] = acc[f][j];
    }
    __syncthreads();
    if (wk != 0)
        return;
#pragma unroll
    for (int f = 0; f < S::FM; ++f)
#pragma unroll
        for (int j = 0; j < S::FN; ++j)
#pragma unroll
            for (int w = 0; w < S::WK - 1; ++w)
                acc[f][j] += part[w][f * S::FN + j][lane];

    // Register r of lane l is channel 4*(l/16) + r, token l%16.
#pragma unroll
    for (int f = 0; f < S::FM; ++f) {
        const int m = m0 + 16 * f + r16;
        if (m >= a.M)
            continue;
#pragma unroll
        for (int j = 0; j < S::FN; ++j) {
            const int n = 16 * (nb0 + j) + 4 * sub;
            if (n >= a.N)
                continue;
            f32x4 v = acc[f][j];
            const bool whole = a.vec_store && n + 3 < a.N;
            if constexpr (RAW) {
                float *o = reinterpret_cast<float *>(a.out) + (int64_t)m * a.ldo + n;
                if (whole) {
                    *reinterpret_cast<f32x4 *>(o) = v;
                } else {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (n + r < a.N)
                            o[r] = v[r];
                }
            } else {
                if (a.bias) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const unsigned b = a.bias[min(n + r, a.N - 1)];
                        v[r] += OUT_F16 ? quant_rule::f16_to_float(b) : __uint_as_float(b << 16);
                    }
                }
                u32 lo, hi;
                if constexpr (OUT_F16) {
                    lo = __builtin_bit_cast(u32, __builtin_convertvector((f32x2){v[0], v[1]}, f16x2));
                    hi = __builtin_bit_cast(u32, __builtin_convertvector((f32x2){v[2], v[3]}, f16x2));
                } else {
                    lo = __builtin_bit_cast(u32, __builtin_convertvector((f32x2){v[0], v[1]}, bf16x2));
                    hi = __builtin_bit_cast(u32, __builtin_convertvector((f32x2){v[2], v[3]}, bf16x2));
                }
                uint16_t *o = reinterpret_cast<uint16_t *>(a.out) + (int64_t)m * a.ldo + n;
                if (whole) {
                    *reinterpret_cast<uint2 *>(o) = make_uint2(lo, hi);
                } else {
                    const u32 hv[4] = {lo & 0xffffu, lo >> 16, hi & 0xffffu, hi >> 16};
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (n + r < a.N)
                            o[r] = (uint16_t)hv[r];
                }
            }
        }
    }
}

template <class S>
constexpr Fp4Skinny entry(const char *name)
{
    return Fp4Skinny{
        TileEntry{name, S::BM, S::BN, S::THREADS, true,
                  {skinny_fp4_kernel<S, kOutBF16, kCodes>, skinny_fp4_kernel<S, kOutI32, kCodes>,
                   skinny_fp4_kernel<S, kOutF16, kCodes>},
                  {nullptr, nullptr, nullptr}},
        {{skinny_fp4_kernel<S, kOutBF16, kBF16>, skinny_fp4_kernel<S, kOutI32, kBF16>,
          skinny_fp4_kernel<S, kOutF16, kBF16>},
         {skinny_fp4_kernel<S, kOutBF16, kF32>, skinny_fp4_kernel<S, kOutI32, kF32>,
          skinny_fp4_kernel<S, kOutF16, kF32>},
         {skinny_fp4_kernel<S, kOutBF16, kF16>, skinny_fp4_kernel<S, kOutI32, kF16>,
          skinny_fp4_kernel<S, kOutF16, kF16>}}};
}

// 16*FM token rows x 16*FN channels / WK waves along K.
const Fp4Skinny kSkinny4[] = {
    entry<Skinny4<1, 1, 8>>("s16x16/k8"),
    entry<Skinny4<1, 2, 8>>("s16x32/k8"),
};

}  // namespace

int fp4_skinny_count() { return (int)(sizeof(kSkinny4) / sizeof(kSkinny4[0])); }
const Fp4Skinny &fp4_skinny(int i) { return kSkinny4[i]; }

hipError_t launch_skinny_quant_fp4(const MmArgs &a, int x_kind, int mode, int i, hipStream_t stream)
{
    const Fp4Skinny &s = kSkinny4[i];
    const int64_t rows = std::min<int64_t>(a.M, s.tile.bm);
    if (ceil_div(rows * a.blocks * 4, s.tile.threads) > kSlots)
        return hipErrorNotSupported;
    const int64_t tiles = ceil_div(a.M, s.tile.bm) * ceil_div(a.N, s.tile.bn);
    hipLaunchKernelGGL(s.quant[x_kind][mode], dim3((unsigned)tiles), dim3(s.tile.threads),
                       (size_t)(rows * row_bytes(a.blocks)), stream, a);
    return hipGetLastError();
}

}  // namespace w8a8
