// Projection on 4-bit weights (lores_mx_matmul): out[m][j] = sum_k a[m][k] w[j][k].
//
// The scaled matrix instruction 16 x 16 x 128 takes a lane's 32 neighbours of a
// row as they lie in memory, with the block's scale in a register: lane l
// holds block l / 16 of row l % 16.  Weights are its first operand, so a lane
// ends with 4 neighbouring outputs of one row.  E4M3 rows lie otherwise: lane l
// holds 16 neighbours from 16 (l / 16) and 16 from 64 + 16 (l / 16); their one
// factor per row is multiplied in at the end.
#include "lores_layer.h"

namespace lores {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint16_t to_bf16(float f) {
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
}

template <bool FP8>
__device__ __forceinline__ f32x4 product(const i32x8 &w, const i32x8 &a, f32x4 c, int ws, int as) {
    // format 4: E2M1, 0: E4M3
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, FP8 ? 0 : 4, 0, ws, 0, as);
}

// 4 outputs of row m from column j on
template <bool FP8, bool BF16>
__device__ __forceinline__ void put(const MxProduct &p, int64_t m, int j, f32x4 c) {
    if (m >= p.M) return;
    if constexpr (FP8) c *= p.a_rows[m];
    const int64_t at = m * p.N + j;
    if ((p.N & 3) == 0 && j + 3 < p.N) {
        if constexpr (BF16) *(u16x4 *)((uint16_t *)p.out + at) = u16x4{to_bf16(c[0]), to_bf16(c[1]), to_bf16(c[2]), to_bf16(c[3])};
        else *(f32x4 *)((float *)p.out + at) = c;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (j + i < p.N) {
            if constexpr (BF16) ((uint16_t *)p.out)[at + i] = to_bf16(c[i]);
            else ((float *)p.out)[at + i] = c[i];
        }
}

// Few rows: a work-group has 16 columns and 16 MT rows, its wavefronts share k.
template <bool FP8, bool BF16, int MT, int W>
__global__ void __launch_bounds__(64 * W) lores_mx_few_kernel(const MxProduct p) {
    __shared__ f32x4 sm[W][MT][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int tiles = (p.N + 15) / 16;
    const int64_t b = block_at(blockIdx.x, blockIdx.y), mb = b / tiles;
    const int j0 = (int)(b - mb * tiles) * 16;
    const int64_t m0 = mb * (16 * MT);
    if (m0 >= p.M) return;
    const int blocks = p.K / 32, per = mx_scale_stride(p.K), steps = (p.K + 127) / 128;
    const int64_t wr = min(j0 + r, p.N - 1);
    const uint8_t *wc = p.w + wr * (p.K / 2), *wsc = p.w_scales + wr * per;
    int64_t ar[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ar[i] = min(m0 + 16 * i + r, p.M - 1);
    f32x4 c[MT] = {};
    for (int k = wv; k < steps; k += W) {
        const int blk = 4 * k + g;
        const bool in = blk < blocks;
        i32x8 w = {};
        int ws = 0;
        if (in) {
            const i32x4 x = *(const i32x4 *)(wc + blk * 16);
            w = i32x8{x[0], x[1], x[2], x[3], 0, 0, 0, 0};
            ws = wsc[blk];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            i32x8 a = {};
            int as = 127;
            if constexpr (FP8) {
                const uint8_t *q = p.a + ar[i] * p.K;
                const int at = k * 128 + 16 * g;
                i32x4 x = {}, y = {};
                if (at < p.K) x = *(const i32x4 *)(q + at);
                if (at + 64 < p.K) y = *(const i32x4 *)(q + at + 64);
                a = i32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
            } else if (in) {
                const i32x4 x = *(const i32x4 *)(p.a + ar[i] * (p.K / 2) + blk * 16);
                a = i32x8{x[0], x[1], x[2], x[3], 0, 0, 0, 0};
                as = p.a_scales[ar[i] * per + blk];
            }
            c[i] = product<FP8>(w, a, c[i], ws, as);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sm[wv][i][lane] = c[i];
    __syncthreads();
    for (int i = wv; i < MT; i += W) {               // the wavefronts' sums in their order
        f32x4 s = sm[0][i][lane];
#pragma unroll
        for (int v = 1; v < W; ++v) s += sm[v][i][lane];
        put<FP8, BF16>(p, m0 + 16 * i + r, j0 + 4 * g, s);
    }
}

template <bool FP8, bool BF16, int MT>
hipError_t go_few(const MxProduct &p, hipStream_t s) {
    const int64_t groups = (p.M + 16 * MT - 1) / (16 * MT) * ((p.N + 15) / 16);
    lores_mx_few_kernel<FP8, BF16, MT, 8><<<grid_of(groups), 512, 0, s>>>(p);
    return hipGetLastError();
}

template <bool FP8, bool BF16>
hipError_t go(const MxProduct &p, hipStream_t s) {
    if (p.M <= 16) return go_few<FP8, BF16, 1>(p, s);
    return go_few<FP8, BF16, 4>(p, s);
}

}  // namespace

hipError_t launch_mx_product(bool a_fp8, bool out_bf16, const MxProduct &p, hipStream_t s) {
    if (a_fp8) return go<true, true>(p, s);
    return out_bf16 ? go<false, true>(p, s) : go<false, false>(p, s);
}

}  // namespace lores
