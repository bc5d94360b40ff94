// The norms around a block with its gate and residual scale (lores_block_norm),
// and the backward pass.  Per row:
//   p = x r1 w (x without a weight),  h = rnd(res + sc a(g) p),  y = h r2 wn
// Backward, from dy and the gradient dh that reaches h otherwise:
//   G = dh + r2 (e2 - n2 mean(e2 n2)),  e2 = dy wn, n2 = h r2;  dres = G,  dwn = sum dy n2
//   dg = sc G n1 w a'(g);  dx = r1 (e1 - n1 mean(e1 n1)),  e1 = sc G a w, n1 = x r1;
//   dw = sum sc G a n1;  without a weight dx = sc G a
//
// Bound by memory: a row is read once, kept in registers through both norms
// and written once.
#include "lores_gate.h"
#include "lores_layer.h"

namespace lores {
namespace {

template <typename T, int TPR, int VPT, int VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) lores_block_kernel(const BlockArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;  // rows of a work-group
    __shared__ float sm[TPR > 64 ? TPR / 64 : 1][2];
    const int t = threadIdx.x % TPR;
    const int64_t row = block_at(blockIdx.x, blockIdx.y) * ROWS + threadIdx.x / TPR;
    if (row >= a.rows) return;                       // whole groups of TPR threads; no barrier for TPR <= 64
    float h[VPT][8], w[VPT][8];
    load_row<T, TPR, VPT, VEC>((const T *)a.x + row * a.xs, t, a.n, h);
    Kept<T> kr[VPT], kg[VPT];
    if (a.res) keep_row<T, TPR, VPT, VEC>((const T *)a.res + row * a.rs, t, a.n, kr);
    if (a.gate) keep_row<T, TPR, VPT, VEC>((const T *)a.gate + row * a.gs, t, a.n, kg);
    float f = a.scale;
    if (a.w) {
        load_either<TPR, VPT, VEC>(a.w, a.w_bf16, t, a.n, w);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
        sum = row_sum<TPR>(sum, sm);
        const float r1 = 1.0f / sqrtf(sum / (float)a.n + a.eps);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * r1 * w[i][e];
    }
    load_either<TPR, VPT, VEC>(a.wn, a.w_bf16, t, a.n, w);
    float sum = 0.0f;
    uint32_t bits = 0;                               // a NaN is above all numbers
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float p = f * h[i][e];
            if (a.gate) {
                const float z = kg[i].at(e);
                p = p * gate_value(a.act, z, a.act ? sigmoid<T>(z) : 0.0f);
            }
            h[i][e] = Elem<T>::rnd(a.res ? kr[i].at(e) + p : p);
        }
    store_row<T, TPR, VPT, VEC>((T *)a.h + row * a.n, t, a.n, h);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum = fmaf(h[i][e], h[i][e], sum);
            h[i][e] = h[i][e] * w[i][e];
            bits = max(bits, __float_as_uint(fabsf(h[i][e])));
        }
    float mx = __uint_as_float(min(bits, 0x7f800000u));
    reduce<TPR, true>(sum, mx, sm);
    const float rstd = 1.0f / sqrtf(sum / (float)a.n + a.eps);
    norm_store<TPR, VPT, VEC, true>(a.y, a.scales, a.out_prec, row, t, a.n, sum, mx, rstd, h);
}

// The weights' gradients are summed as the plain norm's: by each work-group over
// its rows, then over the work-groups in a fixed order.  Both stand side by
// side in a work-group's part: dwn, then (with a weight) dw.
template <typename T, int TPR, int VPT, int VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) lores_block_backward_kernel(const BlockArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    __shared__ float sm[TPR > 64 ? TPR / 64 : 1][2];
    __shared__ __attribute__((aligned(16))) float sums[ROWS > 1 ? ROWS : 1][ROWS > 1 ? TPR * VPT * 8 : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float w[VPT][8], wn[VPT][8], dw[VPT][8], dwn[VPT][8];
    load_either<TPR, VPT, VEC>(a.wn, a.w_bf16, t, a.n, wn);
    if (a.w) load_either<TPR, VPT, VEC>(a.w, a.w_bf16, t, a.n, w);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (!a.w) w[i][e] = 1.0f;
            dw[i][e] = dwn[i][e] = 0.0f;
        }
    const float per = 1.0f / (float)a.n;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + sub; row < a.rows; row += (int64_t)a.groups * ROWS) {
        Kept<T> kx[VPT], kh[VPT], kg[VPT], ky[VPT], kd[VPT];
        keep_row<T, TPR, VPT, VEC>((const T *)a.h + row * a.n, t, a.n, kh);
        keep_row<T, TPR, VPT, VEC>((const T *)a.dy + row * a.n, t, a.n, ky);
        keep_row<T, TPR, VPT, VEC>((const T *)a.x + row * a.xs, t, a.n, kx);
        if (a.gate) keep_row<T, TPR, VPT, VEC>((const T *)a.gate + row * a.gs, t, a.n, kg);
        if (a.dh) keep_row<T, TPR, VPT, VEC>((const T *)a.dh + row * a.n, t, a.n, kd);
        float s2 = 0.0f, dot2 = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = kh[i].at(e);
                s2 = fmaf(h, h, s2);
                dot2 = fmaf(h, wn[i][e] * ky[i].at(e), dot2);
            }
        reduce<TPR, false>(s2, dot2, sm);
        const float r2 = 1.0f / sqrtf(s2 / (float)a.n + a.eps);
        const float c2 = dot2 * r2 * per;
        float G[VPT][8], s1 = 0.0f, dot1 = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n2 = kh[i].at(e) * r2, dy = ky[i].at(e);
                dwn[i][e] = fmaf(dy, n2, dwn[i][e]);
                G[i][e] = fmaf(r2, fmaf(-n2, c2, wn[i][e] * dy), a.dh ? kd[i].at(e) : 0.0f);
            }
        store_row<T, TPR, VPT, VEC>((T *)a.dres + row * a.n, t, a.n, G);
        // from here on G is sc G, and with a gate a and a' stand in registers
        float ga[VPT][8], gs[VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                G[i][e] = a.scale * G[i][e];
                ga[i][e] = gs[i][e] = 1.0f;
                if (a.gate) {
                    const float z = kg[i].at(e), sg = a.act ? sigmoid<T>(z) : 0.0f;
                    ga[i][e] = gate_value(a.act, z, sg);
                    gs[i][e] = gate_slope(a.act, z, sg);
                }
                const float x = kx[i].at(e);
                s1 = fmaf(x, x, s1);
                dot1 = fmaf(x, G[i][e] * ga[i][e] * w[i][e], dot1);
            }
        float r1 = 1.0f, c1 = 0.0f;
        if (a.w) {
            reduce<TPR, false>(s1, dot1, sm);
            r1 = 1.0f / sqrtf(s1 / (float)a.n + a.eps);
            c1 = dot1 * r1 * per;
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float n1 = kx[i].at(e) * r1, ge = G[i][e] * ga[i][e];
                dw[i][e] = fmaf(ge, n1, dw[i][e]);
                gs[i][e] = G[i][e] * n1 * w[i][e] * gs[i][e];
                G[i][e] = r1 * fmaf(-n1, c1, ge * w[i][e]);
            }
        store_row<T, TPR, VPT, VEC>((T *)a.dx + row * a.n, t, a.n, G);
        if (a.gate) store_row<T, TPR, VPT, VEC>((T *)a.dgate + row * a.n, t, a.n, gs);
    }
    const int cols = a.w ? 2 * a.n : a.n;
    float *part = a.part + (int64_t)blockIdx.x * cols;
    if constexpr (ROWS > 1) {                        // the rows side by side, in their order
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k && !a.w) return;
            if (k) __syncthreads();                  // the first sums have been read
            store_row<float, TPR, VPT, VEC>(sums[sub], t, a.n, k ? dw : dwn);
            __syncthreads();
            for (int c = threadIdx.x; c < a.n; c += 256) {
                float x = sums[0][c];
#pragma unroll
                for (int i = 1; i < ROWS; ++i) x += sums[i][c];
                part[k * a.n + c] = x;
            }
        }
    } else {
        store_row<float, TPR, VPT, VEC>(part, t, a.n, dwn);
        if (a.w) store_row<float, TPR, VPT, VEC>(part + a.n, t, a.n, dw);
    }
}

template <typename T, int TPR, int VPT>
hipError_t go(int mode, bool back, const BlockArgs &a, hipStream_t s) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, TH = TPR < 256 ? 256 : TPR;
    if (back) {
        const dim3 grid((uint32_t)a.groups);
        if (mode == ROWS_VEC) lores_block_backward_kernel<T, TPR, VPT, ROWS_VEC><<<grid, TH, 0, s>>>(a);
        else lores_block_backward_kernel<T, TPR, VPT, ROWS_ANY><<<grid, TH, 0, s>>>(a);
        return hipGetLastError();
    }
    const dim3 grid = grid_of((a.rows + ROWS - 1) / ROWS);
    if (mode == ROWS_VEC) lores_block_kernel<T, TPR, VPT, ROWS_VEC><<<grid, TH, 0, s>>>(a);
    else if (mode == ROWS_BLOCKS) lores_block_kernel<T, TPR, VPT, ROWS_BLOCKS><<<grid, TH, 0, s>>>(a);
    else lores_block_kernel<T, TPR, VPT, ROWS_ANY><<<grid, TH, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t by_width(int mode, bool back, const BlockArgs &a, hipStream_t s) {
    if (a.n <= 128) return go<T, 16, 1>(mode, back, a, s);
    if (a.n <= 512) return go<T, 64, 1>(mode, back, a, s);
    if (a.n <= 1024) return go<T, 64, 2>(mode, back, a, s);
    if (a.n <= 2048) return go<T, 256, 1>(mode, back, a, s);
    if (a.n <= 4096) return go<T, 256, 2>(mode, back, a, s);
    if (a.n <= 8192) return go<T, 1024, 1>(mode, back, a, s);
    return go<T, 1024, 2>(mode, back, a, s);
}

}  // namespace

int block_groups(int64_t rows, int32_t n) { return norm_groups(rows, n); }

hipError_t launch_block(bool in_bf16, int mode, const BlockArgs &a, hipStream_t s) {
    return in_bf16 ? by_width<uint16_t>(mode, false, a, s) : by_width<float>(mode, false, a, s);
}

hipError_t launch_block_backward(bool in_bf16, int mode, const BlockArgs &a, hipStream_t s) {
    if (a.rows) {                                    // without rows the sums are of nothing
        const hipError_t e = in_bf16 ? by_width<uint16_t>(mode, true, a, s) : by_width<float>(mode, true, a, s);
        if (e != hipSuccess) return e;
    }
    return launch_group_sums(a.part, a.rows ? a.groups : 0, a.w ? 2 * a.n : a.n, a.n, a.dwn, a.dw, s);
}

}  // namespace lores
