// The norms around a block with its gate and residual scale (lores_block_norm),
// and the backward pass.  Per row:
//   p = x r1 w (x without a weight),  h = rnd(res + sc a(g) p),  y = h r2 wn
// Backward, from dy and the gradient dh that reaches h otherwise:
//   G = dh + r2 (e2 - n2 mean(e2 n2)),  e2 = dy wn, n2 = h r2;  dres = G,  dwn = sum dy n2
//   dg = sc G n1 w a'(g);  dx = r1 (e1 - n1 mean(e1 n1)),  e1 = sc G a w, n1 = x r1;
//   dw = sum sc G a n1;  without a weight dx = sc G a
//
// Bound by memory: a row is read once, kept in registers through both norms
// and written once, past the caches' recent lines (16384 x 4096 with a gate: forward
// 128 -> 117 us, backward 206 -> 202; followed by a read of y, 1024 to 32768 rows take as
// long or less).  16384 x 4096 with a gate: forward 118 us, 5.7 TB/s, backward 205, 5.2 TB/s;
// 8192 x 4096 of fp32 124, 5.4 TB/s, and 215, 5.0 TB/s.
#include "lores_gate.h"
#include "lores_layer.h"

namespace lores {
namespace {

// Whether rows are read past the caches' recent lines too: the longest ones (4096 x 16384 forward
// and backward 426 -> 379 us), not the others (1024 x 4096 37 -> 39, 16384 x 4096 297 -> 293).
template <int TPR, int VPT> constexpr bool kFar = TPR * VPT > 1024;

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
    if (a.res) keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.res + row * a.rs, t, a.n, kr);
    if (a.gate) keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.gate + row * a.gs, t, a.n, kg);
    float f = a.scale;
    if (a.w) {
        load_either<TPR, VPT, VEC>(a.w, a.w_bf16, t, a.n, w);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = e >= own_from<TPR, VEC>(t, i, a.n) ? h[i][e] : 0.0f;
                sum = fmaf(u, u, sum);
            }
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
    store_row<T, TPR, VPT, VEC, true>((T *)a.h + row * a.n, t, a.n, h);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float u = e >= own_from<TPR, VEC>(t, i, a.n) ? h[i][e] : 0.0f;
            sum = fmaf(u, u, sum);
            h[i][e] = h[i][e] * w[i][e];
            bits = max(bits, __float_as_uint(fabsf(h[i][e])));
        }
    float mx = __uint_as_float(min(bits, 0x7f800000u));
    reduce<TPR, true>(sum, mx, sm);
    const float rstd = 1.0f / sqrtf(sum / (float)a.n + a.eps);
    norm_store<TPR, VPT, VEC, true, true>(a.y, a.scales, a.out_prec, row, t, a.n, sum, mx, rstd, h);
}

// The weights' gradients are summed as the plain norm's: by each work-group over
// its rows, then over the work-groups in a fixed order.  Both stand side by
// side in a work-group's part: dwn, then (with a weight) dw.
//
// 1024 threads leave a thread 128 registers, which two vectors of five rows, two
// weights and their sums do not fit (4096 x 16384 with all kept: 630 us).  LEAN
// keeps the sums in LDS and reads the weights and the gate's row where they are used (271 us; 92 to
// 124 bytes of scratch a lane are left, and of odd rows 550 to 600).
template <typename T, int TPR, int VPT, int VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) lores_block_backward_kernel(const BlockArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    constexpr bool LEAN = TPR * VPT > 1024;
    __shared__ float sm[TPR > 64 ? TPR / 64 : 1][2];
    __shared__ __attribute__((aligned(16))) float sums[ROWS > 1 ? ROWS : 1][ROWS > 1 ? TPR * VPT * 8 : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    __shared__ float far[LEAN ? 2 : 1][LEAN ? VPT * 8 : 1][LEAN ? TPR : 1];
    float w[VPT][8], wn[VPT][8], dw[LEAN ? 1 : VPT][8], dwn[LEAN ? 1 : VPT][8];
    // the thread's sums of dwn (k = 0) and dw (1)
    auto sum = [&](int k, int i, int e) -> float & {
        if constexpr (LEAN) return far[k][i * 8 + e][t];
        else return k ? dw[i][e] : dwn[i][e];
    };
    auto weight_next = [&] { load_either<TPR, VPT, VEC>(a.wn, a.w_bf16, t, a.n, wn); };
    auto weight = [&] {
        if (a.w) {
            load_either<TPR, VPT, VEC>(a.w, a.w_bf16, t, a.n, w);
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) w[i][e] = 1.0f;
        }
    };
    if constexpr (!LEAN) {
        weight_next();
        weight();
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum(0, i, e) = sum(1, i, e) = 0.0f;
    const float per = 1.0f / (float)a.n;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + sub; row < a.rows; row += (int64_t)a.groups * ROWS) {
        Kept<T> kx[VPT], kh[VPT], kg[VPT], ky[VPT], kd[VPT];
        keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.h + row * a.n, t, a.n, kh);
        keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.dy + row * a.n, t, a.n, ky);
        keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.x + row * a.xs, t, a.n, kx);
        if (a.gate && !LEAN) keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.gate + row * a.gs, t, a.n, kg);
        if (a.dh) keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.dh + row * a.n, t, a.n, kd);
        if constexpr (LEAN) weight_next();
        float s2 = 0.0f, dot2 = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float h = kh[i].at(e);
                const bool own = e >= own_from<TPR, VEC>(t, i, a.n);
                const float hc = own ? h : 0.0f;
                s2 = fmaf(hc, hc, s2);
                dot2 = fmaf(hc, own ? wn[i][e] * ky[i].at(e) : 0.0f, dot2);
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
                sum(0, i, e) = fmaf(dy, n2, sum(0, i, e));
                G[i][e] = fmaf(r2, fmaf(-n2, c2, wn[i][e] * dy), a.dh ? kd[i].at(e) : 0.0f);
            }
        store_row<T, TPR, VPT, VEC, true>((T *)a.dres + row * a.n, t, a.n, G);
        if constexpr (LEAN) {
            weight();
            if (a.gate) keep_row<T, TPR, VPT, VEC, kFar<TPR, VPT>>((const T *)a.gate + row * a.gs, t, a.n, kg);
        }
        // from here on G is sc G
        auto gate_of = [&](int i, int e, float &value, float &slope) {
            value = slope = 1.0f;
            if (a.gate) {
                const float z = kg[i].at(e), sg = a.act ? sigmoid<T>(z) : 0.0f;
                value = gate_value(a.act, z, sg);
                slope = gate_slope(a.act, z, sg);
            }
        };
        float ga[LEAN ? 1 : VPT][8], gs[LEAN ? 1 : VPT][8];
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                G[i][e] = a.scale * G[i][e];
                float value, slope;
                gate_of(i, e, value, slope);
                if constexpr (!LEAN) { ga[i][e] = value; gs[i][e] = slope; }
                const float x = kx[i].at(e);
                const bool own = e >= own_from<TPR, VEC>(t, i, a.n);
                const float xc = own ? x : 0.0f;
                s1 = fmaf(xc, xc, s1);
                dot1 = fmaf(xc, own ? G[i][e] * value * w[i][e] : 0.0f, dot1);
            }
        float r1 = 1.0f, c1 = 0.0f;
        if (a.w) {
            reduce<TPR, false>(s1, dot1, sm);
            r1 = 1.0f / sqrtf(s1 / (float)a.n + a.eps);
            c1 = dot1 * r1 * per;
        }
        // G becomes dx
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float dz[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float value, slope;
                if constexpr (LEAN) gate_of(i, e, value, slope);
                else { value = ga[i][e]; slope = gs[i][e]; }
                const float n1 = kx[i].at(e) * r1, ge = G[i][e] * value;
                sum(1, i, e) = fmaf(ge, n1, sum(1, i, e));
                dz[e] = G[i][e] * n1 * w[i][e] * slope;
                // (without a weight x has no part in it: an infinite x times 0 would be NaN)
                G[i][e] = a.w ? r1 * fmaf(-n1, c1, ge * w[i][e]) : ge;
            }
            if (a.gate) store_vector<T, TPR, VEC, true>((T *)a.dgate + row * a.n, t, i, a.n, dz);
        }
        store_row<T, TPR, VPT, VEC, true>((T *)a.dx + row * a.n, t, a.n, G);
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
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k && !a.w) return;
            float x[VPT][8];
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = sum(k, i, e);
            store_row<float, TPR, VPT, VEC>(part + k * a.n, t, a.n, x);
        }
    }
}

template <typename T, int TPR, int VPT>
hipError_t go(int mode, bool back, const BlockArgs &a, hipStream_t s) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, TH = TPR < 256 ? 256 : TPR;
    if (back) {
        const dim3 grid((uint32_t)a.groups);
        if (mode == ROWS_VEC) lores_block_backward_kernel<T, TPR, VPT, ROWS_VEC><<<grid, TH, 0, s>>>(a);
        else lores_block_backward_kernel<T, TPR, VPT, ROWS_ODD><<<grid, TH, 0, s>>>(a);
        return hipGetLastError();
    }
    const dim3 grid = grid_of((a.rows + ROWS - 1) / ROWS);
    if (mode == ROWS_VEC) lores_block_kernel<T, TPR, VPT, ROWS_VEC><<<grid, TH, 0, s>>>(a);
    else lores_block_kernel<T, TPR, VPT, ROWS_ODD><<<grid, TH, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t by_width(int mode, bool back, const BlockArgs &a, hipStream_t s) {
    if (a.n <= 64) return go<T, 8, 1>(mode, back, a, s);
    if (a.n <= 128) return go<T, 16, 1>(mode, back, a, s);
    if (a.n <= 256) return go<T, 32, 1>(mode, back, a, s);
    if (a.n <= 512) return go<T, 64, 1>(mode, back, a, s);
    if (a.n <= 1024) return go<T, 64, 2>(mode, back, a, s);
    if (a.n <= 2048) return go<T, 256, 1>(mode, back, a, s);
    if (a.n <= 4096) return go<T, 256, 2>(mode, back, a, s);
    if (a.n <= 8192) return go<T, 1024, 1>(mode, back, a, s);
    return go<T, 1024, 2>(mode, back, a, s);
}

}  // namespace

// Work-groups that sum apart; us of the backward pass at 256 / 512 / 1024 of them, bf16, with a gate:
//   8192 x 1024   42  34  40    16384 x 2048  190 115 115    16384 x 4096  295 209 213
//   65536 x 128   46  34  40    8192 x 8192   248 254 271
int block_groups(int64_t rows, int32_t n) {
    const int side = n <= 64 ? 32 : n <= 128 ? 16 : n <= 256 ? 8 : n <= 1024 ? 4 : 1;     // rows of a work-group at once
    const int64_t most = n <= 4096 ? 512 : 256, need = (rows + side - 1) / side;
    return (int)(need < most ? need : most);
}

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
