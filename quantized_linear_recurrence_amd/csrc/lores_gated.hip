// The norm of the recurrence's readout with its gate (lores_gated_norm), and
// its backward pass.  Rows are (token, head); with a(z) the gate, s its slope:
//   norm first: y = n w a(z), n = x r       gate first: u = x a(z), y = n w, n = u r
// Backward, from dy:
//   norm first: e = dy w a,  dx = r (e - n mean(e n)),  dz = dy w n s,  dw = sum dy a n
//   gate first: e = dy w,  du = r (e - n mean(e n)),  dx = du a,  dz = du x s,  dw = sum dy n
//
// Bound by memory: a row is read once, kept in registers and written once.  8192 x 32 x 128
// bf16, rows that no cache holds: forward 40 us, 5.0 TB/s (to 4-bit rows 41), backward 67 and
// 5 for the groups' sums, 5.0 TB/s; fp32 73 us, 5.5 TB/s, and 131, 5.1 TB/s; heads of 100 bf16 44
// and 68.  A row of up to 512 elements takes 8, 16, 32 or 64 threads, one vector each, longer ones
// 64, 256 or 1024 with one or two (16384 x 32 x 64, 8 threads a row: forward 40 us; 16: 62).
#include "lores_gate.h"
#include "lores_layer.h"

namespace lores {
namespace {

// the token of a row: the quotient by the reciprocal is at most one too small
__device__ __forceinline__ void split_row(const GatedArgs &a, uint32_t row, uint32_t &token, uint32_t &head) {
    token = __umulhi(row, a.per_heads);
    head = row - token * (uint32_t)a.heads;
    if (head >= (uint32_t)a.heads) { ++token; head -= (uint32_t)a.heads; }
}

template <typename T, int TPR, int VPT, int VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) lores_gated_kernel(const GatedArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;  // rows of a work-group
    __shared__ float sm[TPR > 64 ? TPR / 64 : 1][2];
    const int t = threadIdx.x % TPR;
    const int64_t row = block_at(blockIdx.x, blockIdx.y) * ROWS + threadIdx.x / TPR;
    if (row >= a.rows) return;                       // whole groups of TPR threads; no barrier for TPR <= 64
    uint32_t token, head;
    split_row(a, (uint32_t)row, token, head);
    float x[VPT][8], z[VPT][8], w[VPT][8];
    load_row<T, TPR, VPT, VEC>((const T *)a.x + token * a.xs[0] + head * a.xs[1], t, a.n, x);
    load_row<T, TPR, VPT, VEC>((const T *)a.gate + token * a.gs[0] + head * a.gs[1], t, a.n, z);
    const int64_t w_at = a.per_head ? (int64_t)head * a.n : 0;
    load_either<TPR, VPT, VEC>((const uint8_t *)a.w + w_at * (a.w_bf16 ? 2 : 4), a.w_bf16, t, a.n, w);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float g = gate_value(a.act, z[i][e], a.act ? sigmoid<T>(z[i][e]) : 0.0f);
            if (a.gate_first) x[i][e] = x[i][e] * g;
            const float u = e >= own_from<TPR, VEC>(t, i, a.n) ? x[i][e] : 0.0f;
            sum = fmaf(u, u, sum);
            w[i][e] = a.gate_first ? w[i][e] : w[i][e] * g;
        }
    sum = row_sum<TPR>(sum, sm);
    float rstd = 1.0f / sqrtf(sum / (float)a.n + a.eps);
    // Without an epsilon the r of a row of zeros is an infinity: its codes are 0.  So is that
    // of other rows whose squares are below fp32: they go on, to scales of NaN.
    if (a.out_prec == LORES_MXFP4 && rstd == __builtin_inff()) {
        float some = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) some = x[i][e] == 0.0f ? some : 1.0f;
        if (row_sum<TPR>(some, sm) == 0.0f) rstd = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) x[i][e] = x[i][e] * rstd * w[i][e];
    if (a.out_prec == LORES_FP32) {
        store_row<float, TPR, VPT, VEC>((float *)a.y + row * a.n, t, a.n, x);
    } else if (a.out_prec == LORES_BF16) {
        store_row<uint16_t, TPR, VPT, VEC>((uint16_t *)a.y + row * a.n, t, a.n, x);
    } else {                                         // a token's heads are one row of blocks
        const int per = mx_scale_stride((int64_t)a.heads * a.n), blocks = a.n / 32;
        store_mx<TPR, VPT>((uint8_t *)a.y + row * (a.n / 2), a.scales + (int64_t)token * per + head * blocks,
                           head + 1 == (uint32_t)a.heads ? per - a.heads * blocks : 0, t, a.n,
                           !(sum < __builtin_inff()), x);
    }
}

// dw is summed by each work-group over its rows (with weights per head, the
// rows of one head), in registers and over the rows side by side in LDS; a
// second kernel adds the work-groups' sums in a fixed order.  (Rows read past the
// caches' recent lines: 8192 x 32 x 128 alone 74 -> 68 us, but behind its forward pass, whose
// rows the last cache still holds, 110 -> 121 for both.)  LEAN: 1024 threads leave
// a thread 128 registers, so with two vectors the sums stand in LDS and the weights
// are read where they are used.
template <typename T, int TPR, int VPT, int VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) lores_gated_backward_kernel(const GatedArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    __shared__ float sm[TPR > 64 ? TPR / 64 : 1][2];
    __shared__ __attribute__((aligned(16))) float sums[ROWS > 1 ? ROWS : 1][ROWS > 1 ? TPR * VPT * 8 : 1];
    constexpr bool LEAN = TPR * VPT > 1024;
    __shared__ float far[LEAN ? VPT * 8 : 1][LEAN ? TPR : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    // weights per head: the work-groups of neighbouring heads are neighbours
    const uint32_t own = a.per_head ? blockIdx.x % (uint32_t)a.heads : 0;
    const uint32_t group = a.per_head ? blockIdx.x / (uint32_t)a.heads : blockIdx.x;
    const int64_t count = a.per_head ? a.rows / a.heads : a.rows;    // rows the groups share out
    float w[VPT][8], dw[LEAN ? 1 : VPT][8];
    auto sum = [&](int i, int e) -> float & {
        if constexpr (LEAN) return far[i * 8 + e][t];
        else return dw[i][e];
    };
    auto weight = [&] {
        load_either<TPR, VPT, VEC>((const uint8_t *)a.w + (int64_t)own * a.n * (a.w_bf16 ? 2 : 4), a.w_bf16, t, a.n, w);
    };
    if constexpr (!LEAN) weight();
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum(i, e) = 0.0f;
    for (int64_t r = (int64_t)group * ROWS + sub; r < count; r += (int64_t)a.groups * ROWS) {
        uint32_t token = (uint32_t)r, head = own;
        if (!a.per_head) split_row(a, (uint32_t)r, token, head);
        const int64_t row = (int64_t)token * a.heads + head;
        Kept<T> kx[VPT], kz[VPT], kg[VPT];
        keep_row<T, TPR, VPT, VEC>((const T *)a.x + token * a.xs[0] + head * a.xs[1], t, a.n, kx);
        keep_row<T, TPR, VPT, VEC>((const T *)a.gate + token * a.gs[0] + head * a.gs[1], t, a.n, kz);
        keep_row<T, TPR, VPT, VEC>((const T *)a.dy + row * a.n, t, a.n, kg);
        if constexpr (LEAN) weight();
        float s[LEAN ? 1 : VPT][8], ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = kz[i].at(e), x = kx[i].at(e);
                const float sg = a.act ? sigmoid<T>(z) : 0.0f;
                if constexpr (!LEAN) s[i][e] = sg;
                const float g = gate_value(a.act, z, sg), u = a.gate_first ? x * g : x;
                const float d = kg[i].at(e) * w[i][e];
                const bool own = e >= own_from<TPR, VEC>(t, i, a.n);
                const float uc = own ? u : 0.0f;
                ss = fmaf(uc, uc, ss);
                dot = fmaf(uc, !own ? 0.0f : a.gate_first ? d : d * g, dot);
            }
        reduce<TPR, false>(ss, dot, sm);
        const float rstd = 1.0f / sqrtf(ss / (float)a.n + a.eps);
        const float c = dot * rstd / (float)a.n;     // mean(e n)
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float dx[8], dz[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float z = kz[i].at(e), x = kx[i].at(e), dy = kg[i].at(e);
                float sg = 0.0f;                     // (LEAN makes it twice)
                if constexpr (LEAN) sg = a.act ? sigmoid<T>(z) : 0.0f;
                else sg = s[i][e];
                const float g = gate_value(a.act, z, sg), sl = gate_slope(a.act, z, sg);
                if (a.gate_first) {
                    const float n = x * g * rstd, du = rstd * fmaf(-n, c, dy * w[i][e]);
                    sum(i, e) = fmaf(dy, n, sum(i, e));
                    dx[e] = du * g;
                    dz[e] = du * x * sl;
                } else {
                    const float n = x * rstd, d = dy * w[i][e];
                    sum(i, e) = fmaf(dy * g, n, sum(i, e));
                    dx[e] = rstd * fmaf(-n, c, d * g);
                    dz[e] = d * n * sl;
                }
            }
            store_vector<T, TPR, VEC>((T *)a.dx + row * a.n, t, i, a.n, dx);
            store_vector<T, TPR, VEC>((T *)a.dgate + row * a.n, t, i, a.n, dz);
        }
    }
    float *part = a.part + ((int64_t)group * (a.per_head ? a.heads : 1) + own) * a.n;
    if constexpr (ROWS > 1) {                        // the rows side by side, in their order
        store_row<float, TPR, VPT, VEC>(sums[sub], t, a.n, dw);
        __syncthreads();
        for (int c = threadIdx.x; c < a.n; c += 256) {
            float x = sums[0][c];
#pragma unroll
            for (int i = 1; i < ROWS; ++i) x += sums[i][c];
            part[c] = x;
        }
    } else {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = sum(i, e);
            store_vector<float, TPR, VEC>(part, t, i, a.n, x);
        }
    }
}

template <typename T, int TPR, int VPT>
hipError_t go(int mode, bool back, const GatedArgs &a, hipStream_t s) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, TH = TPR < 256 ? 256 : TPR;
    if (back) {
        const dim3 grid((uint32_t)a.groups * (a.per_head ? a.heads : 1));
        if (mode == ROWS_VEC) lores_gated_backward_kernel<T, TPR, VPT, ROWS_VEC><<<grid, TH, 0, s>>>(a);
        else lores_gated_backward_kernel<T, TPR, VPT, ROWS_ODD><<<grid, TH, 0, s>>>(a);
        return hipGetLastError();
    }
    const dim3 grid = grid_of((a.rows + ROWS - 1) / ROWS);
    if (mode == ROWS_VEC) lores_gated_kernel<T, TPR, VPT, ROWS_VEC><<<grid, TH, 0, s>>>(a);
    else lores_gated_kernel<T, TPR, VPT, ROWS_ODD><<<grid, TH, 0, s>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t by_width(int mode, bool back, const GatedArgs &a, hipStream_t s) {
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

// Work-groups that sum dw apart (with weights per head: of all heads); us of the backward
// pass at 512 / 1024 / 2048 of them, bf16:
//   8192 x 32 x 128, one weight  84  76  77    per head  81  75  68
//   8192 x 4 x 1024, per head    73  74  79    8192 x 1 x 4096  77  81  89    4096 x 1 x 8192  116 128 154 (256: 111)
int gated_groups(int64_t tokens, int32_t heads, int32_t n, int32_t per_head) {
    const int side = n <= 64 ? 32 : n <= 128 ? 16 : n <= 256 ? 8 : n <= 1024 ? 4 : 1;     // rows of a work-group at once
    const int64_t most = n <= 512 ? (per_head ? 2048 : 1024) : n <= 4096 ? 512 : 256;
    const int64_t need = ((per_head ? tokens : tokens * heads) + side - 1) / side;
    const int64_t share = per_head ? (most + heads - 1) / heads : most;
    return (int)(need < share ? need : share);
}

hipError_t launch_gated(bool in_bf16, int mode, const GatedArgs &a, hipStream_t s) {
    return in_bf16 ? by_width<uint16_t>(mode, false, a, s) : by_width<float>(mode, false, a, s);
}

hipError_t launch_gated_backward(bool in_bf16, int mode, const GatedArgs &a, hipStream_t s) {
    if (a.rows) {                                    // without rows dw is a sum of nothing
        const hipError_t e = in_bf16 ? by_width<uint16_t>(mode, true, a, s) : by_width<float>(mode, true, a, s);
        if (e != hipSuccess) return e;
    }
    const int cols = a.n * (a.per_head ? a.heads : 1);
    return launch_group_sums(a.part, a.rows ? a.groups : 0, cols, cols, a.dw, nullptr, s);
}

}  // namespace lores
