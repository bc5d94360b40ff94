// Root-mean-square norm with the residual's addition and 8-bit outputs
// (lores_rmsnorm), and its backward pass.
//
// Per row, with h = rnd(x + res) in the inputs' type, z_j = fl(h_j w_j):
//   r = (mean_j h_j^2 + eps)^(-1/2),  y_j = rnd(z_j r)
// 8-bit outputs: m = max_j |z_j| (at least 2^-119), code_j = rnd(z_j fl(top fl(1 / m))), scale =
// fl(fl(m / top) r): the row's factor r cancels in the codes, so they depend
// on elementwise roundings alone and not on the order of the row's sum.
// Backward, with dy and the gradient dres that arrives at h by itself:
//   dx_j = r (w_j dy_j - h_j r^2 mean_i(w_i dy_i h_i)) + dres_j
//   dw_j = sum over rows of dy_j h_j r
//
// Everything is bound by memory: a row is read once, kept in registers (8
// elements per thread and vector), reduced once and written.  Rows take 16,
// 64, 256 or 1024 threads so that a thread holds one or two vectors: a decode
// batch of 64 rows of 4096 then spreads its loads over 64 x 256 threads, and
// heads of 128 elements fill whole wavefronts (four rows in each).  Sums are
// fp32.  dw is summed by work-groups, each over its rows in registers and over
// the rows it takes side by side in LDS, and the work-groups' sums are added by
// a second kernel in a fixed order: the result does not depend on scheduling.
//
// Measured (bf16, 16384 x 4096, residual): forward 87 us, 0.54 GB at 6.2 TB/s;
// backward 112 us, 0.55 GB at 5.0 TB/s, and 7 us for the groups' sums.
// 64 x 4096 to int8 take 5.0 us, launch and two waits on memory.
#include "lores_seq.h"

namespace lores {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf2f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
// round to nearest even; a NaN stays one
__device__ __forceinline__ uint16_t f2bf(float f) {
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
}

template <typename T> struct Elem;
template <> struct Elem<float> {
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float x) { *p = x; }
    static __device__ __forceinline__ float rnd(float x) { return x; }
    static __device__ __forceinline__ void get8(const float *p, float *x) {
        const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
    }
    static __device__ __forceinline__ void put8(float *p, const float *x) {
        *(f32x4 *)p = f32x4{x[0], x[1], x[2], x[3]};
        *(f32x4 *)(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
    }
};
template <> struct Elem<uint16_t> {
    static __device__ __forceinline__ float get(const uint16_t *p) { return bf2f(*p); }
    static __device__ __forceinline__ void put(uint16_t *p, float x) { *p = f2bf(x); }
    static __device__ __forceinline__ float rnd(float x) { return bf2f(f2bf(x)); }
    static __device__ __forceinline__ void get8(const uint16_t *p, float *x) {
        const u32x4 a = *(const u32x4 *)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(a[e] << 16);
            x[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void put8(uint16_t *p, const float *x) {
        u32x4 a;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            a[e] = (uint32_t)f2bf(x[2 * e]) | ((uint32_t)f2bf(x[2 * e + 1]) << 16);
        *(u32x4 *)p = a;
    }
};

// One thread's elements of a row: VPT vectors of 8.  VEC: 8 neighbours per
// vector and thread (16-byte accesses); else element e of vector i is 8 i + e
// strides of TPR away, so that neighbouring threads read neighbouring
// elements of rows at any alignment.
template <int TPR, bool VEC>
__device__ __forceinline__ int col(int t, int i, int e) {
    return VEC ? (i * TPR + t) * 8 + e : (i * 8 + e) * TPR + t;
}

template <typename T, int TPR, int VPT, bool VEC>
__device__ __forceinline__ void load_row(const T *p, int t, int n, float (&x)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            const int c = (i * TPR + t) * 8;
            if (c < n) {
                Elem<T>::get8(p + c, x[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
            }
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = col<TPR, VEC>(t, i, e);
                x[i][e] = c < n ? Elem<T>::get(p + c) : 0.0f;
            }
        }
    }
}

template <typename T, int TPR, int VPT, bool VEC>
__device__ __forceinline__ void store_row(T *p, int t, int n, const float (&x)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            const int c = (i * TPR + t) * 8;
            if (c < n) Elem<T>::put8(p + c, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = col<TPR, VEC>(t, i, e);
                if (c < n) Elem<T>::put(p + c, x[i][e]);
            }
        }
    }
}

template <int TPR, int VPT, bool VEC>
__device__ __forceinline__ void store_bytes(uint8_t *p, int t, int n, const uint8_t (&x)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC) {
            const int c = (i * TPR + t) * 8;
            u32x2 w = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)x[i][e] << (8 * (e & 3));
            if (c < n) *(u32x2 *)(p + c) = w;
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const int c = col<TPR, VEC>(t, i, e);
                if (c < n) p[c] = x[i][e];
            }
        }
    }
}

// Over one row's threads: the sum of `a`, and the maximum (MAX) or the sum of
// `b`, in every one of them.
template <int TPR, bool MAX>
__device__ __forceinline__ void reduce(float &a, float &b, float (*sm)[2]) {
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int d = 1; d < W; d <<= 1) {
        a += __shfl_xor(a, d);
        const float o = __shfl_xor(b, d);
        b = MAX ? fmaxf(b, o) : b + o;
    }
    if constexpr (TPR > 64) {
        const int wv = threadIdx.x >> 6;
        __syncthreads();                             // the last row's values have been read
        if ((threadIdx.x & 63) == 0) { sm[wv][0] = a; sm[wv][1] = b; }
        __syncthreads();
        a = sm[0][0];
        b = sm[0][1];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) {
            a += sm[i][0];
            b = MAX ? fmaxf(b, sm[i][1]) : b + sm[i][1];
        }
    }
}

template <typename T, int TPR, int VPT, bool VEC>
__device__ __forceinline__ void load_weight(const NormArgs &a, int t, float (&w)[VPT][8]) {
    if (a.w_bf16) load_row<uint16_t, TPR, VPT, VEC>((const uint16_t *)a.w, t, a.n, w);
    else load_row<float, TPR, VPT, VEC>((const float *)a.w, t, a.n, w);
}

template <typename T, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) lores_norm_kernel(const NormArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;  // rows of a work-group
    __shared__ float sm[TPR > 64 ? TPR / 64 : 1][2];
    const int t = threadIdx.x % TPR;
    const int64_t row = block_at(blockIdx.x, blockIdx.y) * ROWS + threadIdx.x / TPR;
    if (row >= a.rows) return;                       // whole groups of TPR threads; no barrier for TPR <= 64
    float h[VPT][8], w[VPT][8];
    load_row<T, TPR, VPT, VEC>((const T *)a.x + row * a.x_stride, t, a.n, h);
    if (a.res) {
        float r[VPT][8];
        load_row<T, TPR, VPT, VEC>((const T *)a.res + row * a.res_stride, t, a.n, r);
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = Elem<T>::rnd(h[i][e] + r[i][e]);
        store_row<T, TPR, VPT, VEC>((T *)a.h + row * a.n, t, a.n, h);
    }
    load_weight<T, TPR, VPT, VEC>(a, t, w);
    // magnitudes are compared as bits, where a NaN is above all numbers: the
    // floating-point maximum would drop it.  It goes on as an infinity.
    const float inf = __builtin_inff();
    float sum = 0.0f;
    uint32_t bits = 0;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            sum = fmaf(h[i][e], h[i][e], sum);
            h[i][e] = h[i][e] * w[i][e];             // z
            bits = max(bits, __float_as_uint(fabsf(h[i][e])));
        }
    float mx = __uint_as_float(min(bits, __float_as_uint(inf)));
    reduce<TPR, true>(sum, mx, sm);
    const float rstd = 1.0f / sqrtf(sum / (float)a.n + a.eps);
    if (a.out_prec == LORES_FP32 || a.out_prec == LORES_BF16) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) h[i][e] = h[i][e] * rstd;
        if (a.out_prec == LORES_FP32)
            store_row<float, TPR, VPT, VEC>((float *)a.y + row * a.n, t, a.n, h);
        else
            store_row<uint16_t, TPR, VPT, VEC>((uint16_t *)a.y + row * a.n, t, a.n, h);
        return;
    }
    const float top = a.out_prec == LORES_INT8 ? 127.0f : 448.0f;
    // a row with a z that is not finite, or with squares beyond fp32, has the
    // scale NaN and the codes 0
    const bool lost = !(mx < inf) || !(sum < inf);
    const float nan = __builtin_nanf("");
    // a maximum under 2^-119 (top / m would leave fp32's range) counts as
    // 2^-119, in the codes and in the scale: such a row uses fewer codes
    const float m = fmaxf(mx, 0x1p-119f);
    const float inv = lost ? nan : top * (1.0f / m);
    uint8_t c[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float x = h[i][e] * inv;
            if (a.out_prec == LORES_INT8) {
                const float q = rintf(fminf(fmaxf(x, -127.0f), 127.0f));
                c[i][e] = x == x ? (uint8_t)(int8_t)(int)q : (uint8_t)0;
            } else {
                const float q = fminf(fmaxf(x, -448.0f), 448.0f);
                c[i][e] = x == x ? (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false)
                                 : (uint8_t)0;
            }
        }
    store_bytes<TPR, VPT, VEC>((uint8_t *)a.y + row * a.n, t, a.n, c);
    // (without an epsilon the r of a row of zeros is an infinity)
    if (t == 0) a.scales[row] = lost ? nan : mx == 0.0f ? 0.0f : m / top * rstd;
}

template <typename T, int TPR, int VPT, bool VEC>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) lores_norm_backward_kernel(const NormArgs a) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1;
    __shared__ float sm[TPR > 64 ? TPR / 64 : 1][2];
    __shared__ __attribute__((aligned(16))) float sums[ROWS > 1 ? ROWS : 1][ROWS > 1 ? TPR * VPT * 8 : 1];
    const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
    float w[VPT][8], dw[VPT][8];
    load_weight<T, TPR, VPT, VEC>(a, t, w);
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
    for (int64_t row = (int64_t)blockIdx.x * ROWS + sub; row < a.rows; row += (int64_t)a.groups * ROWS) {
        float h[VPT][8], g[VPT][8], d[VPT][8];
        load_row<T, TPR, VPT, VEC>((const T *)a.x + row * a.x_stride, t, a.n, h);
        load_row<T, TPR, VPT, VEC>((const T *)a.dy + row * a.n, t, a.n, g);
        if (a.dres) {
            load_row<T, TPR, VPT, VEC>((const T *)a.dres + row * a.n, t, a.n, d);
        } else {
#pragma unroll
            for (int i = 0; i < VPT; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) d[i][e] = 0.0f;
        }
        float ss = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                ss = fmaf(h[i][e], h[i][e], ss);
                dot = fmaf(h[i][e], w[i][e] * g[i][e], dot);
            }
        reduce<TPR, false>(ss, dot, sm);
        const float rstd = 1.0f / sqrtf(ss / (float)a.n + a.eps);
        const float c = dot * rstd / (float)a.n;     // mean of w dy against h r
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float x = h[i][e] * rstd;
                dw[i][e] = fmaf(g[i][e], x, dw[i][e]);
                d[i][e] = fmaf(rstd, fmaf(-x, c, w[i][e] * g[i][e]), d[i][e]);
            }
        store_row<T, TPR, VPT, VEC>((T *)a.dx + row * a.n, t, a.n, d);
    }
    float *part = a.part + (int64_t)blockIdx.x * a.n;
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
        store_row<float, TPR, VPT, VEC>(part, t, a.n, dw);
    }
}

// dw = the groups' sums added up: 16 columns per work-group, 64 slices of the
// groups in parallel, the slices joined in LDS.
__global__ void __launch_bounds__(1024) lores_norm_dw_kernel(const NormArgs a) {
    __shared__ float sm[64][17];
    const int c = blockIdx.x * 16 + (threadIdx.x & 15), sl = threadIdx.x >> 4;
    float s = 0.0f;
    if (c < a.n)
        for (int g = sl; g < a.groups; g += 64) s += a.part[(int64_t)g * a.n + c];
    sm[sl][threadIdx.x & 15] = s;
    __syncthreads();
    for (int d = 32; d >= 1; d >>= 1) {
        if (sl < d) sm[sl][threadIdx.x & 15] += sm[sl + d][threadIdx.x & 15];
        __syncthreads();
    }
    if (sl == 0 && c < a.n) a.dw[c] = sm[0][threadIdx.x];
}

template <typename T, int TPR, int VPT>
hipError_t go(bool vec, bool back, const NormArgs &a, hipStream_t s) {
    constexpr int ROWS = TPR < 256 ? 256 / TPR : 1, TH = TPR < 256 ? 256 : TPR;
    const dim3 grid = grid_of(back ? a.groups : (a.rows + ROWS - 1) / ROWS);
    if (back) {
        if (vec) lores_norm_backward_kernel<T, TPR, VPT, true><<<grid, TH, 0, s>>>(a);
        else lores_norm_backward_kernel<T, TPR, VPT, false><<<grid, TH, 0, s>>>(a);
    } else {
        if (vec) lores_norm_kernel<T, TPR, VPT, true><<<grid, TH, 0, s>>>(a);
        else lores_norm_kernel<T, TPR, VPT, false><<<grid, TH, 0, s>>>(a);
    }
    return hipGetLastError();
}

// Threads per row: one or two vectors each.  Measured (us forward / backward,
// bf16): a quarter of the threads with four times the vectors is the same at
// 128 and 8192 elements, 17.2 / 46 instead of 15.3 / 36 at 8192 x 1024 and
// 125 / 217 instead of 92 / 116 at 16384 x 4096, and a small batch (64 x 4096)
// waits 10 instead of 4.6 us; four times the threads with idle ones take 34 instead of 14 us at
// 65536 x 128 and 150 instead of 92 at 16384 x 4096.
template <typename T>
hipError_t by_width(bool vec, bool back, const NormArgs &a, hipStream_t s) {
    if (a.n <= 128) return go<T, 16, 1>(vec, back, a, s);
    if (a.n <= 512) return go<T, 64, 1>(vec, back, a, s);
    if (a.n <= 1024) return go<T, 64, 2>(vec, back, a, s);
    if (a.n <= 2048) return go<T, 256, 1>(vec, back, a, s);
    if (a.n <= 4096) return go<T, 256, 2>(vec, back, a, s);
    if (a.n <= 8192) return go<T, 1024, 1>(vec, back, a, s);
    return go<T, 1024, 2>(vec, back, a, s);
}

}  // namespace

// As many as run at once, or fewer where the groups' sums would then weigh: us
// of both kernels, bf16, without dresidual:
//   rows x n        256    512   1024   2048  work-groups
//   65536 x 128       -   18.7   18.9   23.7
//   8192 x 1024       -   19.0   19.8   28.2
//   16384 x 2048      -   55.6   45.2   51.4
//   16384 x 4096      -      -   90.6   98.6
//   8192 x 8192     109    114      -      -
//   4096 x 16384    102    110      -      -
int norm_groups(int64_t rows, int32_t n) {
    const int side = n <= 128 ? 16 : n <= 1024 ? 4 : 1;      // rows a work-group takes side by side
    const int64_t most = n <= 1024 ? 512 : n <= 4096 ? 1024 : 256, need = (rows + side - 1) / side;
    return (int)(need < most ? need : most);
}

hipError_t launch_norm(bool in_bf16, bool vec, const NormArgs &a, hipStream_t s) {
    return in_bf16 ? by_width<uint16_t>(vec, false, a, s) : by_width<float>(vec, false, a, s);
}

hipError_t launch_norm_backward(bool in_bf16, bool vec, const NormArgs &a, hipStream_t s) {
    if (a.rows) {                                    // without rows dw is a sum of nothing
        const hipError_t e = in_bf16 ? by_width<uint16_t>(vec, true, a, s) : by_width<float>(vec, true, a, s);
        if (e != hipSuccess) return e;
    }
    lores_norm_dw_kernel<<<dim3((unsigned)((a.n + 15) / 16)), 1024, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace lores
