// Rows in registers, as the norms hold them: element access in bf16 or fp32, a
// thread's columns of a row, loads and stores of them, sums over a row's
// threads, and a norm's output in any of its forms.  A row takes TPR threads (8 to 64,
// 256 or 1024) of VPT vectors of 8.
#pragma once

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
    // past the caches' recent lines: for rows that are not read again soon
    static __device__ __forceinline__ void put8_far(float *p, const float *x) {
        __builtin_nontemporal_store(f32x4{x[0], x[1], x[2], x[3]}, (f32x4 *)p);
        __builtin_nontemporal_store(f32x4{x[4], x[5], x[6], x[7]}, (f32x4 *)(p + 4));
    }
    // at any multiple of an element: the hardware takes such addresses
    typedef f32x4 Odd __attribute__((aligned(4)));
    static __device__ __forceinline__ void get8_odd(const float *p, float *x) {
        const f32x4 a = *(const Odd *)p, b = *(const Odd *)(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
    }
    static __device__ __forceinline__ void put8_odd(float *p, const float *x) {
        *(Odd *)p = f32x4{x[0], x[1], x[2], x[3]};
        *(Odd *)(p + 4) = f32x4{x[4], x[5], x[6], x[7]};
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
    static __device__ __forceinline__ u32x4 pack8(const float *x) {
        u32x4 a;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            a[e] = (uint32_t)f2bf(x[2 * e]) | ((uint32_t)f2bf(x[2 * e + 1]) << 16);
        return a;
    }
    static __device__ __forceinline__ void put8(uint16_t *p, const float *x) { *(u32x4 *)p = pack8(x); }
    static __device__ __forceinline__ void put8_far(uint16_t *p, const float *x) {
        __builtin_nontemporal_store(pack8(x), (u32x4 *)p);
    }
    typedef u32x4 Odd __attribute__((aligned(2)));
    static __device__ __forceinline__ void get8_odd(const uint16_t *p, float *x) {
        const u32x4 a = *(const Odd *)p;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[2 * e] = __uint_as_float(a[e] << 16);
            x[2 * e + 1] = __uint_as_float(a[e] & 0xffff0000u);
        }
    }
    static __device__ __forceinline__ void put8_odd(uint16_t *p, const float *x) { *(Odd *)p = pack8(x); }
};

// One thread's elements of a row: VPT vectors of 8.  VEC 1: 8 neighbours per
// vector and thread (16-byte accesses); 0: element e of vector i is 8 i + e
// strides of TPR away, so that neighbouring threads read neighbouring
// elements of rows at any alignment; 2: the columns of 1 in rows of any length
// and alignment (of 8 elements or more), by vectors at odd addresses.  A row's last
// vector then ends with the row, over part of its neighbour's: both compute the same
// there, and only elements from own_from() on count in sums (the others as 0 in every
// factor: 0 times an infinity is none).
template <int TPR, int VEC>
__device__ __forceinline__ int col(int t, int i, int e) {
    return VEC ? (i * TPR + t) * 8 + e : (i * 8 + e) * TPR + t;
}

// vector i of a thread: its first column, and its first element that is not a neighbour's
template <int TPR>
__device__ __forceinline__ int odd_at(int t, int i, int n) { return min((i * TPR + t) * 8, n - 8); }
template <int TPR, int VEC>
__device__ __forceinline__ int own_from(int t, int i, int n) {
    return VEC == 2 && n >= 8 ? (i * TPR + t) * 8 - odd_at<TPR>(t, i, n) : 0;
}

template <typename T, int TPR, int VPT, int VEC>
__device__ __forceinline__ void load_row(const T *p, int t, int n, float (&x)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC == 1) {
            const int c = (i * TPR + t) * 8;
            if (c < n) {
                Elem<T>::get8(p + c, x[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 8; ++e) x[i][e] = 0.0f;
            }
        } else if (VEC == 2 && n >= 8) {
            if ((i * TPR + t) * 8 < n) {
                Elem<T>::get8_odd(p + odd_at<TPR>(t, i, n), x[i]);
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

// vector i of a thread's part of a row (FAR: with VEC 1 by put8_far)
template <typename T, int TPR, int VEC, bool FAR = false>
__device__ __forceinline__ void store_vector(T *p, int t, int i, int n, const float (&x)[8]) {
    if constexpr (VEC == 1) {
        const int c = (i * TPR + t) * 8;
        if (c < n) {
            if constexpr (FAR) Elem<T>::put8_far(p + c, x);
            else Elem<T>::put8(p + c, x);
        }
    } else {
        if (VEC == 2 && n >= 8) {
            if ((i * TPR + t) * 8 < n) Elem<T>::put8_odd(p + odd_at<TPR>(t, i, n), x);
            return;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int c = col<TPR, VEC>(t, i, e);
            if (c < n) Elem<T>::put(p + c, x[e]);
        }
    }
}

template <typename T, int TPR, int VPT, int VEC, bool FAR = false>
__device__ __forceinline__ void store_row(T *p, int t, int n, const float (&x)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) store_vector<T, TPR, VEC, FAR>(p, t, i, n, x[i]);
}

template <int TPR, int VPT, int VEC>
__device__ __forceinline__ void store_bytes(uint8_t *p, int t, int n, const uint8_t (&x)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        if constexpr (VEC == 1) {
            const int c = (i * TPR + t) * 8;
            u32x2 w = {0, 0};
#pragma unroll
            for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)x[i][e] << (8 * (e & 3));
            if (c < n) *(u32x2 *)(p + c) = w;
        } else {
            if (VEC == 2 && n >= 8) {
                typedef u32x2 Odd __attribute__((aligned(1)));
                u32x2 w = {0, 0};
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e >> 2] |= (uint32_t)x[i][e] << (8 * (e & 3));
                if ((i * TPR + t) * 8 < n) *(Odd *)(p + odd_at<TPR>(t, i, n)) = w;
                continue;
            }
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


// The sum of `a` over one row's threads, in every one of them.
template <int TPR>
__device__ __forceinline__ float row_sum(float a, float (*sm)[2]) {
    constexpr int W = TPR < 64 ? TPR : 64;
#pragma unroll
    for (int d = 1; d < W; d <<= 1) a += __shfl_xor(a, d);
    if constexpr (TPR > 64) {
        __syncthreads();                             // the last row's values have been read
        if ((threadIdx.x & 63) == 0) sm[threadIdx.x >> 6][0] = a;
        __syncthreads();
        a = sm[0][0];
#pragma unroll
        for (int i = 1; i < TPR / 64; ++i) a += sm[i][0];
    }
    return a;
}

template <int TPR, int VPT, int VEC>
__device__ __forceinline__ void load_either(const void *p, int bf16, int t, int n, float (&w)[VPT][8]) {
    if (bf16) load_row<uint16_t, TPR, VPT, VEC>((const uint16_t *)p, t, n, w);
    else load_row<float, TPR, VPT, VEC>((const float *)p, t, n, w);
}

// A thread's part of a row as it lies in memory: a bf16 row that waits for its
// turn takes half the registers.
template <typename T> struct Kept;
template <> struct Kept<float> {
    float x[8];
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = v[e];
    }
    __device__ __forceinline__ float at(int e) const { return x[e]; }
    template <bool FAR> __device__ __forceinline__ void read(const float *p) {
        const f32x4 *q = (const f32x4 *)p;
        const f32x4 a = FAR ? __builtin_nontemporal_load(q) : *q, b = FAR ? __builtin_nontemporal_load(q + 1) : q[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
    }
    __device__ __forceinline__ void read_odd(const float *p) { Elem<float>::get8_odd(p, x); }
};
template <> struct Kept<uint16_t> {
    u32x4 x;
    __device__ __forceinline__ void set(const float (&v)[8]) {
#pragma unroll
        for (int e = 0; e < 4; ++e)                  // the values are bf16 already
            x[e] = (__float_as_uint(v[2 * e]) >> 16) | (__float_as_uint(v[2 * e + 1]) & 0xffff0000u);
    }
    __device__ __forceinline__ float at(int e) const {
        return __uint_as_float(e & 1 ? x[e >> 1] & 0xffff0000u : x[e >> 1] << 16);
    }
    template <bool FAR> __device__ __forceinline__ void read(const uint16_t *p) {
        x = FAR ? __builtin_nontemporal_load((const u32x4 *)p) : *(const u32x4 *)p;
    }
    __device__ __forceinline__ void read_odd(const uint16_t *p) { x = *(const Elem<uint16_t>::Odd *)p; }
};

// (FAR: with VEC 1 past the caches' recent lines, as put8_far)
template <typename T, int TPR, int VPT, int VEC, bool FAR = false>
__device__ __forceinline__ void keep_row(const T *p, int t, int n, Kept<T> (&k)[VPT]) {
    if constexpr (VEC == 1) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int c = (i * TPR + t) * 8;
            if (c < n) {
                k[i].template read<FAR>(p + c);
            } else {
                const float zero[8] = {};
                k[i].set(zero);
            }
        }
    } else if (VEC == 2 && n >= 8) {
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const float zero[8] = {};
            if ((i * TPR + t) * 8 < n) k[i].read_odd(p + odd_at<TPR>(t, i, n));
            else k[i].set(zero);
        }
    } else {
        float x[VPT][8];
        load_row<T, TPR, VPT, VEC>(p, t, n, x);
#pragma unroll
        for (int i = 0; i < VPT; ++i) k[i].set(x[i]);
    }
}

// ------------------------------------------------------------ 4-bit blocks
//
// 32 neighbours of a row share the scale 2^e: the smallest power of two with
// max |x| < 7 2^e, so that the largest value is rounded (to 6 at most), never
// cut off.  In the bits of the maximum: its exponent, one more if the mantissa
// is at least 1.75, less the grid's top exponent 2.  The scale's byte is
// e + 127, at least 0 (e >= -127), and 255 (NaN) for a block that holds a value
// that is not finite.
__device__ __forceinline__ uint32_t mx_scale(uint32_t max_bits) {
    return max_bits >= 0x7f800000u ? 255u : max((max_bits + (1u << 21)) >> 23, 2u) - 2u;
}

// 8 values as E2M1 codes (nearest, ties to the even code), the first in the low
// half of the first byte.  The product with 2^-e is exact.
__device__ __forceinline__ uint32_t mx_codes(const float (&x)[8], uint32_t scale) {
    if (scale == 255u) return 0;
    const float inv = __uint_as_float((254u - scale) << 23);
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0] * inv, x[1] * inv, 1.0f, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2] * inv, x[3] * inv, 1.0f, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4] * inv, x[5] * inv, 1.0f, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6] * inv, x[7] * inv, 1.0f, 3);
    return w;
}

// The largest magnitude of 8 values, as bits: a NaN is above all numbers there.
__device__ __forceinline__ uint32_t max_bits8(const float (&x)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(fabsf(x[e])));
    return m;
}

// A row in registers (VEC 1 or 2: 8 neighbours a thread, a block in 4 threads)
// as codes and scales; `pad` bytes of 0 behind the scales.
template <int TPR, int VPT>
__device__ __forceinline__ void store_mx(uint8_t *codes, uint8_t *scales, int pad, int t, int n, bool lost,
                                         const float (&y)[VPT][8]) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int c = (i * TPR + t) * 8;
        uint32_t m = max_bits8(y[i]);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        const uint32_t s = lost ? 255u : mx_scale(m);
        const uint32_t w = mx_codes(y[i], s);
        if (c < n) {
            *(uint32_t *)(codes + c / 2) = w;
            if ((t & 3) == 0) scales[c / 32] = (uint8_t)s;
        }
    }
    if (t == 0)
        for (int i = 0; i < pad; ++i) scales[n / 32 + i] = 0;
}

// ------------------------------------------------------------ a norm's output

// A row of z = h w with the row's sum of h^2 and largest |z| (infinite for a
// NaN): y in fp32 or bf16, 8-bit codes with a scale, or 4-bit blocks.
template <int TPR, int VPT, int VEC, bool MX, bool FAR = false>
__device__ __forceinline__ void norm_store(void *y, void *scales, int out_prec, int64_t row, int t, int n, float sum,
                                           float mx, float rstd, float (&z)[VPT][8]) {
    const float inf = __builtin_inff();
    // a z that is not finite, or squares beyond fp32
    const bool lost = !(mx < inf) || !(sum < inf);
    if (out_prec == LORES_FP32 || out_prec == LORES_BF16 || (MX && out_prec == LORES_MXFP4)) {
#pragma unroll
        for (int i = 0; i < VPT; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) z[i][e] = z[i][e] * rstd;
        if (out_prec == LORES_FP32)
            store_row<float, TPR, VPT, VEC, FAR>((float *)y + row * n, t, n, z);
        else if (out_prec == LORES_BF16)
            store_row<uint16_t, TPR, VPT, VEC, FAR>((uint16_t *)y + row * n, t, n, z);
        else if constexpr (MX && VEC != 0) {
            const int per = mx_scale_stride(n);
            // (without an epsilon the r of a row of zeros is an infinity: its y are 0)
            if (mx == 0.0f) {
#pragma unroll
                for (int i = 0; i < VPT; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) z[i][e] = 0.0f;
            }
            store_mx<TPR, VPT>((uint8_t *)y + row * (n / 2), (uint8_t *)scales + row * per, per - n / 32, t, n,
                               lost, z);
        }
        return;
    }
    const float top = out_prec == LORES_INT8 ? 127.0f : 448.0f;
    // a lost row has the scale NaN and the codes 0
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
            const float x = z[i][e] * inv;
            if (out_prec == LORES_INT8) {
                const float q = rintf(fminf(fmaxf(x, -127.0f), 127.0f));
                c[i][e] = x == x ? (uint8_t)(int8_t)(int)q : (uint8_t)0;
            } else {
                const float q = fminf(fmaxf(x, -448.0f), 448.0f);
                c[i][e] = x == x ? (uint8_t)__builtin_amdgcn_cvt_pk_fp8_f32(q, q, 0, false)
                                 : (uint8_t)0;
            }
        }
    store_bytes<TPR, VPT, VEC>((uint8_t *)y + row * n, t, n, c);
    // (without an epsilon the r of a row of zeros is an infinity)
    if (t == 0) ((float *)scales)[row] = lost ? nan : mx == 0.0f ? 0.0f : m / top * rstd;
}

}  // namespace
}  // namespace lores
