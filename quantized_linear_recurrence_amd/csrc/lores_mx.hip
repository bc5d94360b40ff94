// Rows to microscaled 4-bit blocks (lores_mx_quant) and back (lores_mx_dequant).
//   e = the smallest power of two, at least 2^-127, with max |x| < 7 2^e over 32 neighbours,
//   code = x 2^-e rounded to the nearest E2M1 value
//
// Bound by memory.  A thread takes 8 neighbours (16 bytes of bf16, 4 bytes of
// codes), a block lies in 4 threads; a row's threads are a power of two that
// leaves few of them idle, and a thread has the same columns of 4 rows in flight.
// 8192 x 4096 bf16: 17 us, 5.0 TB/s, and back 14, 6.2 TB/s; fp32 30, 5.0 TB/s, and 25, 6.1 TB/s.
#include "lores_layer.h"
#include "lores_rows.h"

namespace lores {
namespace {

constexpr int kRows = 4;

struct Shape {
    int32_t log_threads;               // threads of a row
    int32_t chunks;                    // work-groups along a row
};

// The widest of 4 .. 256 threads whose idle share is at most an eighth (4, a block's, leave none idle).
Shape shape_of(int32_t n) {
    const int32_t pieces = n / 8;
    int32_t l = 8;
    while ((((int64_t)pieces + (1 << l) - 1) >> l << l) * 7 > (int64_t)pieces * 8) --l;
    return {l, (pieces + (1 << l) - 1) >> l};
}

__device__ __forceinline__ void place(const MxRows &a, const Shape &sh, int64_t &row, int &c) {
    const int64_t b = block_at(blockIdx.x, blockIdx.y), rb = b / sh.chunks;
    const int chunk = (int)(b - rb * sh.chunks);
    row = rb * (kRows << (8 - sh.log_threads)) + (threadIdx.x >> sh.log_threads);
    c = ((chunk << sh.log_threads) + (threadIdx.x & ((1 << sh.log_threads) - 1))) * 8;
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) lores_mx_quant_kernel(const MxRows a, const Shape sh) {
    int64_t row0;
    int c;
    place(a, sh, row0, c);
    const int step = 256 >> sh.log_threads, per = mx_scale_stride(a.n);
    float x[kRows][8];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t row = row0 + i * step;
        const T *p = (const T *)a.x + row * a.xs + c;
        const bool in = row < a.rows && c < a.n;
        if (in && VEC) {
            Elem<T>::get8(p, x[i]);
        } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[i][e] = in ? Elem<T>::get(p + e) : 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t row = row0 + i * step;
        uint32_t m = max_bits8(x[i]);
        m = max(m, (uint32_t)__shfl_xor((int)m, 1));
        m = max(m, (uint32_t)__shfl_xor((int)m, 2));
        const uint32_t s = mx_scale(m), w = mx_codes(x[i], s);
        if (row >= a.rows || c >= a.n) continue;
        *(uint32_t *)(a.codes + row * (a.n / 2) + c / 2) = w;
        uint8_t *to = a.scales + row * per + c / 32;
        if ((c & 31) == 0) *to = (uint8_t)s;
        if (c + 8 == a.n)                            // zeros behind the last block
            for (int k = a.n / 32; k < per; ++k) a.scales[row * per + k] = 0;
    }
}

template <typename T>
__global__ void __launch_bounds__(256) lores_mx_dequant_kernel(const MxRows a, const Shape sh) {
    int64_t row0;
    int c;
    place(a, sh, row0, c);
    const int step = 256 >> sh.log_threads, per = mx_scale_stride(a.n);
    uint32_t w[kRows], s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t row = row0 + i * step;
        const bool in = row < a.rows && c < a.n;
        w[i] = in ? *(const uint32_t *)(a.codes + row * (a.n / 2) + c / 2) : 0;
        s[i] = in ? a.scales[row * per + c / 32] : 0;
    }
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        const int64_t row = row0 + i * step;
        if (row >= a.rows || c >= a.n) continue;
        // 2^(s - 127); s = 0 is below the normal numbers, 255 is NaN
        const float f = __uint_as_float(s[i] == 0 ? 0x00400000u : s[i] == 255 ? 0x7fc00000u : s[i] << 23);
        const auto p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0);
        const auto p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1);
        const auto p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2);
        const auto p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3);
        const float y[8] = {p0[0] * f, p0[1] * f, p1[0] * f, p1[1] * f, p2[0] * f, p2[1] * f, p3[0] * f, p3[1] * f};
        Elem<T>::put8((T *)a.out + row * a.n + c, y);
    }
}

dim3 grid_for(const MxRows &a, const Shape &sh) {
    const int64_t side = kRows << (8 - sh.log_threads);
    return grid_of((a.rows + side - 1) / side * sh.chunks);
}

}  // namespace

hipError_t launch_mx_quant(bool in_bf16, bool vec, const MxRows &a, hipStream_t s) {
    const Shape sh = shape_of(a.n);
    const dim3 grid = grid_for(a, sh);
    if (in_bf16) {
        if (vec) lores_mx_quant_kernel<uint16_t, true><<<grid, 256, 0, s>>>(a, sh);
        else lores_mx_quant_kernel<uint16_t, false><<<grid, 256, 0, s>>>(a, sh);
    } else {
        if (vec) lores_mx_quant_kernel<float, true><<<grid, 256, 0, s>>>(a, sh);
        else lores_mx_quant_kernel<float, false><<<grid, 256, 0, s>>>(a, sh);
    }
    return hipGetLastError();
}

hipError_t launch_mx_dequant(bool out_bf16, const MxRows &a, hipStream_t s) {
    const Shape sh = shape_of(a.n);
    const dim3 grid = grid_for(a, sh);
    if (out_bf16) lores_mx_dequant_kernel<uint16_t><<<grid, 256, 0, s>>>(a, sh);
    else lores_mx_dequant_kernel<float><<<grid, 256, 0, s>>>(a, sh);
    return hipGetLastError();
}

}  // namespace lores
