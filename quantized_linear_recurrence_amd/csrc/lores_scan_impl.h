// Device pieces shared by the chunked scan kernels (lores_scan_prep / state /
// back / grad .hip).
//
// A chunk is C tokens of one (sequence, head).  With D_ij = prod_{j<l<=i}
// alpha_l, gamma_i = D_i0, S the state the chunk starts from (value rows x
// keys) and S_C the one it leaves:
//   M_ij = (k_i . k_j) D_ij (i > j),   P_ij = (q_i . k_j) D_ij (i >= j)
//   X = (I + delta diag(beta) M)^-1,   U = X diag(beta) (V - delta gamma K S^T)
//   O = gamma Q S^T + P U,             S_C = gamma_C S + sum_j D_Cj u_j k_j^T
// Decays are products of the alphas between two tokens, never quotients or
// differences of logarithms: a decay of 0 is an ordinary value, and nothing
// under- or overflows that the recurrence itself would keep.
//
// Products run on the bf16 matrix instructions.  An fp32 operand is split
// into bf16 planes x = p0 + p1 + p2 (8 bits of significand each, |x - p0| <=
// 2^-9 |x|, and so on), a bf16 one is its own only plane; a product of planes
// i and j is kept for i + j < ORD.  ORD = 3 (six products of two fp32
// operands, three of an fp32 with a bf16 one) leaves out less than 2^-24 of
// a term: fp32 accuracy at 2.7 to 5.3 times the rate of the fp32 matrix
// instructions.  ORD = 2 leaves out 2^-17, for sums that end in bf16.
#pragma once

#include "lores_seq.h"

namespace lores {
namespace scan {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 b16x8 __attribute__((ext_vector_type(8)));

// Chunk length and planes of an input type: fp32 operands take three times
// the LDS, so their chunks are half as long.
template <typename IN> struct Cfg;
template <> struct Cfg<uint16_t> { static constexpr int C = 64, NIN = 1; };
template <> struct Cfg<float> { static constexpr int C = 32, NIN = 3; };

__device__ __forceinline__ float bf2f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f2bf(float f) {
    const __bf16 b = (__bf16)f;                      // to nearest even
    return __builtin_bit_cast(uint16_t, b);
}
__device__ __forceinline__ float get1(const float *p) { return *p; }
__device__ __forceinline__ float get1(const uint16_t *p) { return bf2f(*p); }
__device__ __forceinline__ void put1(float *p, float x) { *p = x; }
__device__ __forceinline__ void put1(uint16_t *p, float x) { *p = f2bf(x); }

// 16 bytes to memory, from ordinary vector registers (the state lives in the
// accumulation registers where a kernel needs more than 256)
__device__ __forceinline__ void store4(float *p, f32x4 x) {
    asm volatile("" : "+v"(x));
    *(f32x4 *)p = x;
}

// x = p[0] + p[1] + ... up to the last plane's rounding
template <int NP>
__device__ __forceinline__ void split8(const float (&x)[8], b16x8 (&p)[NP]) {
    float r[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) r[e] = x[e];
#pragma unroll
    for (int i = 0; i < NP; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[i][e] = (__bf16)r[e];
            if (i + 1 < NP) r[e] -= (float)p[i][e];
        }
}

// 8 neighbours of a row at p, the first `n` of which exist (vec: 16-byte
// aligned and n is 0 or 8 or more)
__device__ __forceinline__ void get8(const float *p, int n, bool vec, float (&x)[8]) {
    if (vec && n >= 8) {
        const f32x4 a = *(const f32x4 *)p, b = *(const f32x4 *)(p + 4);
#pragma unroll
        for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = e < n ? p[e] : 0.0f;
    }
}
__device__ __forceinline__ void get_planes(const float *p, int n, bool vec, b16x8 (&o)[3]) {
    float x[8];
    get8(p, n, vec, x);
    split8(x, o);
}
__device__ __forceinline__ void get_planes(const uint16_t *p, int n, bool vec, b16x8 (&o)[1]) {
    if (vec && n >= 8) {
        o[0] = __builtin_bit_cast(b16x8, *(const u32x4 *)p);
    } else {
        s16x8 w;
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = e < n ? (short)p[e] : (short)0;
        o[0] = __builtin_bit_cast(b16x8, w);
    }
}

__device__ __forceinline__ f32x4 mfma(b16x8 a, b16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// c += a b over the planes' products i + j < ORD, the smallest first
template <int ORD, int NA, int NB>
__device__ __forceinline__ f32x4 mma(const b16x8 (&a)[NA], const b16x8 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int o = ORD - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i <= o; ++i)
            if (i < NA && o - i < NB) c = mfma(a[i], b[o - i], c);
    return c;
}

// An LDS matrix of bf16 planes, [NP][R][LD]; rows are 16-byte aligned and
// start in different banks.
template <int NP, int R, int W>
struct Planes {
    static constexpr int LD = W + 8;
    uint16_t x[NP][R][LD];
    // operand whose lane holds row `row`, columns c .. c + 7
    template <int N>
    __device__ __forceinline__ void rows(int row, int c, b16x8 (&o)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = *(const b16x8 *)&x[i][row][c];
    }
    // operand whose lane holds 8 rows r0 + 8 g .. + 7 (g = lane / 16) of one
    // column: the transposing read hands lane i of 16 the column i of the
    // 4 x 16 block that the lanes address (lane i: row i / 4, columns 4 (i % 4)
    // on).  STEP: those groups of four columns lie STEP columns apart.
    template <int STEP, int N>
    __device__ __forceinline__ void cols(int r0, int c0, int lane, b16x8 (&o)[N]) const {
        const int i = lane & 15, r = r0 + 8 * (lane >> 4) + (i >> 2), c = c0 + STEP * (i & 3);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)&x[k][r][c]);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)&x[k][r + 4][c]);
            const s16x8 w = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            o[k] = __builtin_bit_cast(b16x8, w);
        }
    }
    template <int N>
    __device__ __forceinline__ void put8(int row, int c, const b16x8 (&o)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) *(b16x8 *)&x[i][row][c] = o[i];
    }
    __device__ __forceinline__ float at(int row, int c) const {
        float s = bf2f(x[0][row][c]);
#pragma unroll
        for (int i = 1; i < NP; ++i) s += bf2f(x[i][row][c]);
        return s;
    }
    __device__ __forceinline__ void put(int row, int c, float v) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            x[i][row][c] = f2bf(v);
            if (i + 1 < NP) v -= bf2f(x[i][row][c]);
        }
    }
};

// The tokens that a matrix instruction's 16 result rows stand for where the
// result is the next product's operand from registers: lane group g of tile
// mt holds rows 4 g + r, and an operand of 32 tokens wants 8 neighbours per
// lane group, so tiles 2 s and 2 s + 1 take the tokens of block s as 32 s +
// 8 g + 4 (mt & 1) + r.
__device__ __forceinline__ int token_of(int mt, int m) {
    return 32 * (mt >> 1) + 8 * (m >> 2) + 4 * (mt & 1) + (m & 3);
}

// Decays of one chunk, computed by one wavefront's first C lanes.
template <int C>
struct Gates {
    float al[C];     // alpha (1 behind the sequence's end)
    float be[C];     // beta (0 behind it)
    float gam[C];    // gamma_i = alpha_0 .. alpha_i of the chunk
    float end[C];    // D_Cj: alpha_{j+1} .. alpha_{C-1}
    __device__ __forceinline__ void load(const float *alpha, const float *beta, int64_t stride,
                                         int n, int lane) {
        if (lane >= C) return;
        const float a = lane < n ? alpha[lane * stride] : 1.0f;
        const float b = lane < n ? beta[lane * stride] : 0.0f;
        float g = a, e = a;
#pragma unroll
        for (int d = 1; d < C; d <<= 1) {
            const float x = __shfl_up(g, d, C), y = __shfl_down(e, d, C);
            if (lane >= d) g *= x;
            if (lane + d < C) e *= y;
        }
        e = __shfl_down(e, 1, C);
        al[lane] = a;
        be[lane] = b;
        gam[lane] = g;
        end[lane] = lane == C - 1 ? 1.0f : e;
    }
};

// D_ij of the 16 x 16 tile (mt, nt <= mt) for the lane's column j = 16 nt +
// (lane & 15) and rows i = 16 mt + 4 (lane / 16) + r; zero above the diagonal.
// Each is a product of the alphas between, in an order that depends on the
// tile alone.
template <int C>
__device__ __forceinline__ void decay_tile(const Gates<C> &g, int mt, int nt, int lane, float (&d)[4]) {
    const int j = 16 * nt + (lane & 15), i0 = 16 * mt + 4 * (lane >> 4);
    float x = 1.0f;
    if (nt < mt) {
        for (int l = 16 * nt + 1; l < 16 * mt; ++l) x *= l > j ? g.al[l] : 1.0f;
        for (int l = 16 * mt; l < i0; ++l) x *= g.al[l];
    } else {
        for (int l = 16 * mt + 1; l < i0; ++l) x *= l > j ? g.al[l] : 1.0f;
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) {
        if (i0 + r > j) x *= g.al[i0 + r];
        d[r] = i0 + r >= j ? x : 0.0f;
    }
}

// Rows of q or k: C tokens from t0, zeros behind the sequence's end and d_k.
template <typename IN, int NP, int R, int W>
__device__ __forceinline__ void stage_rows(Planes<NP, R, W> &dst, const IN *src, int64_t tok_stride,
                                           int n, int dk, bool vec, int tid, int threads) {
    for (int x = tid; x < R * (W / 8); x += threads) {
        const int row = x / (W / 8), c = (x % (W / 8)) * 8;
        b16x8 p[NP];
        get_planes(src + row * tok_stride + c, row < n ? dk - c : 0, vec, p);
        dst.put8(row, c, p);
    }
}

// A [NP][R][W] block of planes in memory, rows of W elements without padding.
template <int NP, int R, int W>
__device__ __forceinline__ void stage_planes(Planes<NP, R, W> &dst, const uint16_t *src, int tid,
                                             int threads) {
    for (int x = tid; x < NP * R * (W / 8); x += threads) {
        const int pl = x / (R * (W / 8)), y = x % (R * (W / 8)), row = y / (W / 8), c = (y % (W / 8)) * 8;
        *(u32x4 *)&dst.x[pl][row][c] = *(const u32x4 *)(src + (int64_t)(pl * R + row) * W + c);
    }
}

}  // namespace scan
}  // namespace lores
