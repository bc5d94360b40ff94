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

#include "lores_direct.h"
#include "lores_seq.h"

namespace lores {
namespace scan {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
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

// Two values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 b16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, b16x2));
}

// Four neighbours of a row to memory (vec: the address is a multiple of their
// size; four words need no more than their own alignment).
__device__ __forceinline__ void put4(float *p, f32x4 v, bool) {
    // the instruction itself: the compiler would store these results from
    // accumulation registers.  The wait state keeps the data registers from
    // being rewritten before the store has read them.
    asm volatile("global_store_dwordx4 %0, %1, off\n\ts_nop 0" :: "v"(p), "v"(v) : "memory");
}
__device__ __forceinline__ void put4(uint16_t *p, f32x4 v, bool vec) {
    const u32x2 w = {pack2(v[0], v[1]), pack2(v[2], v[3])};
    if (vec) {
        *(u32x2 *)p = w;
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
    }
}

// x = p[0] + p[1] + ... up to the last plane's rounding
template <int NP>
__device__ __forceinline__ void split8(const float (&x)[8], b16x8 (&p)[NP]) {
    u32x4 w[NP];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        float a = x[2 * e], b = x[2 * e + 1];
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            w[i][e] = pack2(a, b);
            if (i + 1 < NP) {
                a -= __uint_as_float(w[i][e] << 16);
                b -= __uint_as_float(w[i][e] & 0xffff0000u);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < NP; ++i) p[i] = __builtin_bit_cast(b16x8, w[i]);
}

// The planes of four values, each handed to put(plane, bits).
template <int NP, typename F>
__device__ __forceinline__ void split4(const float (&v)[4], F put) {
    float a[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        const u32x2 w = {pack2(a[0], a[1]), pack2(a[2], a[3])};
        put(i, w);
        if (i + 1 < NP) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                a[e] -= __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
        }
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

// c += a b over the planes' products i + j < 3, the smallest first
template <int NA, int NB>
__device__ __forceinline__ f32x4 mma(const b16x8 (&a)[NA], const b16x8 (&b)[NB], f32x4 c) {
#pragma unroll
    for (int o = 2; o >= 0; --o)
#pragma unroll
        for (int i = 0; i <= o; ++i)
            if (i < NA && o - i < NB) c = mfma(a[i], b[o - i], c);
    return c;
}

// The same for MT results at once: products of planes outermost, so that
// neighbouring instructions add to different results.
template <int MT, int NA, int NB>
__device__ __forceinline__ void mma_all(const b16x8 (*a)[NA], const b16x8 (&b)[NB], f32x4 *c) {
#pragma unroll
    for (int o = 2; o >= 0; --o)
#pragma unroll
        for (int i = 0; i <= o; ++i)
            if (i < NA && o - i < NB) {
#pragma unroll
                for (int t = 0; t < MT; ++t) c[t] = mfma(a[t][i], b[o - i], c[t]);
            }
}

// Nothing is scheduled across: LDS reads written before it are in flight
// while what stands behind it runs.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Order of what stands before it back to the last fence: N times a matrix
// instruction, then V vector instructions.  A wavefront issues in order and a
// matrix instruction occupies its unit for 16 cycles, the time of four vector
// instructions: the splitting of one operand hides behind the products of
// another.
template <int N, int V>
__device__ __forceinline__ void mix() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x2, V, 0);
    }
}

// Two neighbouring result tiles as one operand's 8 values.
__device__ __forceinline__ void pair8(const f32x4 &a, const f32x4 &b, float (&x)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[4 + i] = b[i]; }
}

// The order of a row's 16-byte pieces in LDS: piece j lies at j ^ turn(row),
// so that the 16 rows a matrix operand reads at one piece (rows 8 a + 4 p + b of
// a block of 32, p fixed) hit different banks, without padding: 64 lanes'
// 16-byte direct loads land in LDS one behind the other.  Rows r and r + 4 of
// an aligned 8 turn alike.
template <int W>
__device__ __forceinline__ constexpr int turn(int r) {
    return W >= 128 ? 4 * ((r >> 3) & 3) + (r & 3)
           : W == 64 ? 2 * ((r >> 3) & 3) + ((r >> 1) & 1) : (r >> 3) & 3;
}

// Sum over the 16 lanes of a row, in all of them.
__device__ __forceinline__ float sum16(float x) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int v = __float_as_int(x);
        const int r = i == 0 ? __builtin_amdgcn_update_dpp(0, v, 0x128, 0xf, 0xf, true)     // row_ror:8
                      : i == 1 ? __builtin_amdgcn_update_dpp(0, v, 0x124, 0xf, 0xf, true)
                      : i == 2 ? __builtin_amdgcn_update_dpp(0, v, 0x122, 0xf, 0xf, true)
                               : __builtin_amdgcn_update_dpp(0, v, 0x121, 0xf, 0xf, true);
        x += __int_as_float(r);
    }
    return x;
}

// An LDS matrix of bf16 planes, R rows of W.
template <int NP, int R, int W>
struct Planes {
    uint16_t x[NP][R * W];
    static __device__ __forceinline__ int at_(int row, int c) {
        return row * W + (((c >> 3) ^ turn<W>(row)) << 3) + (c & 7);
    }
    // operand whose lane holds row `row`, columns c .. c + 7
    template <int N>
    __device__ __forceinline__ void rows(int row, int c, b16x8 (&o)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = *(const b16x8 *)&x[i][at_(row, c)];
    }
    // operand whose lane holds 8 rows r0 + 8 g .. + 7 (g = lane / 16) of one
    // column: the transposing read hands lane i of 16 the column i of the
    // 4 x 16 block that the lanes address (lane i: row i / 4, columns 4 (i % 4)
    // on).  STEP: those groups of four columns lie STEP columns apart.
    template <int STEP, int N>
    __device__ __forceinline__ void cols(int r0, int c0, int lane, b16x8 (&o)[N]) const {
        const int i = lane & 15, r = r0 + 8 * (lane >> 4) + (i >> 2), c = c0 + STEP * (i & 3);
        const int at = at_(r, c);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)&x[k][at]);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)&x[k][at + 4 * W]);
            const s16x8 w = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            o[k] = __builtin_bit_cast(b16x8, w);
        }
    }
    template <int N>
    __device__ __forceinline__ void put8(int row, int c, const b16x8 (&o)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) *(b16x8 *)&x[i][at_(row, c)] = o[i];
    }
    // four neighbours c .. c + 3 of a row (c a multiple of 4)
    __device__ __forceinline__ f32x4 get4(int row, int c) const {
        const int at = at_(row, c);
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const u32x2 w = *(const u32x2 *)&x[k][at];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                s[e] += __uint_as_float(e & 1 ? w[e >> 1] & 0xffff0000u : w[e >> 1] << 16);
        }
        return s;
    }
    __device__ __forceinline__ void put4(int row, int c, const float (&v)[4]) {
        split4<NP>(v, [&](int i, u32x2 w) { *(u32x2 *)&x[i][at_(row, c)] = w; });
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

// Gates of one chunk: the prep kernel makes them and keeps them in the
// workspace for the others.
template <int C>
struct Gates {
    float al[C];     // alpha (1 behind the sequence's end)
    float be[C];     // beta (0 behind it)
    float gam[C];    // gamma_i = alpha_0 .. alpha_i of the chunk
    float end[C];    // D_Cj: alpha_{j+1} .. alpha_{C-1}
    // within the 16-token strips, for D_ij between tokens of different strips:
    // pre_i (the strips between, multiplied up) suf_j
    float pre[C];    // alpha from the strip's first token to i
    float suf[C];    // alpha behind j to the strip's last token
};

// Inclusive products over the lanes before (UP) or behind, in groups of W.
template <int W, bool UP>
__device__ __forceinline__ float scan_product(float x, int lane) {
#pragma unroll
    for (int d = 1; d < W; d <<= 1) {
        const float y = UP ? __shfl_up(x, d, W) : __shfl_down(x, d, W);
        const int l = lane & (W - 1);
        if (UP ? l >= d : l + d < W) x *= y;
    }
    return x;
}

// One wavefront's share `part` of 4 of a chunk's gates, from the lane's alpha
// and beta (of token lane mod C; 1 and 0 behind the sequence's end).
template <int C>
__device__ __forceinline__ void make_gates(Gates<C> &g, int part, float a, float b, int lane) {
    const int l = lane & (C - 1);
    if (part == 0) {
        const float x = scan_product<C, true>(a, lane);
        if (lane < C) { g.al[l] = a; g.be[l] = b; g.gam[l] = x; }
    } else if (part == 1) {
        const float x = __shfl_down(scan_product<C, false>(a, lane), 1, C);
        if (lane < C) g.end[l] = l == C - 1 ? 1.0f : x;
    } else if (part == 2) {
        const float x = scan_product<16, true>(a, lane);
        if (lane < C) g.pre[l] = x;
    } else {
        const float x = __shfl_down(scan_product<16, false>(a, lane), 1, 16);
        if (lane < C) g.suf[l] = (l & 15) == 15 ? 1.0f : x;
    }
}

// D_ij of the tile (mt, nt <= mt) turned over: the lane's row i = 16 mt + (lane &
// 15) and columns j = 16 nt + 4 (lane / 16) + r; zero where j > i.
template <int C>
__device__ __forceinline__ void decay_turned(const Gates<C> &g, int mt, int nt, int lane, float (&d)[4]) {
    const int m = lane & 15, q = lane >> 4, i = 16 * mt + m;
    if (nt < mt) {
        float x = g.pre[i];
        for (int k = nt + 1; k < mt; ++k) x *= g.pre[16 * k + 15];
        const f32x4 sj = *(const f32x4 *)&g.suf[16 * nt + 4 * q];
#pragma unroll
        for (int r = 0; r < 4; ++r) d[r] = x * sj[r];
    } else {
        float x = 1.0f;
#pragma unroll
        for (int l = 4; l < 16; ++l) {
            const float al = g.al[16 * mt + l];
            if (l >= 4 * q + 4 && l <= m) x *= al;
        }
        const f32x4 al = *(const f32x4 *)&g.al[16 * mt + 4 * q];
#pragma unroll
        for (int r = 3; r >= 0; --r) {
            d[r] = 4 * q + r <= m ? x : 0.0f;
            if (4 * q + r <= m) x *= al[r];
        }
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

// The lower triangle of a C x C matrix of bf16 planes in blocks of 32 x 32,
// block (I, J <= I) at I (I + 1) / 2 + J: what X and P are in memory and in LDS.
// The operand reads of a block take whole 256-byte groups of its 64-byte rows,
// so they need no padding.
__host__ __device__ constexpr int tri_blocks(int C) { return (C / 32) * (C / 32 + 1) / 2; }
__device__ __forceinline__ constexpr int tri_block(int I, int J) { return I * (I + 1) / 2 + J; }

template <int NP, int C>
struct Tri {
    static constexpr int NB = tri_blocks(C);
    uint16_t x[NP][NB][32][32];
    // rows `row` of block (I, J), columns 8 g .. 8 g + 7
    template <int N>
    __device__ __forceinline__ void rows(int I, int J, int row, int g, b16x8 (&o)[N]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = *(const b16x8 *)&x[i][tri_block(I, J)][row][8 * g];
    }
    // the transpose's: 8 rows 8 g .. + 7 of one column of block (I, J) (see Planes::cols)
    // four neighbours of one row, as planes
    __device__ __forceinline__ void put4(int I, int J, int row, int c, const float (&v)[4]) {
        split4<NP>(v, [&](int i, u32x2 w) { *(u32x2 *)&x[i][tri_block(I, J)][row][c] = w; });
    }
    template <int STEP, int N>
    __device__ __forceinline__ void cols(int I, int J, int c0, int lane, b16x8 (&o)[N]) const {
        const int i = lane & 15, r = 8 * (lane >> 4) + (i >> 2), c = c0 + STEP * (i & 3);
#pragma unroll
        for (int k = 0; k < N; ++k) {
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)&x[k][tri_block(I, J)][r][c]);
            const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)&x[k][tri_block(I, J)][r + 4][c]);
            const s16x8 w = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
            o[k] = __builtin_bit_cast(b16x8, w);
        }
    }
};

// The same triangle in fp32, on its way from the prep kernel to the forward pass
// over bf16 chunks: as many bytes as two planes, and the wavefronts make three of
// it as they read.  (Three planes in LDS would not leave room for two chunks.)  A
// row's 16-byte pieces lie in turned order, so that the 16 rows token_of(mt, m)
// that an operand reads at one piece hit different banks.
template <int C>
struct TriWords {
    static constexpr int NB = tri_blocks(C);
    float x[NB][32 * 32];
    static __device__ __forceinline__ int at_(int row, int piece) {
        return row * 32 + ((piece ^ (((row >> 1) & 1) | (((row >> 3) & 3) << 1))) << 2);
    }
    // rows `row` of block (I, J), columns 8 g .. 8 g + 7
    __device__ __forceinline__ void rows(int I, int J, int row, int g, f32x4 (&o)[2]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) o[i] = *(const f32x4 *)&x[tri_block(I, J)][at_(row, 2 * g + i)];
    }
    // four neighbours c .. c + 3 of a row (c a multiple of 4)
    __device__ __forceinline__ void put4(int I, int J, int row, int c, const float (&v)[4]) {
        *(f32x4 *)&x[tri_block(I, J)][at_(row, c >> 2)] = f32x4{v[0], v[1], v[2], v[3]};
    }
};

// Contiguous bytes (a multiple of 16) to LDS, by the work-group's NW wavefronts.
template <int BYTES, int NW>
__device__ __forceinline__ void direct_block(const void *src, void *lds, int wv, int lane) {
#pragma unroll
    for (int i = 0; i < (BYTES + 1023) / 1024; i += NW) {
        const int k = (i + wv) * 1024;
        // whole pieces of 1 KiB but for the end
        if (BYTES % 1024 == 0 ? k < BYTES : k + lane * 16 < BYTES)
            direct16((const uint8_t *)src + k, (uint32_t)lane * 16, (uint8_t *)lds + k);
    }
}

// bf16 rows to LDS (q, k, dO, or a plane of what the passes keep): R rows,
// zeros from row n and column dk on.  For rows that can be read 16 bytes at a
// time (a.vec also bounds the stride: a chunk's offsets fit 32 bits).
template <int R, int W, int NW>
__device__ __forceinline__ void direct_rows(uint16_t *dst, const uint16_t *src, int64_t stride, int n,
                                            int dk, int wv, int lane) {
    constexpr int PPR = W / 8, RPI = 64 / PPR;       // pieces of a row, rows of an instruction
    const uint32_t bytes = (uint32_t)stride * 2;
    const bool whole = n == R && dk == W;
    // the lane's piece of the wavefront's first rows; its later rows are whole
    // 8s further on, where all lanes' turns change alike
    const int row0 = wv * RPI + lane / PPR;
    const uint32_t piece0 = (uint32_t)((lane % PPR) ^ turn<W>(row0)) * 16, row_at = (uint32_t)(lane / PPR) * bytes;
#pragma unroll
    for (int i = 0; i < R / RPI; i += NW) {
        const int blk = i + wv;
        if (R / RPI % NW != 0 && blk >= R / RPI) break;
        const uint32_t piece = piece0 ^ (uint32_t)(turn<W>(blk * RPI) ^ turn<W>(wv * RPI)) * 16;
        uint16_t *to = dst + blk * RPI * W;
        if (whole || (row0 + i * RPI < n && (int)piece < dk * 2))
            direct16((const uint8_t *)src + (int64_t)(blk * RPI) * bytes, piece + row_at, to);
        else
            *(u32x4 *)(to + lane * 8) = u32x4{0, 0, 0, 0};
    }
}

// A wavefront's 16 value columns of C tokens in LDS, [C][16] of the inputs'
// type: v or dO on the way in (directly, 16 bytes per lane), o on the way out.
// For rows of 16-byte pieces (a.vec_v: aligned, and d_v a whole number of
// pieces); columns from d_v on are not written.
template <typename IN, int C>
struct Tile {
    static constexpr int PPR = sizeof(IN), RPI = 64 / PPR;   // 16-byte pieces of a row, rows of an instruction
    IN x[C * 16];
    // n tokens from src (the tile's first column), rows `stride` apart
    __device__ __forceinline__ void fetch(const IN *src, int64_t stride, int n, int cols, int lane) {
        const uint32_t bytes = (uint32_t)stride * sizeof(IN);
        const int piece = lane % PPR, row = lane / PPR;
#pragma unroll
        for (int i = 0; i < C / RPI; ++i)
            if (i * RPI + row < n && piece * (16 / (int)sizeof(IN)) < cols)
                direct16((const uint8_t *)src + (int64_t)(i * RPI) * bytes, (uint32_t)row * bytes + piece * 16,
                         &x[i * RPI * 16]);
    }
    // the lane's column m = lane & 15 at tokens token_of(mt, 4 g + r)
    __device__ __forceinline__ void get(int mt, int lane, float (&v)[4]) const {
        const int g = lane >> 4, t0 = 32 * (mt >> 1) + 8 * g + 4 * (mt & 1);
        if constexpr (sizeof(IN) == 2) {
            typedef __attribute__((address_space(3))) s16x4 lds4;
            const int i = lane & 15;
            const s16x4 w = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4 *)&x[(t0 + (i >> 2)) * 16 + 4 * (i & 3)]);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = bf2f((uint16_t)w[r]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = x[(t0 + r) * 16 + (lane & 15)];
        }
    }
    __device__ __forceinline__ void put(int mt, int lane, const f32x4 &v) {
        const int g = lane >> 4, t0 = 32 * (mt >> 1) + 8 * g + 4 * (mt & 1);
#pragma unroll
        for (int r = 0; r < 4; r += 2) {
            if constexpr (sizeof(IN) == 2) {
                const uint32_t w = pack2(v[r], v[r + 1]);
                x[(t0 + r) * 16 + (lane & 15)] = (IN)(w & 0xffff);
                x[(t0 + r + 1) * 16 + (lane & 15)] = (IN)(w >> 16);
            } else {
                x[(t0 + r) * 16 + (lane & 15)] = v[r];
                x[(t0 + r + 1) * 16 + (lane & 15)] = v[r + 1];
            }
        }
    }
    // the tile's n first rows to dst
    __device__ __forceinline__ void store(IN *dst, int64_t stride, int n, int cols, int lane) const {
        const uint32_t bytes = (uint32_t)stride * sizeof(IN);
        const int piece = lane % PPR, row = lane / PPR;
#pragma unroll
        for (int i = 0; i < C / RPI; ++i) {
            f32x4 w = *(const f32x4 *)((const uint8_t *)&x[i * RPI * 16] + lane * 16);
            if (i * RPI + row < n && piece * (16 / (int)sizeof(IN)) < cols)
                store4((float *)((uint8_t *)dst + (int64_t)(i * RPI) * bytes + ((uint32_t)row * bytes + piece * 16)), w);
        }
    }
};

// fp32 rows on their way to LDS, where they become planes: held in registers
// while the chunk before is worked on.  Every thread reads inside the rows,
// what is not there is blanked on the way to LDS, so no branch and no wait
// stands between the loads.
template <int R, int W, int TH>
struct RowFetch {
    static constexpr int N = (R * (W / 8) + TH - 1) / TH;
    f32x4 w[N][2];
    __device__ __forceinline__ void load(const float *src, int64_t stride, int n, int dk, int tid) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = tid + i * TH, row = x / (W / 8), c = (x % (W / 8)) * 8;
            const uint32_t at = (uint32_t)min(row, n - 1) * (uint32_t)stride + (uint32_t)(c < dk ? c : 0);
#pragma unroll
            for (int j = 0; j < 2; ++j) w[i][j] = ((const f32x4 *)(src + at))[j];
        }
    }
    __device__ __forceinline__ void store(Planes<3, R, W> &dst, int n, int dk, int tid) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int x = tid + i * TH, row = x / (W / 8), c = (x % (W / 8)) * 8;
            if (R * (W / 8) % TH != 0 && x >= R * (W / 8)) continue;
            float f[8];
            pair8(w[i][0], w[i][1], f);
            if (row >= n || c >= dk) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = 0.0f;
            }
            b16x8 p[3];
            split8(f, p);
            dst.put8(row, c, p);
        }
    }
};

// Wavefronts of a work-group in the passes over the chunks (16 value rows
// each).  Eight share a chunk's rows in LDS and fill a compute unit's SIMDs
// twice, which pays where that still leaves a work-group for each of the 256
// compute units; with fewer units the rows are spread over more of them.
// Measured at bf16, d_k = d_v = 128, all kernels of the call: 256 units x 4096
// tokens 723 us by eight, 859 by four; 32 units 439 and 351; backward, 256 units
// x 1024 tokens 836 and 875, 128 units x 2048 1050 and 868.  With 64 value rows
// four of the eight only fetch, and 256 units x 2048 tokens still take 267 us
// by eight and 279 by four (512 units without delta 286 and 319).  At d_k = 256
// eight wavefronts have too few registers for the state (256 units x 512 tokens,
// d_v = 256: 395 us by eight, 331 by four; fp32 1359 and 770), so the callers ask
// only at d_k <= 128.
inline int scan_waves(const ScanArgs &a) {
    return (int64_t)a.B * a.H * ((a.dv + 127) / 128) >= 256 ? 8 : 4;
}

// The units' order along the grid: work-groups go round the 8 XCDs, so the
// `groups` work-groups of a unit, which read the same rows, are 8 apart and
// share an L2.
__device__ __forceinline__ bool unit_of(int block, int groups, int units, int *unit, int *grp) {
    const int x = block & 7, y = block >> 3;
    *grp = y % groups;
    *unit = y / groups * 8 + x;
    return *unit < units;
}

// The chunks' order along the grid of the kernels that take all at once: an
// XCD gets all key heads of a chunk one after the other, which read and write
// neighbouring words of alpha and beta's lines.
__device__ __forceinline__ bool chunk_of(int block, const ScanArgs &a, const ScanWork &w, int *b, int *hk,
                                         int *chunk) {
    const int x = block & 7, y = block >> 3;
    const int at = y / a.Hk * 8 + x;                 // sequence and chunk
    *hk = y % a.Hk;
    *b = at / w.chunks;
    *chunk = at - *b * w.chunks;
    return *b < a.B;
}
inline dim3 chunk_grid(const ScanArgs &a, const ScanWork &w) {
    return grid_of(((int64_t)a.B * w.chunks + 7) / 8 * 8 * a.Hk);
}

}  // namespace scan
}  // namespace lores
