// Internal declarations of the sequence operators (lores_scan*, lores_rmsnorm*):
// launch descriptions shared by the host API (lores_seq_api.cpp) and the HIP
// kernels (lores_scan_*.hip, lores_norm.hip).  Not part of the public ABI.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/lores.h"

namespace lores {

// The calling thread's error text (lores_last_error); returns `code`.
int set_error(int code, const char *msg);
int set_ok();

// A launch takes fewer than 2^32 work-items along x, so more work-groups than
// kGridRow (of at most 1024 threads; a multiple of the 8 XCDs) go over rows of the
// grid.  The last row may be longer than what is left: kernels return at a
// block_at() behind their work.
constexpr int kGridRow = 1 << 21;
inline dim3 grid_of(int64_t groups) {
    return groups <= kGridRow ? dim3((uint32_t)groups) : dim3(kGridRow, (uint32_t)((groups + kGridRow - 1) / kGridRow));
}
__host__ __device__ constexpr int64_t block_at(uint32_t x, uint32_t y) { return (int64_t)y * kGridRow + x; }

// ------------------------------------------------------------ the norm

struct NormArgs {
    int64_t rows;
    int32_t n;
    int32_t w_bf16, out_prec;
    float eps;
    int64_t x_stride, res_stride;      // elements between rows
    const void *x, *res, *w;
    void *y, *h;
    float *scales;
    // backward: x is the stored sum h
    const void *dy, *dres;
    void *dx;
    float *dw, *part;
    int32_t groups;                    // work-groups that sum dw apart
};

// Work-groups of the backward pass: each keeps its own column sums of dw.
int norm_groups(int64_t rows, int32_t n);
hipError_t launch_norm(bool in_bf16, bool vec, const NormArgs &a, hipStream_t s);
hipError_t launch_norm_backward(bool in_bf16, bool vec, const NormArgs &a, hipStream_t s);

// `cols` columns summed over `groups` rows of `part`; columns from `split` on go to out1.
hipError_t launch_group_sums(const float *part, int groups, int cols, int split, float *out0, float *out1,
                             hipStream_t s);

// Bytes between the scales of rows of 4-bit blocks: whole words of 4 blocks.
__host__ __device__ constexpr int mx_scale_stride(int64_t n) { return (int)((n + 127) / 128 * 4); }

// ------------------------------------------------------------ the recurrence

struct ScanArgs {
    int32_t B, T, H, Hk, dk, dv, delta;
    int32_t vec;                       // q and k rows can be read 16 bytes at a time, and
                                       // tokens lie less than 2^24 elements apart
    int32_t vec_v;                     // the same of v, with d_v a multiple of 16 bytes, and of
                                       // o, dout and dv
    int64_t qs[3], ks[3], vs[3];       // elements between sequences, tokens, heads
    const void *q, *k, *v;
    const float *alpha, *beta;         // [B][T][H]
    const int32_t *lengths;            // [B], or NULL: every sequence has T tokens
    const float *S0;                   // [B][H][dv][dk], or NULL: zero
    void *o;                           // [B][T][H][dv], input type
    float *S;                          // [B][H][dv][dk], or NULL
    int32_t vec_g;                     // dq and dk rows are 16-byte aligned
    // backward
    const void *dout;                  // [B][T][H][dv], input type
    const float *dS;                   // [B][H][dv][dk], or NULL: zero
    void *dq, *dkey, *dvalue;          // [B][T][Hk][dk], [B][T][Hk][dk], [B][T][H][dv]
    float *dalpha, *dbeta;             // [B][T][H]
    float *dS0;                        // [B][H][dv][dk], or NULL
};

// Sequences of at most this many tokens take the token-by-token kernel, whose
// time grows with them, others the chunked ones.  At d_k = d_v = 128, 2, 4 and
// 8 tokens: 512 (sequence, head) units 19, 24 and 35 us against 43 by chunks;
// 2048 units 70, 97 and 153 us against 136.
inline int scan_rows_tokens(int64_t units) { return units <= 1024 ? 8 : 6; }

// Chunked scans: tokens of a chunk (the products' operands are held as bf16
// planes, and an fp32 input has three).
__host__ __device__ constexpr int scan_chunk(bool in_bf16) { return in_bf16 ? 64 : 32; }

// Workspace of a chunked scan, cut from the caller's buffer.  Per (sequence,
// head, chunk): the planes of X and P, the gates, and for the backward pass the state
// and its gradient at the chunk's two ends and U and H, value rows first.
struct ScanWork {
    uint16_t *X;                       // [B][H][chunks][3][blocks][32][32]
    uint16_t *P;                       // [B][H][chunks][3][blocks][32][32], or fp32 words (p_words)
    float *G;                          // [B][H][chunks][6][C]: Gates
    float *S, *dS;                     // [B][H][chunks][dvp][dk]
    float *U, *Hm;                     // [B][H][chunks][dvp][C]
    int32_t chunks, p_words, dvp;
};
// Lays `w` out over `base` (which may be NULL) and returns the bytes.
uint64_t plan_scan_work(bool in_bf16, bool backward, const ScanArgs &a, void *base, ScanWork *w);

// X and P of every chunk.
hipError_t launch_scan_prep(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s);
// The pass over the chunks: outputs and the last state, or (backward) every
// chunk's first state and U.
hipError_t launch_scan_state(bool in_bf16, bool backward, const ScanArgs &a, const ScanWork &w,
                             hipStream_t s);
// The pass back over the chunks: the state's gradients and H.
hipError_t launch_scan_back(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s);
// The inputs' gradients of every chunk.
hipError_t launch_scan_grad(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s);

hipError_t launch_scan_rows(bool in_bf16, const ScanArgs &a, hipStream_t s);

}  // namespace lores
