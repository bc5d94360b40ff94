// Internal declarations of the layer operators (gated norm, norms around a
// block, 4-bit rows and their product): launch descriptions shared by the host
// API (lores_layer_api.cpp) and the HIP kernels.  Not part of the public ABI.
#pragma once

#include "lores_seq.h"

namespace lores {

// How a kernel reads its rows (VEC of lores_rows.h): aligned rows of whole
// vectors, or rows of any length and alignment.
enum { ROWS_VEC = 1, ROWS_ODD = 2 };

struct GatedArgs {
    int64_t rows;                      // tokens x heads
    int32_t heads, n;
    uint32_t per_heads;                // floor((2^32 - 1) / heads), for a row's token
    int32_t w_bf16, per_head, act, gate_first, out_prec;
    float eps;
    int64_t xs[2], gs[2];              // elements between tokens, heads
    const void *x, *gate, *w;
    void *y;
    uint8_t *scales;
    // backward
    const void *dy;
    void *dx, *dgate;
    float *dw, *part;
    int32_t groups;                    // work-groups (with weights per head: of each head) that sum dw apart
};
int gated_groups(int64_t tokens, int32_t heads, int32_t n, int32_t per_head);
hipError_t launch_gated(bool in_bf16, int mode, const GatedArgs &a, hipStream_t s);
hipError_t launch_gated_backward(bool in_bf16, int mode, const GatedArgs &a, hipStream_t s);

struct BlockArgs {
    int64_t rows;
    int32_t n, w_bf16, act, out_prec;
    float eps, scale;
    int64_t xs, rs, gs;
    const void *x, *res, *gate, *w, *wn;
    void *y, *scales, *h;
    // backward
    const void *dy, *dh;
    void *dx, *dres, *dgate;
    float *dw, *dwn, *part;
    int32_t groups;
};
int block_groups(int64_t rows, int32_t n);
hipError_t launch_block(bool in_bf16, int mode, const BlockArgs &a, hipStream_t s);
hipError_t launch_block_backward(bool in_bf16, int mode, const BlockArgs &a, hipStream_t s);

struct MxRows {
    int64_t rows;
    int32_t n;
    int64_t xs;                        // elements between rows of x
    const void *x;
    uint8_t *codes, *scales;
    void *out;
};
hipError_t launch_mx_quant(bool in_bf16, bool vec, const MxRows &a, hipStream_t s);
hipError_t launch_mx_dequant(bool out_bf16, const MxRows &a, hipStream_t s);

struct MxProduct {
    int64_t M;
    int32_t N, K;
    const uint8_t *a, *w, *a_scales, *w_scales;   // a_scales: of 4-bit rows
    const float *a_rows;                          // of E4M3 rows
    void *out;
};
hipError_t launch_mx_product(bool a_fp8, bool out_bf16, const MxProduct &p, hipStream_t s);

}  // namespace lores
