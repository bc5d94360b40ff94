// Host side of the layer operators' C ABI (lores_gated_norm*, lores_block_norm*,
// lores_mx_*): argument validation and launches.  Every exported function
// validates first and launches nothing on error; no exception leaves this file.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "lores_layer.h"

namespace {

int fail(int code, const char *fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    return lores::set_error(code, buf);
}

bool aligned(const void *p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Errors of earlier work on this thread are not this call's.
void consume_stale_hip_error() { (void)hipGetLastError(); }

int hip_status(hipError_t e, const char *what) {
    if (e != hipSuccess) return fail(LORES_EHIP, "%s launch failed: %s", what, hipGetErrorString(e));
    return lores::set_ok();
}

bool flag(int32_t x) { return x == 0 || x == 1; }
constexpr int64_t kMaxStride = (int64_t)1 << 40;
// elements of a matrix of one call: more than the memory holds, and the grids'
// work-groups stay countable
constexpr int64_t kMaxCells = (int64_t)1 << 38;

int check_rows(int32_t n, int32_t in_bf16, int32_t w_bf16, int32_t act, float eps) {
    if (n < 1 || n > LORES_MAX_NORM)
        return fail(LORES_EINVAL, "n must be in [1, %d] (got %d)", LORES_MAX_NORM, n);
    if (!flag(in_bf16) || !flag(w_bf16)) return fail(LORES_EINVAL, "in_bf16 and w_bf16 must be 0 or 1");
    if (act != LORES_ACT_NONE && act != LORES_ACT_SILU && act != LORES_ACT_SIGMOID)
        return fail(LORES_EINVAL, "act must be LORES_ACT_NONE, LORES_ACT_SILU or LORES_ACT_SIGMOID (got %d)", act);
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(LORES_EINVAL, "eps must be finite and >= 0");
    return LORES_OK;
}

int check_gated(const lores_gated_dims *d) {
    if (!d) return fail(LORES_EINVAL, "dims is NULL");
    if (const int rc = check_rows(d->n, d->in_bf16, d->w_bf16, d->act, d->eps)) return rc;
    if (d->heads < 1 || d->heads > LORES_MAX_HEADS)
        return fail(LORES_EINVAL, "heads must be in [1, %d] (got %d)", LORES_MAX_HEADS, d->heads);
    if (d->tokens < 0 || d->tokens > 0x7fffffff / d->heads)
        return fail(LORES_EINVAL, "tokens x heads must be in [0, 2^31)");
    if (!flag(d->per_head) || !flag(d->gate_first))
        return fail(LORES_EINVAL, "per_head and gate_first must be 0 or 1");
    for (int i = 0; i < 2; ++i)
        if (d->x_stride[i] < 0 || d->gate_stride[i] < 0 || d->x_stride[i] > kMaxStride || d->gate_stride[i] > kMaxStride)
            return fail(LORES_EINVAL, "strides must be in [0, 2^40]");
    return LORES_OK;
}

int check_block(const lores_block_dims *d) {
    if (!d) return fail(LORES_EINVAL, "dims is NULL");
    if (const int rc = check_rows(d->n, d->in_bf16, d->w_bf16, d->act, d->eps)) return rc;
    if (d->rows < 0 || d->rows > 0x7fffffff) return fail(LORES_EINVAL, "rows must be in [0, 2^31)");
    if (!std::isfinite(d->scale)) return fail(LORES_EINVAL, "scale must be finite");
    for (const int64_t s : {d->x_stride, d->res_stride, d->gate_stride})
        if (s < 0 || (s > 0 && s < d->n) || s > kMaxStride)
            return fail(LORES_EINVAL, "strides must be 0 or in [n, 2^40]");
    return LORES_OK;
}

lores::GatedArgs gated_args(const lores_gated_dims *d, const void *x, const void *gate, const void *w) {
    lores::GatedArgs a;
    std::memset(&a, 0, sizeof a);
    a.rows = d->tokens * d->heads;
    a.heads = d->heads;
    a.n = d->n;
    a.per_heads = 0xffffffffu / (uint32_t)d->heads;
    a.w_bf16 = d->w_bf16;
    a.per_head = d->per_head;
    a.act = d->act;
    a.gate_first = d->gate_first;
    a.eps = d->eps;
    for (int i = 0; i < 2; ++i) {
        a.xs[i] = d->x_stride[i];
        a.gs[i] = d->gate_stride[i];
    }
    a.x = x;
    a.gate = gate;
    a.w = w;
    return a;
}

bool gated_vec(const lores_gated_dims *d, const void *x, const void *gate, const void *w) {
    const int64_t el = d->in_bf16 ? 2 : 4;
    bool vec = d->n % 8 == 0 && aligned(x, 16) && aligned(gate, 16) && aligned(w, 16);
    for (int i = 0; i < 2; ++i)
        if (d->x_stride[i] * el % 16 != 0 || d->gate_stride[i] * el % 16 != 0) vec = false;
    return vec;
}

lores::BlockArgs block_args(const lores_block_dims *d, const void *x, const void *gate, const void *w,
                            const void *wn) {
    lores::BlockArgs a;
    std::memset(&a, 0, sizeof a);
    a.rows = d->rows;
    a.n = d->n;
    a.w_bf16 = d->w_bf16;
    a.act = d->act;
    a.eps = d->eps;
    a.scale = d->scale;
    a.xs = d->x_stride;
    a.rs = d->res_stride;
    a.gs = d->gate_stride;
    a.x = x;
    a.gate = gate;
    a.w = w;
    a.wn = wn;
    return a;
}

bool block_vec(const lores_block_dims *d, const void *x, const void *gate, const void *w, const void *wn) {
    const int64_t el = d->in_bf16 ? 2 : 4;
    return d->n % 8 == 0 && aligned(x, 16) && aligned(gate, 16) && aligned(w, 16) && aligned(wn, 16) &&
           d->x_stride * el % 16 == 0 && (!gate || d->gate_stride * el % 16 == 0);
}

int check_work(uint64_t need, const void *work, size_t bytes) {
    if (!need) return LORES_OK;
    if (!work) return fail(LORES_EINVAL, "work is NULL (%llu bytes needed)", (unsigned long long)need);
    if (!aligned(work, 16)) return fail(LORES_EINVAL, "work must be 16-byte aligned");
    if (bytes < need)
        return fail(LORES_ESIZE, "work holds %llu bytes, %llu needed", (unsigned long long)bytes,
                    (unsigned long long)need);
    return LORES_OK;
}

uint64_t gated_work(const lores_gated_dims *d) {
    return (uint64_t)lores::gated_groups(d->tokens, d->heads, d->n, d->per_head) * d->n *
           (d->per_head ? d->heads : 1) * sizeof(float);
}

// both weights' sums, whether there are two or not
uint64_t block_work(const lores_block_dims *d) {
    return (uint64_t)lores::block_groups(d->rows, d->n) * d->n * 2 * sizeof(float);
}

int check_mx_rows(int64_t rows, int32_t n) {
    if (rows < 0 || rows > 0x7fffffff) return fail(LORES_EINVAL, "rows must be in [0, 2^31)");
    if (n < 32 || n > (1 << 24) || n % 32 != 0)
        return fail(LORES_EINVAL, "n must be a multiple of 32 in [32, 2^24] (got %d)", n);
    if (rows > kMaxCells / n) return fail(LORES_EINVAL, "rows x n must be at most 2^38");
    return LORES_OK;
}

int check_mx_out(int32_t n, const void *codes, const void *scales) {
    if (n % 32 != 0) return fail(LORES_EINVAL, "LORES_MXFP4 needs n in multiples of 32 (got %d)", n);
    if (!scales) return fail(LORES_EINVAL, "LORES_MXFP4 needs scales");
    if (!aligned(codes, 16)) return fail(LORES_EINVAL, "codes must be 16-byte aligned");
    return LORES_OK;
}

}  // namespace

extern "C" {

int lores_gated_norm(const lores_gated_dims *dims, const void *x, const void *gate, const void *weight,
                     int32_t out_prec, void *y, uint8_t *scales, void *stream) {
    if (const int rc = check_gated(dims)) return rc;
    if (out_prec != LORES_FP32 && out_prec != LORES_BF16 && out_prec != LORES_MXFP4)
        return fail(LORES_EINVAL, "out_prec must be LORES_FP32, LORES_BF16 or LORES_MXFP4 (got %d)", out_prec);
    const bool mx = out_prec == LORES_MXFP4;
    if (dims->tokens == 0) return lores::set_ok();
    if (!x || !gate || !weight || !y)
        return fail(LORES_EINVAL, "x, gate, weight and y must be non-NULL device pointers");
    if (mx)
        if (const int rc = check_mx_out(dims->n, y, scales)) return rc;
    const uintptr_t el = dims->in_bf16 ? 2 : 4, wel = dims->w_bf16 ? 2 : 4;
    const uintptr_t yel = mx ? 16 : out_prec == LORES_FP32 ? 4 : 2;
    if (!aligned(x, el) || !aligned(gate, el) || !aligned(weight, wel) || !aligned(y, yel))
        return fail(LORES_EINVAL, "pointers must be aligned to their element size");
    lores::GatedArgs a = gated_args(dims, x, gate, weight);
    a.out_prec = out_prec;
    a.y = y;
    a.scales = scales;
    const bool vec = gated_vec(dims, x, gate, weight) && aligned(y, 16);
    consume_stale_hip_error();
    return hip_status(lores::launch_gated(dims->in_bf16, vec ? lores::ROWS_VEC : lores::ROWS_ODD,
                                          a, (hipStream_t)stream),
                      "gated norm");
}

int lores_gated_norm_workspace(const lores_gated_dims *dims, size_t *bytes) {
    if (!bytes) return fail(LORES_EINVAL, "bytes is NULL");
    if (const int rc = check_gated(dims)) return rc;
    *bytes = (size_t)gated_work(dims);
    return lores::set_ok();
}

int lores_gated_norm_backward(const lores_gated_dims *dims, const void *x, const void *gate, const void *weight,
                              const void *dy, void *dx, void *dgate, float *dw, void *work, size_t work_bytes,
                              void *stream) {
    if (const int rc = check_gated(dims)) return rc;
    if (!dw) return fail(LORES_EINVAL, "dw must be a non-NULL device pointer");
    if (dims->tokens && (!x || !gate || !weight || !dy || !dx || !dgate))
        return fail(LORES_EINVAL, "x, gate, weight, dy, dx and dgate must be non-NULL device pointers");
    const uintptr_t el = dims->in_bf16 ? 2 : 4, wel = dims->w_bf16 ? 2 : 4;
    if (!aligned(x, el) || !aligned(gate, el) || !aligned(dy, el) || !aligned(dx, el) || !aligned(dgate, el) ||
        !aligned(weight, wel) || !aligned(dw, 4))
        return fail(LORES_EINVAL, "pointers must be aligned to their element size");
    if (const int rc = check_work(gated_work(dims), work, work_bytes)) return rc;
    lores::GatedArgs a = gated_args(dims, x, gate, weight);
    a.dy = dy;
    a.dx = dx;
    a.dgate = dgate;
    a.dw = dw;
    a.part = (float *)work;
    a.groups = lores::gated_groups(dims->tokens, dims->heads, dims->n, dims->per_head);
    const bool vec = gated_vec(dims, x, gate, weight) && aligned(dy, 16) && aligned(dx, 16) && aligned(dgate, 16);
    consume_stale_hip_error();
    return hip_status(lores::launch_gated_backward(dims->in_bf16, vec ? lores::ROWS_VEC : lores::ROWS_ODD, a,
                                                   (hipStream_t)stream),
                      "gated norm backward");
}

int lores_block_norm(const lores_block_dims *dims, const void *x, const void *residual, const void *gate,
                     const void *weight, const void *weight_next, int32_t out_prec, void *y, void *scales, void *h,
                     void *stream) {
    if (const int rc = check_block(dims)) return rc;
    if (out_prec != LORES_FP32 && out_prec != LORES_BF16 && out_prec != LORES_INT8 && out_prec != LORES_FP8 &&
        out_prec != LORES_MXFP4)
        return fail(LORES_EINVAL, "out_prec must be LORES_FP32, LORES_BF16, LORES_INT8, LORES_FP8 or LORES_MXFP4 "
                                  "(got %d)", out_prec);
    const bool mx = out_prec == LORES_MXFP4, bytes = out_prec == LORES_INT8 || out_prec == LORES_FP8;
    if (dims->rows == 0) return lores::set_ok();
    if (!x || !weight_next || !y || !h)
        return fail(LORES_EINVAL, "x, weight_next, y and h must be non-NULL device pointers");
    if (mx)
        if (const int rc = check_mx_out(dims->n, y, scales)) return rc;
    if (bytes && !scales) return fail(LORES_EINVAL, "8-bit outputs need scales");
    const uintptr_t el = dims->in_bf16 ? 2 : 4, wel = dims->w_bf16 ? 2 : 4;
    const uintptr_t yel = mx ? 16 : out_prec == LORES_FP32 ? 4 : out_prec == LORES_BF16 ? 2 : 1;
    if (!aligned(x, el) || !aligned(residual, el) || !aligned(gate, el) || !aligned(h, el) || !aligned(weight, wel) ||
        !aligned(weight_next, wel) || !aligned(y, yel) || (bytes && !aligned(scales, 4)))
        return fail(LORES_EINVAL, "pointers must be aligned to their element size");
    lores::BlockArgs a = block_args(dims, x, gate, weight, weight_next);
    a.out_prec = out_prec;
    a.res = residual;
    a.y = y;
    a.scales = scales;
    a.h = h;
    const bool vec = block_vec(dims, x, gate, weight, weight_next) && aligned(residual, 16) && aligned(h, 16) &&
                     (!residual || dims->res_stride * (int64_t)el % 16 == 0) && aligned(y, bytes ? 8 : 16);
    consume_stale_hip_error();
    return hip_status(lores::launch_block(dims->in_bf16, vec ? lores::ROWS_VEC : lores::ROWS_ODD,
                                          a, (hipStream_t)stream),
                      "block norm");
}

int lores_block_norm_workspace(const lores_block_dims *dims, size_t *bytes) {
    if (!bytes) return fail(LORES_EINVAL, "bytes is NULL");
    if (const int rc = check_block(dims)) return rc;
    *bytes = (size_t)block_work(dims);
    return lores::set_ok();
}

int lores_block_norm_backward(const lores_block_dims *dims, const void *x, const void *h, const void *gate,
                              const void *weight, const void *weight_next, const void *dy, const void *dh, void *dx,
                              void *dresidual, void *dgate, float *dw, float *dw_next, void *work, size_t work_bytes,
                              void *stream) {
    if (const int rc = check_block(dims)) return rc;
    if (!dw_next || (weight && !dw)) return fail(LORES_EINVAL, "dw and dw_next must be non-NULL device pointers");
    if (dims->rows && (!x || !h || !weight_next || !dy || !dx || !dresidual))
        return fail(LORES_EINVAL, "x, h, weight_next, dy, dx and dresidual must be non-NULL device pointers");
    if (dims->rows && gate && !dgate) return fail(LORES_EINVAL, "a gate needs dgate");
    const uintptr_t el = dims->in_bf16 ? 2 : 4, wel = dims->w_bf16 ? 2 : 4;
    if (!aligned(x, el) || !aligned(h, el) || !aligned(gate, el) || !aligned(dy, el) || !aligned(dh, el) ||
        !aligned(dx, el) || !aligned(dresidual, el) || !aligned(dgate, el) || !aligned(weight, wel) ||
        !aligned(weight_next, wel) || !aligned(dw, 4) || !aligned(dw_next, 4))
        return fail(LORES_EINVAL, "pointers must be aligned to their element size");
    if (const int rc = check_work(block_work(dims), work, work_bytes)) return rc;
    lores::BlockArgs a = block_args(dims, x, gate, weight, weight_next);
    a.h = (void *)h;
    a.dy = dy;
    a.dh = dh;
    a.dx = dx;
    a.dres = dresidual;
    a.dgate = dgate;
    a.dw = dw;
    a.dwn = dw_next;
    a.part = (float *)work;
    a.groups = lores::block_groups(dims->rows, dims->n);
    const bool vec = block_vec(dims, x, gate, weight, weight_next) && aligned(h, 16) && aligned(dy, 16) &&
                     aligned(dh, 16) && aligned(dx, 16) && aligned(dresidual, 16) && aligned(dgate, 16);
    consume_stale_hip_error();
    return hip_status(lores::launch_block_backward(dims->in_bf16, vec ? lores::ROWS_VEC : lores::ROWS_ODD, a,
                                                   (hipStream_t)stream),
                      "block norm backward");
}

int lores_mx_quant(const void *x, int64_t x_stride, int64_t rows, int32_t n, int32_t in_bf16, uint8_t *codes,
                   uint8_t *scales, void *stream) {
    if (const int rc = check_mx_rows(rows, n)) return rc;
    if (!flag(in_bf16)) return fail(LORES_EINVAL, "in_bf16 must be 0 or 1");
    if (rows == 0) return lores::set_ok();
    if (!x || !codes || !scales) return fail(LORES_EINVAL, "x, codes and scales must be non-NULL device pointers");
    const uintptr_t el = in_bf16 ? 2 : 4;
    if (!aligned(x, el)) return fail(LORES_EINVAL, "x must be aligned to its element size");
    if (!aligned(codes, 16) || !aligned(scales, 4))
        return fail(LORES_EINVAL, "codes must be 16-byte and scales 4-byte aligned");
    if ((x_stride < n && x_stride != 0) || x_stride > kMaxStride)
        return fail(LORES_EINVAL, "rows must be 0, or n to 2^40, elements apart");
    lores::MxRows a;
    std::memset(&a, 0, sizeof a);
    a.rows = rows;
    a.n = n;
    a.xs = x_stride;
    a.x = x;
    a.codes = codes;
    a.scales = scales;
    consume_stale_hip_error();
    return hip_status(lores::launch_mx_quant(in_bf16, aligned(x, 16) && x_stride * (int64_t)el % 16 == 0, a,
                                             (hipStream_t)stream),
                      "4-bit rows");
}

int lores_mx_dequant(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t n, int32_t out_bf16, void *out,
                     void *stream) {
    if (const int rc = check_mx_rows(rows, n)) return rc;
    if (!flag(out_bf16)) return fail(LORES_EINVAL, "out_bf16 must be 0 or 1");
    if (rows == 0) return lores::set_ok();
    if (!codes || !scales || !out) return fail(LORES_EINVAL, "codes, scales and out must be non-NULL device pointers");
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(out, 16))
        return fail(LORES_EINVAL, "codes and out must be 16-byte and scales 4-byte aligned");
    lores::MxRows a;
    std::memset(&a, 0, sizeof a);
    a.rows = rows;
    a.n = n;
    a.codes = (uint8_t *)codes;
    a.scales = (uint8_t *)scales;
    a.out = out;
    consume_stale_hip_error();
    return hip_status(lores::launch_mx_dequant(out_bf16, a, (hipStream_t)stream), "values of 4-bit rows");
}

int lores_mx_matmul(const void *a, const void *a_scales, int32_t a_prec, const uint8_t *w, const uint8_t *w_scales,
                    int64_t M, int32_t N, int32_t K, int32_t out_prec, void *out, void *stream) {
    if (M < 0 || M > 0x7fffffff) return fail(LORES_EINVAL, "M must be in [0, 2^31)");
    if (N < 1 || N > (1 << 24)) return fail(LORES_EINVAL, "N must be in [1, 2^24] (got %d)", N);
    if (M > kMaxCells / N) return fail(LORES_EINVAL, "M x N must be at most 2^38");
    if (K < 32 || K > (1 << 24) || K % 32 != 0)
        return fail(LORES_EINVAL, "K must be a multiple of 32 in [32, 2^24] (got %d)", K);
    if (a_prec != LORES_MXFP4 && a_prec != LORES_FP8)
        return fail(LORES_EINVAL, "a_prec must be LORES_MXFP4 or LORES_FP8 (got %d)", a_prec);
    if (out_prec != LORES_BF16 && !(out_prec == LORES_FP32 && a_prec == LORES_MXFP4))
        return fail(LORES_EINVAL, "out_prec must be LORES_BF16, or LORES_FP32 for LORES_MXFP4 rows (got %d)", out_prec);
    if (M == 0) return lores::set_ok();
    if (!a || !a_scales || !w || !w_scales || !out)
        return fail(LORES_EINVAL, "a, w, their scales and out must be non-NULL device pointers");
    if (!aligned(a, 16) || !aligned(w, 16) || !aligned(a_scales, 4) || !aligned(w_scales, 4) || !aligned(out, 16))
        return fail(LORES_EINVAL, "a, w and out must be 16-byte and scales 4-byte aligned");
    lores::MxProduct p;
    std::memset(&p, 0, sizeof p);
    p.M = M;
    p.N = N;
    p.K = K;
    p.a = (const uint8_t *)a;
    p.w = w;
    p.w_scales = w_scales;
    if (a_prec == LORES_FP8) p.a_rows = (const float *)a_scales;
    else p.a_scales = (const uint8_t *)a_scales;
    p.out = out;
    consume_stale_hip_error();
    return hip_status(lores::launch_mx_product(a_prec == LORES_FP8, out_prec == LORES_BF16, p, (hipStream_t)stream),
                      "4-bit product");
}

}  // extern "C"
