// Host side of the sequence operators' C ABI (lores_scan*, lores_rmsnorm*):
// argument validation, workspace planning and launches.  Every exported
// function validates first and launches nothing on error; no exception leaves
// this file.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "lores_seq.h"

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

// work-groups of a launch: with a row of the grid added they number below 2^31
constexpr int64_t kMaxGroups = (int64_t)0x7fffffff - lores::kGridRow;

int check_scan(const lores_scan_dims *d) {
    if (!d) return fail(LORES_EINVAL, "dims is NULL");
    if (d->B < 1 || d->B > 65535) return fail(LORES_EINVAL, "B must be in [1, 65535] (got %d)", d->B);
    if (d->T < 0 || d->T > (1 << 28)) return fail(LORES_EINVAL, "T must be in [0, 2^28] (got %d)", d->T);
    if (d->H < 1 || d->H > LORES_MAX_HEADS)
        return fail(LORES_EINVAL, "H must be in [1, %d] (got %d)", LORES_MAX_HEADS, d->H);
    if (d->H_k < 1 || d->H % d->H_k != 0)
        return fail(LORES_EINVAL, "H_k must divide H = %d (got %d)", d->H, d->H_k);
    if (d->d_k < 32 || d->d_k % 32 != 0 || d->d_k > 256)
        return fail(LORES_EINVAL, "d_k must be a multiple of 32 in [32, 256] (got %d)", d->d_k);
    if (d->d_v < 1 || d->d_v > LORES_MAX_DV)
        return fail(LORES_EINVAL, "d_v must be in [1, %d] (got %d)", LORES_MAX_DV, d->d_v);
    if (d->in_bf16 != 0 && d->in_bf16 != 1) return fail(LORES_EINVAL, "in_bf16 must be 0 or 1");
    if (d->delta != 0 && d->delta != 1) return fail(LORES_EINVAL, "delta must be 0 or 1 (got %d)", d->delta);
    for (int i = 0; i < 3; ++i)
        if (d->q_stride[i] < 0 || d->k_stride[i] < 0 || d->v_stride[i] < 0 ||
            d->q_stride[i] > ((int64_t)1 << 40) || d->k_stride[i] > ((int64_t)1 << 40) ||
            d->v_stride[i] > ((int64_t)1 << 40))
            return fail(LORES_EINVAL, "strides must be in [0, 2^40]");
    // the largest grid: 8 tiles of 32 value rows, or one work-group per chunk
    const int64_t chunks = (d->T + 31) / 32 + 8;     // and rounding up to 8 at the end
    if (((int64_t)d->B * chunks + 8) * d->H > kMaxGroups)
        return fail(LORES_EINVAL, "B x H x T is too large for one call");
    return LORES_OK;
}

lores::ScanArgs scan_args(const lores_scan_dims *d) {
    lores::ScanArgs a;
    std::memset(&a, 0, sizeof a);
    a.B = d->B;
    a.T = d->T;
    a.H = d->H;
    a.Hk = d->H_k;
    a.dk = d->d_k;
    a.dv = d->d_v;
    a.delta = d->delta;
    for (int i = 0; i < 3; ++i) {
        a.qs[i] = d->q_stride[i];
        a.ks[i] = d->k_stride[i];
        a.vs[i] = d->v_stride[i];
    }
    return a;
}

int check_scan_inputs(const lores_scan_dims *d, const void *q, const void *k, const void *v,
                      const float *alpha, const float *beta, const int32_t *lengths,
                      const float *S_first, lores::ScanArgs *a) {
    if (d->T && (!q || !k || !v || !alpha || !beta))
        return fail(LORES_EINVAL, "q, k, v, alpha and beta must be non-NULL device pointers");
    const uintptr_t el = d->in_bf16 ? 2 : 4;
    if (!aligned(q, el) || !aligned(k, el) || !aligned(v, el))
        return fail(LORES_EINVAL, "q, k and v must be aligned to their element size");
    if (!aligned(alpha, 4) || !aligned(beta, 4) || !aligned(lengths, 4))
        return fail(LORES_EINVAL, "alpha, beta and lengths must be 4-byte aligned");
    if (!aligned(S_first, 16)) return fail(LORES_EINVAL, "S_first must be 16-byte aligned");
    *a = scan_args(d);
    a->q = q;
    a->k = k;
    a->v = v;
    a->alpha = alpha;
    a->beta = beta;
    a->lengths = lengths;
    a->S0 = S_first;
    a->vec = aligned(q, 16) && aligned(k, 16);
    for (int i = 0; i < 3; ++i)
        if (a->qs[i] * (int64_t)el % 16 != 0 || a->ks[i] * (int64_t)el % 16 != 0) a->vec = 0;
    // offsets within a chunk of 64 tokens then fit 32 bits
    if (a->qs[1] >= (1 << 24) || a->ks[1] >= (1 << 24)) a->vec = 0;
    a->vec_v = aligned(v, 16) && d->d_v * el % 16 == 0 && a->vs[1] < (1 << 24);
    for (int i = 0; i < 3; ++i)
        if (a->vs[i] * (int64_t)el % 16 != 0) a->vec_v = 0;
    return LORES_OK;
}

// The chunked kernels' workspace, or 0 for a call that does not take them.
uint64_t scan_work(const lores_scan_dims *d, int32_t backward, void *base, lores::ScanWork *w) {
    if (backward ? d->T == 0 : d->T <= lores::scan_rows_tokens((int64_t)d->B * d->H)) return 0;
    return lores::plan_scan_work(d->in_bf16, backward, scan_args(d), base, w);
}

int check_work(uint64_t need, const void *work, size_t bytes) {
    if (!need) return LORES_OK;
    if (!work) return fail(LORES_EINVAL, "work is NULL (%llu bytes needed)", (unsigned long long)need);
    if (!aligned(work, 256)) return fail(LORES_EINVAL, "work must be 256-byte aligned");
    if (bytes < need)
        return fail(LORES_ESIZE, "work holds %llu bytes, %llu needed", (unsigned long long)bytes,
                    (unsigned long long)need);
    return LORES_OK;
}

int check_norm(int64_t rows, int32_t n, int32_t in_bf16, int32_t w_bf16, float eps) {
    if (rows < 0 || rows > 0x7fffffff) return fail(LORES_EINVAL, "rows must be in [0, 2^31)");
    if (n < 1 || n > LORES_MAX_NORM)
        return fail(LORES_EINVAL, "n must be in [1, %d] (got %d)", LORES_MAX_NORM, n);
    if (in_bf16 != 0 && in_bf16 != 1) return fail(LORES_EINVAL, "in_bf16 must be 0 or 1");
    if (w_bf16 != 0 && w_bf16 != 1) return fail(LORES_EINVAL, "w_bf16 must be 0 or 1");
    if (!(eps >= 0.0f) || !std::isfinite(eps)) return fail(LORES_EINVAL, "eps must be finite and >= 0");
    return LORES_OK;
}

}  // namespace

extern "C" {

int lores_scan_workspace(const lores_scan_dims *dims, int32_t backward, size_t *bytes) {
    if (!bytes) return fail(LORES_EINVAL, "bytes is NULL");
    if (const int rc = check_scan(dims)) return rc;
    lores::ScanWork w;
    *bytes = (size_t)scan_work(dims, backward, nullptr, &w);
    return lores::set_ok();
}

int lores_scan(const lores_scan_dims *dims, const void *q, const void *k, const void *v,
               const float *alpha, const float *beta, const int32_t *lengths,
               const float *S_first, void *o, float *S_last, void *work, size_t work_bytes,
               void *stream) {
    if (const int rc = check_scan(dims)) return rc;
    lores::ScanArgs a;
    if (const int rc = check_scan_inputs(dims, q, k, v, alpha, beta, lengths, S_first, &a)) return rc;
    if (dims->T && !o) return fail(LORES_EINVAL, "o must be a non-NULL device pointer");
    if (!aligned(o, dims->in_bf16 ? 2 : 4)) return fail(LORES_EINVAL, "o must be aligned to its element size");
    if (!aligned(S_last, 16)) return fail(LORES_EINVAL, "S_last must be 16-byte aligned");
    a.o = o;
    a.S = S_last;
    if (!aligned(o, 16)) a.vec_v = 0;
    lores::ScanWork w;
    const uint64_t need = scan_work(dims, 0, work, &w);
    if (const int rc = check_work(need, work, work_bytes)) return rc;
    const hipStream_t s = (hipStream_t)stream;
    consume_stale_hip_error();
    if (!need) return hip_status(lores::launch_scan_rows(dims->in_bf16, a, s), "scan");
    hipError_t e = lores::launch_scan_prep(dims->in_bf16, a, w, s);
    if (e == hipSuccess) e = lores::launch_scan_state(dims->in_bf16, false, a, w, s);
    return hip_status(e, "scan");
}

int lores_scan_backward(const lores_scan_dims *dims, const void *q, const void *k, const void *v,
                        const float *alpha, const float *beta, const int32_t *lengths,
                        const float *S_first, const void *dout, const float *dS_last, void *dq,
                        void *dk, void *dv, float *dalpha, float *dbeta, float *dS_first,
                        void *work, size_t work_bytes, void *stream) {
    if (const int rc = check_scan(dims)) return rc;
    lores::ScanArgs a;
    if (const int rc = check_scan_inputs(dims, q, k, v, alpha, beta, lengths, S_first, &a)) return rc;
    if (dims->T && (!dout || !dq || !dk || !dv || !dalpha || !dbeta))
        return fail(LORES_EINVAL, "dout, dq, dk, dv, dalpha and dbeta must be non-NULL device pointers");
    const uintptr_t el = dims->in_bf16 ? 2 : 4;
    if (!aligned(dout, el) || !aligned(dq, el) || !aligned(dk, el) || !aligned(dv, el) ||
        !aligned(dalpha, 4) || !aligned(dbeta, 4))
        return fail(LORES_EINVAL, "gradients must be aligned to their element size");
    if (!aligned(dS_last, 16) || !aligned(dS_first, 16))
        return fail(LORES_EINVAL, "dS_last and dS_first must be 16-byte aligned");
    a.dout = dout;
    a.dS = dS_last;
    a.dq = dq;
    a.dkey = dk;
    a.dvalue = dv;
    a.dalpha = dalpha;
    a.dbeta = dbeta;
    a.dS0 = dS_first;
    if (!aligned(dout, 16) || !aligned(dv, 16)) a.vec_v = 0;
    a.vec_g = aligned(dq, 16) && aligned(dk, 16);
    lores::ScanWork w;
    std::memset(&w, 0, sizeof w);
    const uint64_t need = scan_work(dims, 1, work, &w);
    if (const int rc = check_work(need, work, work_bytes)) return rc;
    const hipStream_t s = (hipStream_t)stream;
    consume_stale_hip_error();
    hipError_t e = hipSuccess;
    if (dims->T) {
        e = lores::launch_scan_prep(dims->in_bf16, a, w, s);
        if (e == hipSuccess) e = lores::launch_scan_state(dims->in_bf16, true, a, w, s);
    }
    // without tokens this passes dS_last on to dS_first
    if (e == hipSuccess) e = lores::launch_scan_back(dims->in_bf16, a, w, s);
    if (e == hipSuccess && dims->T) e = lores::launch_scan_grad(dims->in_bf16, a, w, s);
    return hip_status(e, "scan backward");
}

int lores_rmsnorm(const void *x, int64_t x_stride, const void *residual, int64_t res_stride,
                  const void *weight, int32_t w_bf16, int64_t rows, int32_t n, int32_t in_bf16,
                  float eps, int32_t out_prec, void *y, float *scales, void *h, void *stream) {
    if (const int rc = check_norm(rows, n, in_bf16, w_bf16, eps)) return rc;
    if (out_prec != LORES_FP32 && out_prec != LORES_BF16 && out_prec != LORES_INT8 &&
        out_prec != LORES_FP8)
        return fail(LORES_EINVAL, "out_prec must be LORES_FP32, LORES_BF16, LORES_INT8 or LORES_FP8 "
                                  "(got %d)", out_prec);
    const bool bytes = out_prec == LORES_INT8 || out_prec == LORES_FP8;
    if (rows == 0) return lores::set_ok();
    if (!x || !weight || !y) return fail(LORES_EINVAL, "x, weight and y must be non-NULL device pointers");
    if (bytes && !scales) return fail(LORES_EINVAL, "8-bit outputs need scales");
    if (residual && !h) return fail(LORES_EINVAL, "a residual needs h for the sum");
    const uintptr_t el = in_bf16 ? 2 : 4, wel = w_bf16 ? 2 : 4;
    const uintptr_t yel = out_prec == LORES_FP32 ? 4 : out_prec == LORES_BF16 ? 2 : 1;
    if (!aligned(x, el) || !aligned(residual, el) || !aligned(h, el) || !aligned(weight, wel) ||
        !aligned(y, yel) || !aligned(scales, 4))
        return fail(LORES_EINVAL, "pointers must be aligned to their element size");
    if (x_stride < n || (residual && res_stride < n))
        return fail(LORES_EINVAL, "rows must be at least n elements apart");
    lores::NormArgs a;
    std::memset(&a, 0, sizeof a);
    a.rows = rows;
    a.n = n;
    a.w_bf16 = w_bf16;
    a.out_prec = out_prec;
    a.eps = eps;
    a.x = x;
    a.x_stride = x_stride;
    a.res = residual;
    a.res_stride = residual ? res_stride : 0;
    a.w = weight;
    a.y = y;
    a.h = h;
    a.scales = scales;
    const bool vec = n % 8 == 0 && aligned(x, 16) && aligned(residual, 16) && aligned(h, 16) &&
                     aligned(weight, 16) && aligned(y, bytes ? 8 : 16) &&
                     x_stride * (int64_t)el % 16 == 0 && a.res_stride * (int64_t)el % 16 == 0;
    consume_stale_hip_error();
    return hip_status(lores::launch_norm(in_bf16, vec, a, (hipStream_t)stream), "norm");
}

int lores_rmsnorm_workspace(int64_t rows, int32_t n, size_t *bytes) {
    if (!bytes) return fail(LORES_EINVAL, "bytes is NULL");
    if (const int rc = check_norm(rows, n, 0, 0, 0.0f)) return rc;
    *bytes = (size_t)lores::norm_groups(rows, n) * n * sizeof(float);
    return lores::set_ok();
}

int lores_rmsnorm_backward(const void *h, int64_t h_stride, const void *weight, int32_t w_bf16,
                           const void *dy, const void *dresidual, int64_t rows, int32_t n,
                           int32_t in_bf16, float eps, void *dx, float *dw, void *work,
                           size_t work_bytes, void *stream) {
    if (const int rc = check_norm(rows, n, in_bf16, w_bf16, eps)) return rc;
    if (!dw) return fail(LORES_EINVAL, "dw must be a non-NULL device pointer");
    if (rows && (!h || !weight || !dy || !dx))
        return fail(LORES_EINVAL, "h, weight, dy and dx must be non-NULL device pointers");
    const uintptr_t el = in_bf16 ? 2 : 4, wel = w_bf16 ? 2 : 4;
    if (!aligned(h, el) || !aligned(dy, el) || !aligned(dresidual, el) || !aligned(dx, el) ||
        !aligned(weight, wel) || !aligned(dw, 4))
        return fail(LORES_EINVAL, "pointers must be aligned to their element size");
    if (rows && h_stride < n) return fail(LORES_EINVAL, "rows must be at least n elements apart");
    lores::NormArgs a;
    std::memset(&a, 0, sizeof a);
    a.rows = rows;
    a.n = n;
    a.w_bf16 = w_bf16;
    a.eps = eps;
    a.x = h;
    a.x_stride = h_stride;
    a.w = weight;
    a.dy = dy;
    a.dres = dresidual;
    a.dx = dx;
    a.dw = dw;
    a.groups = lores::norm_groups(rows, n);
    const uint64_t need = (uint64_t)a.groups * n * sizeof(float);
    if (need && !work) return fail(LORES_EINVAL, "work is NULL (%llu bytes needed)", (unsigned long long)need);
    if (!aligned(work, 16)) return fail(LORES_EINVAL, "work must be 16-byte aligned");
    if (work_bytes < need)
        return fail(LORES_ESIZE, "work holds %llu bytes, %llu needed", (unsigned long long)work_bytes,
                    (unsigned long long)need);
    a.part = (float *)work;
    const bool vec = n % 8 == 0 && aligned(h, 16) && aligned(dy, 16) && aligned(dresidual, 16) &&
                     aligned(dx, 16) && aligned(weight, 16) && h_stride * (int64_t)el % 16 == 0;
    consume_stale_hip_error();
    return hip_status(lores::launch_norm_backward(in_bf16, vec, a, (hipStream_t)stream), "norm backward");
}

}  // extern "C"
