// Drives the sequence operators' host code (csrc/lores_seq_api.cpp) against
// stand-in launchers: validation before any launch, the workspace, and that a
// failed launch is this call's error.  Built with AddressSanitizer and
// UndefinedBehaviorSanitizer; no GPU is used.
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <string>

#include "../../quantized_linear_recurrence_amd/csrc/lores_seq.h"

static std::string g_text, g_log;
static hipError_t g_sticky = hipSuccess, g_next = hipSuccess;

extern "C" const char *hipGetErrorString(hipError_t) { return "stub"; }
extern "C" hipError_t hipGetLastError(void) {
    const hipError_t e = g_sticky;
    g_sticky = hipSuccess;
    return e;
}

namespace lores {
int set_error(int code, const char *msg) { g_text = msg; return code; }
int set_ok() { g_text.clear(); return LORES_OK; }
static hipError_t rec(const char *what) {
    g_log += what;
    const hipError_t e = g_next != hipSuccess ? g_next : g_sticky;
    g_next = hipSuccess;
    return e;
}
int norm_groups(int64_t rows, int32_t) { return (int)(rows < 1024 ? rows : 1024); }
hipError_t launch_norm(bool, bool vec, const NormArgs &, hipStream_t) { return rec(vec ? "N" : "n"); }
hipError_t launch_norm_backward(bool, bool vec, const NormArgs &, hipStream_t) { return rec(vec ? "B" : "b"); }
hipError_t launch_scan_rows(bool, const ScanArgs &, hipStream_t) { return rec("r"); }
uint64_t plan_scan_work(bool, bool, const ScanArgs &a, void *base, ScanWork *w) {
    std::memset(w, 0, sizeof *w);
    w->X = (uint16_t *)base;
    return (uint64_t)a.T * 1024;
}
hipError_t launch_scan_prep(bool, const ScanArgs &, const ScanWork &, hipStream_t) { return rec("p"); }
hipError_t launch_scan_state(bool, bool back, const ScanArgs &, const ScanWork &, hipStream_t) { return rec(back ? "S" : "s"); }
hipError_t launch_scan_back(bool, const ScanArgs &, const ScanWork &, hipStream_t) { return rec("k"); }
hipError_t launch_scan_grad(bool, const ScanArgs &, const ScanWork &, hipStream_t) { return rec("g"); }
}  // namespace lores

static int g_bad = 0;
#define CHECK(cond)                                                                 \
    do {                                                                            \
        if (!(cond)) { std::printf("line %d: %s\n", __LINE__, #cond); ++g_bad; }    \
    } while (0)

static lores_scan_dims dims(int T) {
    lores_scan_dims d;
    std::memset(&d, 0, sizeof d);
    d.B = 2; d.T = T; d.H = 4; d.H_k = 2; d.d_k = 64; d.d_v = 32; d.delta = 1;
    const int64_t qs[3] = {(int64_t)T * 128, 128, 64}, vs[3] = {(int64_t)T * 128, 128, 32};
    for (int i = 0; i < 3; ++i) { d.q_stride[i] = d.k_stride[i] = qs[i]; d.v_stride[i] = vs[i]; }
    return d;
}

int main() {
    char *const p = (char *)0x100000;                // never dereferenced
    float *const f = (float *)p;
    auto scan = [&](const lores_scan_dims &d, const void *q, size_t bytes, void *work, float *S, void *o) {
        g_log.clear();
        return lores_scan(&d, q, p, p, f, f, nullptr, nullptr, o, S, work, bytes, nullptr);
    };
    lores_scan_dims d = dims(100);
    size_t n = 0;
    CHECK(lores_scan_workspace(&d, 0, &n) == LORES_OK && n == 102400);
    CHECK(lores_scan_workspace(&d, 0, nullptr) == LORES_EINVAL);
    CHECK(lores_scan_workspace(nullptr, 0, &n) == LORES_EINVAL);
    CHECK(scan(d, p, n, p, f, p) == LORES_OK && g_log == "ps" && g_text.empty());
    CHECK(scan(d, p, n - 1, p, f, p) == LORES_ESIZE && g_log.empty() && !g_text.empty());
    CHECK(scan(d, p, n, nullptr, f, p) == LORES_EINVAL && g_log.empty());
    CHECK(scan(d, p, n, p + 16, f, p) == LORES_EINVAL && g_log.empty());
    CHECK(scan(d, nullptr, n, p, f, p) == LORES_EINVAL && g_log.empty());
    CHECK(scan(d, p + 2, n, p, f, p) == LORES_EINVAL && g_log.empty());
    CHECK(scan(d, p, n, p, f, nullptr) == LORES_EINVAL && g_log.empty());
    CHECK(scan(d, p, n, p, (float *)(p + 4), p) == LORES_EINVAL && g_log.empty());
    CHECK(scan(d, p, n, p, nullptr, p) == LORES_OK && g_log == "ps");
    // few tokens: one kernel, no workspace
    lores_scan_dims few = dims(8);
    CHECK(lores_scan_workspace(&few, 0, &n) == LORES_OK && n == 0);
    CHECK(scan(few, p, 0, nullptr, f, p) == LORES_OK && g_log == "r");
    lores_scan_dims none = dims(0);
    g_log.clear();
    CHECK(lores_scan(&none, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, f, nullptr, f, nullptr, 0,
                     nullptr) == LORES_OK && g_log == "r");
    // every limit
    struct { int lores_scan_dims::*m; int v; } lim[] = {
        {&lores_scan_dims::B, 0}, {&lores_scan_dims::B, 65536}, {&lores_scan_dims::T, -1},
        {&lores_scan_dims::T, (1 << 28) + 1}, {&lores_scan_dims::H, 0}, {&lores_scan_dims::H, 513},
        {&lores_scan_dims::H_k, 3}, {&lores_scan_dims::H_k, 0}, {&lores_scan_dims::d_k, 48},
        {&lores_scan_dims::d_k, 288}, {&lores_scan_dims::d_k, 0}, {&lores_scan_dims::d_v, 0},
        {&lores_scan_dims::d_v, 257}, {&lores_scan_dims::in_bf16, 2}, {&lores_scan_dims::delta, 2}};
    for (auto &l : lim) {
        lores_scan_dims e = dims(100);
        e.*l.m = l.v;
        CHECK(lores_scan_workspace(&e, 0, &n) == LORES_EINVAL);
    }
    lores_scan_dims neg = dims(100);
    neg.v_stride[1] = -1;
    CHECK(lores_scan_workspace(&neg, 0, &n) == LORES_EINVAL);
    lores_scan_dims huge = dims(1 << 28);
    huge.B = 65535;
    huge.H = 512;
    CHECK(lores_scan_workspace(&huge, 1, &n) == LORES_EINVAL);
    // backward
    auto back = [&](const lores_scan_dims &e, void *dq, float *dS0, size_t bytes) {
        g_log.clear();
        return lores_scan_backward(&e, p, p, p, f, f, nullptr, nullptr, p, nullptr, dq, p, p, f, f, dS0, p,
                                   bytes, nullptr);
    };
    CHECK(lores_scan_workspace(&d, 1, &n) == LORES_OK && n);
    CHECK(back(d, p, f, n) == LORES_OK && g_log == "pSkg");
    CHECK(back(d, p, nullptr, n) == LORES_OK && g_log == "pSkg");
    CHECK(back(d, nullptr, f, n) == LORES_EINVAL && g_log.empty());
    CHECK(back(d, p, (float *)(p + 4), n) == LORES_EINVAL && g_log.empty());
    CHECK(back(d, p, f, n - 1) == LORES_ESIZE && g_log.empty());
    CHECK(lores_scan_workspace(&few, 1, &n) == LORES_OK && n && back(few, p, f, n) == LORES_OK && g_log == "pSkg");
    CHECK(back(none, nullptr, f, 0) == LORES_OK && g_log == "k");
    // an earlier error is not this call's; this call's launch error ends it
    g_sticky = hipErrorInvalidValue;
    CHECK(lores_scan_workspace(&d, 0, &n) == LORES_OK && scan(d, p, n, p, f, p) == LORES_OK);
    g_next = hipErrorLaunchFailure;
    CHECK(scan(d, p, n, p, f, p) == LORES_EHIP && g_log == "p");
    // norm
    auto norm = [&](const void *x, int64_t xs, const void *res, int64_t rows, int n_, int prec, void *y, float *sc, void *h, float eps) {
        g_log.clear();
        return lores_rmsnorm(x, xs, res, n_, p, 0, rows, n_, 0, eps, prec, y, sc, h, nullptr);
    };
    CHECK(norm(p, 64, nullptr, 4, 64, LORES_FP32, p, nullptr, nullptr, 1e-6f) == LORES_OK && g_log == "N");
    CHECK(norm(p + 4, 64, nullptr, 4, 64, LORES_FP32, p, nullptr, nullptr, 1e-6f) == LORES_OK && g_log == "n");
    CHECK(norm(p, 65, nullptr, 4, 64, LORES_FP32, p, nullptr, nullptr, 1e-6f) == LORES_OK && g_log == "n");
    CHECK(norm(p, 63, nullptr, 4, 64, LORES_FP32, p, nullptr, nullptr, 1e-6f) == LORES_EINVAL && g_log.empty());
    CHECK(norm(p, 64, nullptr, 4, 64, LORES_INT8, p, nullptr, nullptr, 1e-6f) == LORES_EINVAL && g_log.empty());
    CHECK(norm(p, 64, nullptr, 4, 64, LORES_INT8, p, f, nullptr, 1e-6f) == LORES_OK && g_log == "N");
    CHECK(norm(p, 64, p, 4, 64, LORES_FP8, p, f, nullptr, 1e-6f) == LORES_EINVAL && g_log.empty());
    CHECK(norm(p, 64, p, 4, 64, LORES_FP8, p, f, p, 1e-6f) == LORES_OK && g_log == "N");
    CHECK(norm(p, 64, nullptr, 4, 64, LORES_INT4, p, f, nullptr, 1e-6f) == LORES_EINVAL);
    CHECK(norm(p, 64, nullptr, 4, 64, LORES_FP32, p, f, nullptr, -1.0f) == LORES_EINVAL);
    CHECK(norm(p, 64, nullptr, 4, 0, LORES_FP32, p, f, nullptr, 1e-6f) == LORES_EINVAL);
    CHECK(norm(p, 1 << 15, nullptr, 4, LORES_MAX_NORM + 1, LORES_FP32, p, f, nullptr, 1e-6f) == LORES_EINVAL);
    CHECK(norm(nullptr, 64, nullptr, 0, 64, LORES_FP32, nullptr, nullptr, nullptr, 1e-6f) == LORES_OK && g_log.empty());
    CHECK(norm(p, 64, nullptr, -1, 64, LORES_FP32, p, nullptr, nullptr, 1e-6f) == LORES_EINVAL);
    CHECK(lores_rmsnorm_workspace(4, 64, &n) == LORES_OK && n == 4 * 64 * 4);
    auto nb = [&](size_t bytes, float *dw, void *work) {
        g_log.clear();
        return lores_rmsnorm_backward(p, 64, p, 0, p, nullptr, 4, 64, 0, 1e-6f, p, dw, work, bytes, nullptr);
    };
    CHECK(nb(n, f, p) == LORES_OK && g_log == "B");
    CHECK(nb(n - 1, f, p) == LORES_ESIZE && g_log.empty());
    CHECK(nb(n, nullptr, p) == LORES_EINVAL && nb(n, f, nullptr) == LORES_EINVAL);
    if (!g_bad) std::printf("sequence host check ok\n");
    return g_bad ? 1 : 0;
}
