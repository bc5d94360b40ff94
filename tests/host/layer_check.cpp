// Drives the layer operators' host code (csrc/lores_layer_api.cpp) against
// stand-in launchers: validation before any launch, how rows are read, the
// workspaces, and that a failed launch is this call's error.  Built with
// AddressSanitizer and UndefinedBehaviorSanitizer; no GPU is used.
#include <cmath>
#include <cstdio>
#include <cstring>
#include <string>

#include "../../quantized_linear_recurrence_amd/csrc/lores_layer.h"

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
static hipError_t rec(const std::string &what) {
    g_log = what;
    const hipError_t e = g_next != hipSuccess ? g_next : g_sticky;
    g_next = hipSuccess;
    return e;
}
static std::string mode_name(int mode) { return mode == ROWS_VEC ? "vec" : "odd"; }
int gated_groups(int64_t tokens, int32_t heads, int32_t, int32_t per_head) { return (int)(per_head ? tokens : tokens * heads); }
int block_groups(int64_t rows, int32_t) { return (int)rows; }
hipError_t launch_gated(bool, int mode, const GatedArgs &, hipStream_t) { return rec("gated " + mode_name(mode)); }
hipError_t launch_gated_backward(bool, int mode, const GatedArgs &, hipStream_t) { return rec("gated back " + mode_name(mode)); }
hipError_t launch_block(bool, int mode, const BlockArgs &, hipStream_t) { return rec("block " + mode_name(mode)); }
hipError_t launch_block_backward(bool, int mode, const BlockArgs &, hipStream_t) { return rec("block back " + mode_name(mode)); }
hipError_t launch_mx_quant(bool, bool vec, const MxRows &, hipStream_t) { return rec(vec ? "quant vec" : "quant"); }
hipError_t launch_mx_dequant(bool, const MxRows &, hipStream_t) { return rec("dequant"); }
hipError_t launch_mx_product(bool fp8, bool, const MxProduct &, hipStream_t) { return rec(fp8 ? "product fp8" : "product"); }
}  // namespace lores

static int g_bad = 0;
#define CHECK(cond)                                                                 \
    do {                                                                            \
        g_log.clear();                                                              \
        if (!(cond)) { std::printf("line %d: %s (%s)\n", __LINE__, #cond, g_text.c_str()); ++g_bad; } \
    } while (0)
#define OK(call, what) CHECK((call) == LORES_OK && g_log == what)
#define BAD(call) CHECK((call) == LORES_EINVAL && g_log.empty() && !g_text.empty())

int main() {
    char *p = (char *)0x100000;
    float *f = (float *)p;
    uint8_t *u = (uint8_t *)p;
    size_t n = 0;
    {
        lores_gated_dims d;
        auto fresh = [&] {
            std::memset(&d, 0, sizeof d);
            d.tokens = 6; d.heads = 4; d.n = 64; d.act = LORES_ACT_SILU; d.eps = 1e-6f;
            d.x_stride[0] = d.gate_stride[0] = 256; d.x_stride[1] = d.gate_stride[1] = 64;
        };
        auto go = [&](const void *x, const void *z, int prec, void *y, uint8_t *s) {
            return lores_gated_norm(&d, x, z, p, prec, y, s, nullptr);
        };
        fresh();
        OK(go(p, p, LORES_FP32, p, nullptr), "gated vec");
        OK(go(p + 4, p, LORES_FP32, p, nullptr), "gated odd");
        OK(go(p, p + 4, LORES_MXFP4, p, u), "gated odd");
        OK(go(p, p, LORES_MXFP4, p, u + 1), "gated vec");
        BAD(go(p, p, LORES_MXFP4, p, nullptr));
        BAD(go(p, p, LORES_MXFP4, p + 4, u));
        BAD(go(p + 2, p, LORES_FP32, p, nullptr));
        BAD(go(p, p, LORES_FP32, p + 2, nullptr));
        BAD(go(nullptr, p, LORES_FP32, p, nullptr));
        BAD(go(p, nullptr, LORES_FP32, p, nullptr));
        BAD(go(p, p, LORES_FP32, nullptr, nullptr));
        for (int prec : {(int)LORES_INT8, (int)LORES_FP8, (int)LORES_INT4, -1, 17}) BAD(go(p, p, prec, p, u));
        BAD(lores_gated_norm(nullptr, p, p, p, LORES_FP32, p, nullptr, nullptr));
        d.x_stride[0] = 257;
        OK(go(p, p, LORES_FP32, p, nullptr), "gated odd");
        d.x_stride[0] = 0;
        OK(go(p, p, LORES_FP32, p, nullptr), "gated vec");
        d.x_stride[0] = -1;
        BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.n = 40;
        OK(go(p, p, LORES_BF16, p, nullptr), "gated vec");
        BAD(go(p, p, LORES_MXFP4, p, u));
        fresh(); d.n = 0; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.n = LORES_MAX_NORM + 1; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.heads = 0; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.heads = LORES_MAX_HEADS + 1; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.tokens = -1; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.tokens = (int64_t)1 << 62; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.tokens = 0x7fffffff / 4 + 1; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.act = 3; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.gate_first = 2; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.per_head = -1; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.eps = -1.0f; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.eps = NAN; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.in_bf16 = 2; BAD(go(p, p, LORES_FP32, p, nullptr));
        fresh(); d.tokens = 0;
        OK(go(nullptr, nullptr, LORES_FP32, nullptr, nullptr), "");
        fresh();
        CHECK(lores_gated_norm_workspace(&d, &n) == LORES_OK && n == 24 * 64 * 4);
        d.per_head = 1;
        CHECK(lores_gated_norm_workspace(&d, &n) == LORES_OK && n == 6 * 4 * 64 * 4);
        BAD(lores_gated_norm_workspace(&d, nullptr));
        auto back = [&](const void *dy, void *dx, void *dz, float *dw, void *work, size_t bytes) {
            return lores_gated_norm_backward(&d, p, p, p, dy, dx, dz, dw, work, bytes, nullptr);
        };
        OK(back(p, p, p, f, p, n), "gated back vec");
        OK(back(p + 4, p, p, f, p, n), "gated back odd");
        CHECK(back(p, p, p, f, p, n - 1) == LORES_ESIZE && g_log.empty());
        BAD(back(p, p, p, f, nullptr, n));
        BAD(back(p, p, p, f, p + 8, n));
        BAD(back(p, p, p, nullptr, p, n));
        BAD(back(p, nullptr, p, f, p, n));
        BAD(back(p, p, nullptr, f, p, n));
        BAD(back(nullptr, p, p, f, p, n));
        d.tokens = 0;
        OK(lores_gated_norm_backward(&d, nullptr, nullptr, nullptr, nullptr, nullptr, nullptr, f, nullptr, 0, nullptr),
           "gated back vec");
        fresh();
        g_next = hipErrorLaunchFailure;
        CHECK(go(p, p, LORES_FP32, p, nullptr) == LORES_EHIP);
        g_sticky = hipErrorLaunchFailure;
        OK(go(p, p, LORES_FP32, p, nullptr), "gated vec");
    }
    {
        lores_block_dims d;
        auto fresh = [&] {
            std::memset(&d, 0, sizeof d);
            d.rows = 6; d.n = 64; d.eps = 1e-6f; d.scale = 0.5f;
            d.x_stride = d.res_stride = d.gate_stride = 64;
        };
        auto go = [&](const void *x, const void *r, const void *z, const void *w, int prec, void *y, void *s, void *h) {
            return lores_block_norm(&d, x, r, z, w, p, prec, y, s, h, nullptr);
        };
        fresh();
        OK(go(p, p, p, p, LORES_FP32, p, nullptr, p), "block vec");
        OK(go(p, nullptr, nullptr, nullptr, LORES_FP32, p, nullptr, p), "block vec");
        OK(go(p, p + 4, nullptr, nullptr, LORES_FP32, p, nullptr, p), "block odd");
        OK(go(p, p + 4, nullptr, nullptr, LORES_MXFP4, p, u, p), "block odd");
        OK(go(p, p, p, p, LORES_INT8, p, f, p), "block vec");
        BAD(go(p, p, p, p, LORES_INT8, p, nullptr, p));
        BAD(go(p, p, p, p, LORES_FP8, p, p + 2, p));
        BAD(go(p, p, p, p, LORES_MXFP4, p, nullptr, p));
        BAD(go(p, p, p, p, LORES_MXFP4, p + 8, u, p));
        BAD(go(p, p, p, p, LORES_INT4, p, f, p));
        BAD(go(p, p, p, p, LORES_FP32, p, nullptr, nullptr));
        BAD(go(nullptr, p, p, p, LORES_FP32, p, nullptr, p));
        BAD(go(p, p, p + 2, p, LORES_FP32, p, nullptr, p));
        BAD(lores_block_norm(&d, p, p, p, p, nullptr, LORES_FP32, p, nullptr, p, nullptr));
        d.gate_stride = 0;
        OK(go(p, p, p, p, LORES_FP32, p, nullptr, p), "block vec");
        d.gate_stride = 65;
        OK(go(p, p, p, p, LORES_FP32, p, nullptr, p), "block odd");
        d.gate_stride = 63; BAD(go(p, p, p, p, LORES_FP32, p, nullptr, p));
        fresh(); d.x_stride = (int64_t)1 << 41; BAD(go(p, p, p, p, LORES_FP32, p, nullptr, p));
        fresh(); d.scale = INFINITY; BAD(go(p, p, p, p, LORES_FP32, p, nullptr, p));
        fresh(); d.rows = -1; BAD(go(p, p, p, p, LORES_FP32, p, nullptr, p));
        fresh(); d.rows = (int64_t)1 << 31; BAD(go(p, p, p, p, LORES_FP32, p, nullptr, p));
        fresh(); d.n = 48; BAD(go(p, p, p, p, LORES_MXFP4, p, u, p));
        fresh();
        CHECK(lores_block_norm_workspace(&d, &n) == LORES_OK && n == 6 * 64 * 2 * 4);
        auto back = [&](const void *h, const void *z, const void *w, void *dz, float *dw, size_t bytes) {
            return lores_block_norm_backward(&d, p, h, z, w, p, p, nullptr, p, p, dz, dw, f, p, bytes, nullptr);
        };
        OK(back(p, p, p, p, f, n), "block back vec");
        OK(back(p, nullptr, nullptr, nullptr, nullptr, n), "block back vec");
        OK(back(p + 4, p, p, p, f, n), "block back odd");
        BAD(back(p, p, p, nullptr, f, n));
        BAD(back(p, p, p, p, nullptr, n));
        BAD(back(nullptr, p, p, p, f, n));
        CHECK(back(p, p, p, p, f, n - 1) == LORES_ESIZE);
        fresh(); d.rows = 0;
        OK(lores_block_norm(&d, nullptr, nullptr, nullptr, nullptr, nullptr, LORES_FP32, nullptr, nullptr, nullptr, nullptr), "");
    }
    {
        auto quant = [&](const void *x, int64_t xs, int64_t rows, int n_, int bf, uint8_t *c, uint8_t *s) {
            return lores_mx_quant(x, xs, rows, n_, bf, c, s, nullptr);
        };
        OK(quant(p, 64, 4, 64, 0, u, u), "quant vec");
        OK(quant(p + 2, 64, 4, 64, 1, u, u), "quant");
        OK(quant(p, 65, 4, 64, 1, u, u), "quant");
        OK(quant(nullptr, 64, 0, 64, 0, nullptr, nullptr), "");
        OK(quant(p, 0, 4, 64, 1, u, u), "quant vec");
        BAD(quant(p, 63, 4, 64, 0, u, u));
        BAD(quant(p, -64, 4, 64, 0, u, u));
        BAD(quant(p, 64, 4, 48, 0, u, u));
        BAD(quant(p, 64, 4, 0, 0, u, u));
        BAD(quant(p, 64, -1, 64, 0, u, u));
        BAD(quant(p, (1 << 24) + 32, 4, (1 << 24) + 32, 0, u, u));
        BAD(quant(p, 1 << 24, (1 << 14) + 1, 1 << 24, 0, u, u));
        BAD(quant(p, 64, 4, 64, 2, u, u));
        BAD(quant(p, 64, 4, 64, 0, u + 8, u));
        BAD(quant(p, 64, 4, 64, 0, u, u + 2));
        BAD(quant(p + 2, 64, 4, 64, 0, u, u));
        OK(lores_mx_dequant(u, u, 4, 64, 1, p, nullptr), "dequant");
        BAD(lores_mx_dequant(u, u, 4, 64, 1, p + 8, nullptr));
        BAD(lores_mx_dequant(u, nullptr, 4, 64, 1, p, nullptr));
        BAD(lores_mx_dequant(u, u, 4, 33, 1, p, nullptr));
        auto mul = [&](const void *a, const void *as, int ap, int64_t M, int N, int K, int op, void *out) {
            return lores_mx_matmul(a, as, ap, u, u, M, N, K, op, out, nullptr);
        };
        OK(mul(p, p, LORES_MXFP4, 3, 5, 96, LORES_FP32, p), "product");
        OK(mul(p, p, LORES_FP8, 3, 5, 96, LORES_BF16, p), "product fp8");
        OK(mul(nullptr, nullptr, LORES_MXFP4, 0, 5, 96, LORES_BF16, nullptr), "");
        BAD(mul(p, p, LORES_FP8, 3, 5, 96, LORES_FP32, p));
        BAD(mul(p, p, LORES_INT8, 3, 5, 96, LORES_BF16, p));
        BAD(mul(p, p, LORES_MXFP4, 3, 5, 96, LORES_INT8, p));
        BAD(mul(p, p, LORES_MXFP4, 3, 5, 80, LORES_BF16, p));
        BAD(mul(p, p, LORES_MXFP4, 3, 0, 96, LORES_BF16, p));
        BAD(mul(p, p, LORES_MXFP4, -1, 5, 96, LORES_BF16, p));
        BAD(mul(p, p, LORES_MXFP4, 0x7fffffff, 1 << 24, 96, LORES_BF16, p));
        BAD(mul(p + 8, p, LORES_MXFP4, 3, 5, 96, LORES_BF16, p));
        BAD(mul(p, p + 2, LORES_MXFP4, 3, 5, 96, LORES_BF16, p));
        BAD(mul(p, p, LORES_MXFP4, 3, 5, 96, LORES_BF16, p + 4));
        BAD(mul(p, nullptr, LORES_MXFP4, 3, 5, 96, LORES_BF16, p));
        g_next = hipErrorLaunchFailure;
        CHECK(mul(p, p, LORES_MXFP4, 3, 5, 96, LORES_BF16, p) == LORES_EHIP);
    }
    if (g_bad) return 1;
    std::printf("ok\n");
    return 0;
}
