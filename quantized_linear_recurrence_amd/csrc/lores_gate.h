// A gate's activation and its slope, for the norms that take a gate.
#pragma once

#include "lores_rows.h"

namespace lores {
namespace {

// 1 / (1 + e^-z), as 2^(-z log2 e) and a reciprocal (1 ulp each).  The exponent as one
// float would be off by up to 2^-24 |z| log2 e (s of z = -80 by 3.4e-6 of itself, which
// shows in fp32 results).  A bf16 z has 8 bits: its product with the first 15 of log2 e is
// exact, and the rest goes in as a factor 1 - z 0x1.480fb6p-18 (off by 2^-24 at 70).  For
// fp32 the rounded part is carried on as a factor 1 + x ln 2.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    constexpr float log2e = 0x1.715476p+0f;
    if constexpr (sizeof(T) == 2) {
        // (the factor's z is at most 150, by its bits: an infinity there would meet e = 0)
        const float e = __builtin_amdgcn_exp2f(-z * 0x1.7154p+0f);
        const float f = fmaf(__int_as_float(min(__float_as_int(z), 0x43160000)), -0x1.480fb6p-18f, 1.0f);
        return __builtin_amdgcn_rcpf(fmaf(e, f, 1.0f));
    } else {
        // beyond +-150 the result is 0 or 1; NaN goes by itself
        const float m = -fminf(fmaxf(z, -150.0f), 150.0f);
        const float t = m * log2e;
        const float lo = fmaf(m, 0x1.4ae0cp-26f, fmaf(m, log2e, -t));   // log2 e = log2e + 0x1.4ae0cp-26
        const float e = __builtin_amdgcn_exp2f(t);
        // (a product, whose infinite e stays one whatever lo's sign)
        const float s = __builtin_amdgcn_rcpf(1.0f + e * fmaf(lo, 0x1.62e43p-1f, 1.0f));
        return z != z ? z : s;
    }
}

// a(z) from z and s = 1 / (1 + e^-z)
__device__ __forceinline__ float gate_value(int act, float z, float s) {
    return act == LORES_ACT_SILU ? z * s : act == LORES_ACT_SIGMOID ? s : z;
}
// da/dz
__device__ __forceinline__ float gate_slope(int act, float z, float s) {
    return act == LORES_ACT_SILU ? s * fmaf(z, 1.0f - s, 1.0f) : act == LORES_ACT_SIGMOID ? s * (1.0f - s) : 1.0f;
}

}  // namespace
}  // namespace lores
