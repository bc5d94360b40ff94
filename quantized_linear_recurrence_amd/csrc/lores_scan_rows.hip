// The recurrence over a few tokens (lores_scan at few tokens, scan_rows_tokens), token
// by token in fp32:
//   S' = alpha S,  g = beta (v - delta S' k),  S = S' + g k^T,
//   o = S q = S' q + g (k . q)
// The rows of S do not meet, so 8 lanes hold one value row in registers (4
// neighbouring elements of every 32) for the whole call; the three dot
// products of a token are reduced over 8 lanes together.  With one token the
// call is bound by reading and writing the fp32 state once: 16-byte accesses,
// 128 bytes of a row per instruction and 8 lanes.  64 x 32 units of 128 x 128
// take 48 us (5.6 TB/s); a further token costs about 14 us of issue and of
// waiting for its q and k (fetching them a token ahead took so many registers
// that it cost more: 98 instead of 63, 21 us a token).
#include "lores_seq.h"

namespace lores {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float bf2f(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

__device__ __forceinline__ float get1(const float *p) { return *p; }
__device__ __forceinline__ float get1(const uint16_t *p) { return bf2f(*p); }
__device__ __forceinline__ void put1(float *p, float x) { *p = x; }
__device__ __forceinline__ void put1(uint16_t *p, float x) {
    const __bf16 b = (__bf16)x;                      // to nearest even
    *p = __builtin_bit_cast(uint16_t, b);
}

__device__ __forceinline__ f32x4 get4(const float *p, bool vec) {
    return vec ? *(const f32x4 *)p : f32x4{p[0], p[1], p[2], p[3]};
}
__device__ __forceinline__ f32x4 get4(const uint16_t *p, bool vec) {
    if (vec) {
        const u32x2 w = *(const u32x2 *)p;
        return f32x4{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xffff0000u),
                     __uint_as_float(w.y << 16), __uint_as_float(w.y & 0xffff0000u)};
    }
    return f32x4{bf2f(p[0]), bf2f(p[1]), bf2f(p[2]), bf2f(p[3])};
}

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
    return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, true));
}
// Sum over 8 neighbouring lanes, in all of them: pairs, quads, and the other
// quad mirrored.
__device__ __forceinline__ float sum8(float x) {
    x = dpp_add<0xb1>(x);                            // quad_perm 1 0 3 2
    x = dpp_add<0x4e>(x);                            // quad_perm 2 3 0 1
    return dpp_add<0x141>(x);                        // row_half_mirror
}

// NC = d_k / 32
template <typename IN, int NC>
__global__ void __launch_bounds__(256) lores_scan_rows_kernel(const ScanArgs a, const int tiles) {
    const int block = (int)block_at(blockIdx.x, blockIdx.y), unit = block / tiles, tile = block - unit * tiles;
    if (unit >= a.B * a.H) return;
    const int b = unit / a.H, h = unit - b * a.H, hk = h / (a.H / a.Hk);
    const int l = threadIdx.x & 7, row = tile * 32 + (threadIdx.x >> 3);
    if (row >= a.dv) return;                         // whole groups of 8 lanes
    int len = a.T;
    if (a.lengths) len = min(max(a.lengths[b], 0), a.T);
    const int64_t srow = ((int64_t)unit * a.dv + row) * (32 * NC) + 4 * l;
    f32x4 s[NC], k[NC], q[NC];
#pragma unroll
    for (int c = 0; c < NC; ++c)
        s[c] = a.S0 ? *(const f32x4 *)(a.S0 + srow + 32 * c) : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const IN *qp = (const IN *)a.q + b * a.qs[0] + hk * a.qs[2] + 4 * l;
    const IN *kp = (const IN *)a.k + b * a.ks[0] + hk * a.ks[2] + 4 * l;
    const IN *vp = (const IN *)a.v + b * a.vs[0] + h * a.vs[2] + row;
    IN *op = (IN *)a.o + ((int64_t)b * a.T * a.H + h) * a.dv + row;
    const float *ap = a.alpha + (int64_t)b * a.T * a.H + h, *bp = a.beta + (int64_t)b * a.T * a.H + h;
    const bool vec = a.vec;
    for (int t = 0; t < len; ++t) {
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            k[c] = get4(kp + t * a.ks[1] + 32 * c, vec);
            q[c] = get4(qp + t * a.qs[1] + 32 * c, vec);
        }
        const float al = ap[(int64_t)t * a.H], be = bp[(int64_t)t * a.H];
        const float v = get1(vp + t * a.vs[1]);
        float sk = 0.0f, sq = 0.0f, kq = 0.0f;
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[c][e] *= al;
                sk = fmaf(s[c][e], k[c][e], sk);
                sq = fmaf(s[c][e], q[c][e], sq);
                kq = fmaf(k[c][e], q[c][e], kq);
            }
        sk = sum8(sk);
        sq = sum8(sq);
        kq = sum8(kq);
        const float g = be * (a.delta ? v - sk : v);
#pragma unroll
        for (int c = 0; c < NC; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[c][e] = fmaf(g, k[c][e], s[c][e]);
        if (l == 0) put1(op + (int64_t)t * a.H * a.dv, fmaf(g, kq, sq));
    }
    if (l == 0)
        for (int t = len; t < a.T; ++t) put1(op + (int64_t)t * a.H * a.dv, 0.0f);
    if (a.S) {
#pragma unroll
        for (int c = 0; c < NC; ++c) *(f32x4 *)(a.S + srow + 32 * c) = s[c];
    }
}

template <typename IN>
hipError_t by_width(const ScanArgs &a, hipStream_t s) {
    const int tiles = (a.dv + 31) / 32;
    const dim3 grid = grid_of((int64_t)a.B * a.H * tiles);
    switch (a.dk / 32) {
        case 1: lores_scan_rows_kernel<IN, 1><<<grid, 256, 0, s>>>(a, tiles); break;
        case 2: lores_scan_rows_kernel<IN, 2><<<grid, 256, 0, s>>>(a, tiles); break;
        case 3: lores_scan_rows_kernel<IN, 3><<<grid, 256, 0, s>>>(a, tiles); break;
        case 4: lores_scan_rows_kernel<IN, 4><<<grid, 256, 0, s>>>(a, tiles); break;
        case 5: lores_scan_rows_kernel<IN, 5><<<grid, 256, 0, s>>>(a, tiles); break;
        case 6: lores_scan_rows_kernel<IN, 6><<<grid, 256, 0, s>>>(a, tiles); break;
        case 7: lores_scan_rows_kernel<IN, 7><<<grid, 256, 0, s>>>(a, tiles); break;
        default: lores_scan_rows_kernel<IN, 8><<<grid, 256, 0, s>>>(a, tiles); break;
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_scan_rows(bool in_bf16, const ScanArgs &a, hipStream_t s) {
    return in_bf16 ? by_width<uint16_t>(a, s) : by_width<float>(a, s);
}

}  // namespace lores
