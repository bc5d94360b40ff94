// The pass back over a sequence's chunks (lores_scan_backward): the gradient
// of the state stays in registers from the last chunk to the first.
//
// With dS the gradient at a chunk's end and dO its outputs':
//   dU = P^T dO + diag(D_Cj) K dS^T,   H = X^T dU,
//   dS <- gamma_C dS + (gamma dO)^T Q - delta (beta gamma H)^T K
// The mirror image of the forward pass, in the same layout: a wavefront takes
// 16 value rows and holds dS^T (d_k x 16), the left operands come from LDS (P^T,
// X^T, Q^T and K^T by transposing reads), the right ones from its registers.
// Every chunk's dS and H are stored for the inputs' gradients.
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

constexpr int NW = 4;

template <typename IN, int DKP>
struct BackLds {
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN;
    Planes<NIN, C, DKP> k, q;
    Planes<3, C, C> x, p;
    Gates<C> g;
};

template <typename IN, int DKP, bool DELTA>
__global__ void __launch_bounds__(64 * NW) lores_scan_back_kernel(const ScanArgs a, const ScanWork w, const int groups) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, MT = C / 16, SB = C / 32, KS = DKP / 32;
    __shared__ __attribute__((aligned(16))) BackLds<IN, DKP> sm;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int unit = blockIdx.x / groups, grp = blockIdx.x - unit * groups;
    const int b = unit / a.H, h = unit - b * a.H, hk = h / (a.H / a.Hk);
    const int col = (grp * NW + wv) * 16 + m;
    const bool mine = (grp * NW + wv) * 16 < a.dv, ok = col < a.dv;
    int len = a.T;
    if (a.lengths) len = min(max(a.lengths[b], 0), a.T);
    f32x4 st[2 * KS];
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t) {
        const int key = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
        st[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (a.dS && ok && key < a.dk)
            st[t] = *(const f32x4 *)(a.dS + ((int64_t)unit * a.dv + col) * a.dk + key);
    }
    const IN *kb = (const IN *)a.k + b * a.ks[0] + hk * a.ks[2];
    const IN *qb = (const IN *)a.q + b * a.qs[0] + hk * a.qs[2];
    const IN *ob = (const IN *)a.dout + ((int64_t)b * a.T * a.H + h) * a.dv + col;
    for (int ch = (len + C - 1) / C - 1; ch >= 0; --ch) {
        const int t0 = ch * C, n = min(len - t0, C);
        const int64_t cu = (int64_t)unit * w.chunks + ch;
        __syncthreads();                             // the last chunk's rows have been read
        stage_rows(sm.k, kb + t0 * a.ks[1], a.ks[1], n, a.dk, a.vec, tid, 64 * NW);
        stage_rows(sm.q, qb + t0 * a.qs[1], a.qs[1], n, a.dk, a.vec, tid, 64 * NW);
        stage_planes(sm.p, w.P + cu * 3 * C * C, tid, 64 * NW);
        if constexpr (DELTA) stage_planes(sm.x, w.X + cu * 3 * C * C, tid, 64 * NW);
        if (wv == 0) {
            const int64_t gate = ((int64_t)b * a.T + t0) * a.H + h;
            sm.g.load(a.alpha + gate, a.beta + gate, a.H, n, lane);
        }
        float d[MT][4];                              // dO at tokens token_of(mt, 4 g + r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tk = token_of(mt, 4 * g + r);
                d[mt][r] = ok && tk < n ? get1(ob + (int64_t)(t0 + tk) * a.H * a.dv) : 0.0f;
            }
        __syncthreads();
        if (!mine) continue;
        float *sp = w.dS + cu * a.dk * w.dvp + col;
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r;
                if (key < a.dk) sp[(int64_t)key * w.dvp] = st[t][r];
            }
        f32x4 y[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) y[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = st[2 * ks + (i >> 2)][i & 3];
            b16x8 sp3[3];
            split8(x, sp3);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                b16x8 kv[NIN];
                sm.k.rows(token_of(mt, m), 32 * ks + 8 * g, kv);
                y[mt] = mma<3>(kv, sp3, y[mt]);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) y[mt] *= *(const f32x4 *)&sm.g.end[token_of(mt, 4 * g)];
        // + P^T dO: rows are the written tokens j, the inner index the outputs i >= j
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = d[2 * sb + (i >> 2)][i & 3];
            b16x8 dp[NIN];
            split8(x, dp);
#pragma unroll
            for (int mt = 0; mt < 2 * sb + 2; ++mt) {
                b16x8 pv[3];
                sm.p.template cols<8>(32 * sb, 32 * (mt >> 1) + 4 * (mt & 1), lane, pv);
                y[mt] = mma<3>(pv, dp, y[mt]);
            }
        }
        f32x4 hm[MT];
        if constexpr (DELTA) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) hm[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = y[2 * sb + (i >> 2)][i & 3];
                b16x8 yp[3];
                split8(x, yp);
#pragma unroll
                for (int mt = 0; mt < 2 * sb + 2; ++mt) {
                    b16x8 xv[3];
                    sm.x.template cols<8>(32 * sb, 32 * (mt >> 1) + 4 * (mt & 1), lane, xv);
                    hm[mt] = mma<3>(xv, yp, hm[mt]);
                }
            }
        } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) hm[mt] = y[mt];
        }
        float *hp = w.Hm + cu * C * w.dvp + col;
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) hp[(int64_t)token_of(mt, 4 * g + r) * w.dvp] = hm[mt][r];
        const float ge = sm.g.gam[C - 1];
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t) st[t] *= ge;
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
            float x[8], z[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int tk = 32 * sb + 8 * g + i;
                x[i] = d[2 * sb + (i >> 2)][i & 3] * sm.g.gam[tk];
                z[i] = DELTA ? -hm[2 * sb + (i >> 2)][i & 3] * (sm.g.be[tk] * sm.g.gam[tk]) : 0.0f;
            }
            b16x8 xp[3], zp[3];
            split8(x, xp);
            if constexpr (DELTA) split8(z, zp);
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t) {
                b16x8 rv[NIN];
                sm.q.template cols<8>(32 * sb, 32 * (t >> 1) + 4 * (t & 1), lane, rv);
                st[t] = mma<3>(rv, xp, st[t]);
                if constexpr (DELTA) {
                    sm.k.template cols<8>(32 * sb, 32 * (t >> 1) + 4 * (t & 1), lane, rv);
                    st[t] = mma<3>(rv, zp, st[t]);
                }
            }
        }
    }
    if (a.dS0 && ok) {
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t) {
            const int key = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
            if (key < a.dk) store4(a.dS0 + ((int64_t)unit * a.dv + col) * a.dk + key, st[t]);
        }
    }
}

template <typename IN, int DKP>
hipError_t go(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const int groups = (a.dv + 16 * NW - 1) / (16 * NW);
    const dim3 grid((unsigned)((int64_t)a.B * a.H * groups));
    if (a.delta) lores_scan_back_kernel<IN, DKP, true><<<grid, 64 * NW, 0, s>>>(a, w, groups);
    else lores_scan_back_kernel<IN, DKP, false><<<grid, 64 * NW, 0, s>>>(a, w, groups);
    return hipGetLastError();
}

template <typename IN>
hipError_t by_width(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (a.dk <= 64) return go<IN, 64>(a, w, s);
    if (a.dk <= 128) return go<IN, 128>(a, w, s);
    return go<IN, 256>(a, w, s);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_back(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    return in_bf16 ? scan::by_width<uint16_t>(a, w, s) : scan::by_width<float>(a, w, s);
}

}  // namespace lores
