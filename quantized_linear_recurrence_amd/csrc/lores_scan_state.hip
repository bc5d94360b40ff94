// The pass over a sequence's chunks (lores_scan; lores_scan_backward's first
// pass): the state stays in registers from the first chunk to the last.
//
// A wavefront takes 16 value rows of one (sequence, head) and keeps S^T (d_k x
// 16) in the matrix instructions' result layout.  Every product of a chunk
// then takes its right operand from the wavefront's own registers: S for K S^T
// and Q S^T, E = V - gamma K S^T for U = X beta E, U for P U and K^T U.  This
// works because the order of a product's inner index is free: result row
// 4 g + r of tile 2 s + p stands for key (or token) 32 s + 8 g + 4 p + r, which
// is what lane group g wants of a 32-wide operand.  K, Q, X and P are staged in
// LDS once for the work-group's wavefronts; K^T comes from the same rows by
// transposing LDS reads.  Nothing but the chunks' order is sequential.
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

constexpr int NW = 4;                                // wavefronts of a work-group

template <typename IN, int DKP, bool BACK>
struct StateLds {
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NP = BACK ? 1 : sizeof(IN) == 2 ? 2 : 3;
    Planes<NIN, C, DKP> k;
    Planes<NIN, BACK ? 1 : C, DKP> q;
    Planes<3, C, C> x;
    Planes<NP, BACK ? 1 : C, C> p;
    Gates<C> g;
};

// BACK: store every chunk's first state and U instead of outputs.
template <typename IN, int DKP, bool DELTA, bool BACK>
__global__ void __launch_bounds__(64 * NW) lores_scan_state_kernel(const ScanArgs a, const ScanWork w, const int groups) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, MT = C / 16, SB = C / 32, KS = DKP / 32;
    constexpr bool OUT16 = sizeof(IN) == 2;          // outputs end in bf16: two planes carry them
    constexpr int NO = OUT16 ? 2 : 3;
    __shared__ __attribute__((aligned(16))) StateLds<IN, DKP, BACK> sm;
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int unit = blockIdx.x / groups, grp = blockIdx.x - unit * groups;
    const int b = unit / a.H, h = unit - b * a.H, hk = h / (a.H / a.Hk);
    const int col = (grp * NW + wv) * 16 + m;        // the lane's value row of S
    const bool mine = (grp * NW + wv) * 16 < a.dv, ok = col < a.dv;
    int len = a.T;
    if (a.lengths) len = min(max(a.lengths[b], 0), a.T);
    f32x4 st[2 * KS];
#pragma unroll
    for (int t = 0; t < 2 * KS; ++t) {
        const int key = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
        st[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (a.S0 && ok && key < a.dk)
            st[t] = *(const f32x4 *)(a.S0 + ((int64_t)unit * a.dv + col) * a.dk + key);
    }
    const IN *kb = (const IN *)a.k + b * a.ks[0] + hk * a.ks[2];
    const IN *qb = (const IN *)a.q + b * a.qs[0] + hk * a.qs[2];
    const IN *vb = (const IN *)a.v + b * a.vs[0] + h * a.vs[2] + col;
    const int chunks = (len + C - 1) / C;
    for (int ch = 0; ch < chunks; ++ch) {
        const int t0 = ch * C, n = min(len - t0, C);
        const int64_t cu = (int64_t)unit * w.chunks + ch;
        __syncthreads();                             // the last chunk's rows have been read
        stage_rows(sm.k, kb + t0 * a.ks[1], a.ks[1], n, a.dk, a.vec, tid, 64 * NW);
        if constexpr (!BACK) {
            stage_rows(sm.q, qb + t0 * a.qs[1], a.qs[1], n, a.dk, a.vec, tid, 64 * NW);
            stage_planes(sm.p, w.P + cu * w.p_planes * C * C, tid, 64 * NW);
        }
        if constexpr (DELTA) stage_planes(sm.x, w.X + cu * 3 * C * C, tid, 64 * NW);
        if (wv == 0) {
            const int64_t gate = ((int64_t)b * a.T + t0) * a.H + h;
            sm.g.load(a.alpha + gate, a.beta + gate, a.H, n, lane);
        }
        float u[MT][4];                              // V, then E, then U: tokens token_of(mt, 4 g + r)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int tk = token_of(mt, 4 * g + r);
                u[mt][r] = ok && tk < n ? get1(vb + (t0 + tk) * a.vs[1]) : 0.0f;
            }
        __syncthreads();
        if (!mine) continue;
        if constexpr (BACK) {
            float *sp = w.S + cu * a.dk * w.dvp + col;
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int key = 32 * (t >> 1) + 8 * g + 4 * (t & 1) + r;
                    if (key < a.dk) sp[(int64_t)key * w.dvp] = st[t][r];
                }
        }
        f32x4 o[MT];
        if constexpr (DELTA || !BACK) {
            f32x4 e[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) e[mt] = o[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = st[2 * ks + (i >> 2)][i & 3];
                b16x8 sp[3];
                split8(x, sp);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    const int row = token_of(mt, m);
                    b16x8 av[NIN];
                    if constexpr (DELTA) {
                        sm.k.rows(row, 32 * ks + 8 * g, av);
                        e[mt] = mma<3>(av, sp, e[mt]);
                    }
                    if constexpr (!BACK) {
                        sm.q.rows(row, 32 * ks + 8 * g, av);
                        o[mt] = mma<OUT16 ? 2 : 3>(av, sp, o[mt]);
                    }
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const f32x4 gm = *(const f32x4 *)&sm.g.gam[token_of(mt, 4 * g)];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    if constexpr (DELTA) u[mt][r] = fmaf(-gm[r], e[mt][r], u[mt][r]);
                    o[mt][r] *= gm[r];
                }
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const f32x4 be = *(const f32x4 *)&sm.g.be[token_of(mt, 4 * g)];
#pragma unroll
            for (int r = 0; r < 4; ++r) u[mt][r] *= be[r];
        }
        if constexpr (DELTA) {
            f32x4 y[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) y[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = u[2 * sb + (i >> 2)][i & 3];
                b16x8 ep[3];
                split8(x, ep);
#pragma unroll
                for (int mt = 2 * sb; mt < MT; ++mt) {
                    b16x8 xv[3];
                    sm.x.rows(token_of(mt, m), 32 * sb + 8 * g, xv);
                    y[mt] = mma<3>(xv, ep, y[mt]);
                }
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) u[mt][r] = y[mt][r];
        }
        if constexpr (BACK) {
            float *up = w.U + cu * C * w.dvp + col;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    up[(int64_t)token_of(mt, 4 * g + r) * w.dvp] = u[mt][r];
        } else {
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                float x[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) x[i] = u[2 * sb + (i >> 2)][i & 3];
                b16x8 up[NO];
                split8(x, up);
#pragma unroll
                for (int mt = 2 * sb; mt < MT; ++mt) {
                    b16x8 pv[NO];
                    sm.p.rows(token_of(mt, m), 32 * sb + 8 * g, pv);
                    o[mt] = mma<NO>(pv, up, o[mt]);
                }
            }
            IN *op = (IN *)a.o + ((int64_t)b * a.T + t0) * a.H * a.dv + (int64_t)h * a.dv + col;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int tk = token_of(mt, 4 * g + r);
                    if (ok && t0 + tk < a.T) put1(op + (int64_t)tk * a.H * a.dv, o[mt][r]);
                }
        }
        const float ge = sm.g.gam[C - 1];
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t) st[t] *= ge;
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
            float x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = u[2 * sb + (i >> 2)][i & 3] * sm.g.end[32 * sb + 8 * g + i];
            b16x8 up[3];
            split8(x, up);
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t) {
                b16x8 kv[NIN];
                sm.k.template cols<8>(32 * sb, 32 * (t >> 1) + 4 * (t & 1), lane, kv);
                st[t] = mma<3>(kv, up, st[t]);
            }
        }
    }
    if constexpr (!BACK) {
        // whole chunks behind the sequence's end
        if (ok)
            for (int t = chunks * C + g; t < a.T; t += 4)
                put1((IN *)a.o + (((int64_t)b * a.T + t) * a.H + h) * a.dv + col, 0.0f);
        if (a.S && ok) {
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t) {
                const int key = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
                if (key < a.dk) store4(a.S + ((int64_t)unit * a.dv + col) * a.dk + key, st[t]);
            }
        }
    }
}

template <typename IN, int DKP>
hipError_t go(bool backward, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const int groups = (a.dv + 16 * NW - 1) / (16 * NW);
    const dim3 grid((unsigned)((int64_t)a.B * a.H * groups));
    if (backward) {
        if (a.delta) lores_scan_state_kernel<IN, DKP, true, true><<<grid, 64 * NW, 0, s>>>(a, w, groups);
        else lores_scan_state_kernel<IN, DKP, false, true><<<grid, 64 * NW, 0, s>>>(a, w, groups);
    } else {
        if (a.delta) lores_scan_state_kernel<IN, DKP, true, false><<<grid, 64 * NW, 0, s>>>(a, w, groups);
        else lores_scan_state_kernel<IN, DKP, false, false><<<grid, 64 * NW, 0, s>>>(a, w, groups);
    }
    return hipGetLastError();
}

template <typename IN>
hipError_t by_width(bool backward, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (a.dk <= 64) return go<IN, 64>(backward, a, w, s);
    if (a.dk <= 128) return go<IN, 128>(backward, a, w, s);
    return go<IN, 256>(backward, a, w, s);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_state(bool in_bf16, bool backward, const ScanArgs &a, const ScanWork &w,
                             hipStream_t s) {
    return in_bf16 ? scan::by_width<uint16_t>(backward, a, w, s) : scan::by_width<float>(backward, a, w, s);
}

}  // namespace lores
