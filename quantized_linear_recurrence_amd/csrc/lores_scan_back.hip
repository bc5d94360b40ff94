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
//
// Measured (bf16, d_k = d_v = 128, delta): 128 units x 2048 tokens 230 us, 0.77
// GB at 3.4 TB/s, matrix instructions busy for 21 % of the time.  With 1024
// wavefronts there is one per SIMD, and each waits on its own chain of products;
// issuing products and splits in a fixed interleaving changed it by 1 %.  At
// d_k > 128, fp32 with delta spills 436 to 456 bytes a lane.
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

template <typename IN, int DKP, int NW>
struct BackLds {
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN;
    Planes<NIN, C, DKP> k, q;
    Tri<3, C> x, p;
    Gates<C> g;
    Tile<IN, C> d[NW];
};

// Two chunks' rows where they fit: the next chunk's arrive while one is
// worked on.
template <typename L> __host__ __device__ constexpr int stages() { return 2 * sizeof(L) <= 160 * 1024 ? 2 : 1; }

// FAST: q and k rows that can be read 16 bytes at a time (a.vec); VEC: dO's
// (a.vec_v).  NW: wavefronts of a work-group.
template <typename IN, int DKP, bool DELTA, bool FAST, bool VEC, int NW>
__global__ void __launch_bounds__(64 * NW) lores_scan_back_kernel(const ScanArgs a, const ScanWork w, const int groups) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, MT = C / 16, SB = C / 32, KS = DKP / 32, TH = 64 * NW;
    typedef BackLds<IN, DKP, NW> Lds;
    constexpr bool IN16 = sizeof(IN) == 2;
    constexpr int NS = stages<Lds>();
    __shared__ __attribute__((aligned(16))) Lds lds[NS];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    int unit, grp;
    if (!unit_of((int)block_at(blockIdx.x, blockIdx.y), groups, a.B * a.H, &unit, &grp)) return;
    const int b = unit / a.H, h = unit - b * a.H, hk = h / (a.H / a.Hk);
    const int col0 = (grp * NW + wv) * 16, col = col0 + m;
    const bool mine = col0 < a.dv, ok = col < a.dv;
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
    const int64_t os = (int64_t)a.H * a.dv;
    const IN *ob = (const IN *)a.dout + ((int64_t)b * a.T * a.H + h) * a.dv + (mine ? col0 : 0);
    RowFetch<C, IN16 ? 8 : DKP, TH> kf, qf;          // fp32 only
    IN df[VEC ? 1 : MT][4];
    // a chunk's rows to stage `to`, in parts (see the forward pass)
    auto fetch = [&](int part, int ch, Lds &to) {
        const int t0 = ch * C, n = min(len - t0, C);
        const int64_t cu = (int64_t)unit * w.chunks + ch;
        if (part == 0) {
            if constexpr (FAST && IN16) direct_rows<C, DKP, NW>(to.k.x[0], kb + t0 * a.ks[1], a.ks[1], n, a.dk, wv, lane);
            else if constexpr (FAST) kf.load(kb + t0 * a.ks[1], a.ks[1], n, a.dk, tid);
        } else if (part == 1) {
            if constexpr (FAST && IN16) direct_rows<C, DKP, NW>(to.q.x[0], qb + t0 * a.qs[1], a.qs[1], n, a.dk, wv, lane);
            else if constexpr (FAST) qf.load(qb + t0 * a.qs[1], a.qs[1], n, a.dk, tid);
        } else if (part == 2) {
            direct_block<sizeof(to.p), NW>(w.P + cu * (3 * Tri<1, C>::NB * 1024), &to.p, wv, lane);
            if constexpr (DELTA) direct_block<sizeof(to.x), NW>(w.X + cu * (3 * Tri<1, C>::NB * 1024), &to.x, wv, lane);
            direct_block<sizeof(to.g), NW>(w.G + cu * (6 * C), &to.g, wv, lane);
        } else if (mine) {
            if constexpr (VEC) {
                to.d[wv].fetch(ob + t0 * os, os, n, a.dv - col0, lane);
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        df[mt][r] = ob[(t0 + token_of(mt, r) + min(8 * g, n - 1 - token_of(mt, r))) * os + (ok ? m : 0)];
            }
        }
    };
    // fp32 rows, and rows at odd addresses, through registers
    auto place = [&](int ch, Lds &to) {
        const int t0 = ch * C, n = min(len - t0, C);
        if constexpr (!FAST) {
            stage_rows(to.k, kb + t0 * a.ks[1], a.ks[1], n, a.dk, false, tid, TH);
            stage_rows(to.q, qb + t0 * a.qs[1], a.qs[1], n, a.dk, false, tid, TH);
        } else if constexpr (!IN16) {
            kf.store(to.k, n, a.dk, tid);
            qf.store(to.q, n, a.dk, tid);
        }
    };
    const int chunks = (len + C - 1) / C;
    if (chunks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch(i, chunks - 1, lds[(NS - 1) & (chunks - 1)]);
        place(chunks - 1, lds[(NS - 1) & (chunks - 1)]);
        arrived();
    }
    for (int ch = chunks - 1; ch >= 0; --ch) {
        const int t0 = ch * C, n = min(len - t0, C);
        const int64_t cu = (int64_t)unit * w.chunks + ch;
        const Lds &sm = lds[(NS - 1) & ch];
        Lds &next = lds[(NS - 1) & (ch ^ 1)];
        const bool more = NS == 2 && ch;
        f32x4 d[MT];                                 // dO at tokens token_of(mt, 4 g + r)
        if constexpr (!VEC) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) d[mt][r] = get1(&df[mt][r]);
        }
        __syncthreads();                             // this chunk is there, the other stage has been read
        if (!mine) {                                 // a wavefront without value rows only helps to fetch
            if (more) {
#pragma unroll
                for (int i = 0; i < 4; ++i) fetch(i, ch - 1, next);
            }
        } else {
        if constexpr (VEC) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float x[4];
                sm.d[wv].get(mt, lane, x);
#pragma unroll
                for (int r = 0; r < 4; ++r) d[mt][r] = x[r];
            }
        }
        // nothing behind the sequence's end or d_v counts, whatever stands there
        if (n < C || col0 + 16 > a.dv) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) d[mt][r] = ok && 8 * g < n - token_of(mt, r) ? d[mt][r] : 0.0f;
        }
        if (more) fetch(0, ch - 1, next);
        // the gradient at the chunk's end
        {
            float *sp0 = w.dS + cu * w.dvp * a.dk;
            const uint32_t at = (uint32_t)col * (uint32_t)a.dk + 8 * g;
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t)
                if (32 * (t >> 1) < a.dk) store4(sp0 + (at + 32 * (t >> 1) + 4 * (t & 1)), st[t]);
        }
        f32x4 y[MT], z[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) y[mt] = z[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        // y = K dS^T, and beside it z = P^T dO: P's rows are the outputs i, its
        // columns the tokens j <= i that they read
        b16x8 pv[SB][MT][3], dp[SB][NIN];
        {
            b16x8 kv[2][MT][NIN], sp[2][3];
            auto rows = [&](int ks, int p) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sm.k.rows(token_of(mt, m), 32 * ks + 8 * g, kv[p][mt]);
            };
            auto split = [&](int ks, int p) {
                float x[8];
                pair8(st[2 * ks], st[2 * ks + 1], x);
                split8(x, sp[p]);
            };
            rows(0, 0);
            split(0, 0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                fence();
                if (ks + 1 < KS) rows(ks + 1, (ks + 1) & 1);
                if (ks < SB) {
#pragma unroll
                    for (int mt = 0; mt < 2 * ks + 2; ++mt)
                        sm.p.template cols<8>(ks, mt >> 1, 4 * (mt & 1), lane, pv[ks][mt]);
                    float x[8];
                    pair8(d[2 * ks], d[2 * ks + 1], x);
                    split8(x, dp[ks]);
                }
                fence();
                if (ks + 1 < KS) split(ks + 1, (ks + 1) & 1);
                mma_all<MT>(kv[ks & 1], sp[ks & 1], y);
                if (ks >= 1 && ks - 1 < SB) {
                    if (ks == 1) mma_all<2>(pv[0], dp[0], z);
                    else if constexpr (SB > 1) mma_all<MT>(pv[SB - 1], dp[SB - 1], z);
                }
            }
            fence();
            if (KS - 1 < SB) {
                if (KS == 1) mma_all<2>(pv[0], dp[0], z);
                else if constexpr (SB > 1) mma_all<MT>(pv[SB - 1], dp[SB - 1], z);
            }
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const f32x4 en = *(const f32x4 *)&sm.g.end[token_of(mt, 4 * g)];
#pragma unroll
            for (int r = 0; r < 4; ++r) y[mt][r] = fmaf(en[r], y[mt][r], z[mt][r]);
        }
        if (more) fetch(1, ch - 1, next);
        b16x8 kt[2 * KS][NIN], qt[2 * KS][NIN];
        auto turned = [&](int sb) {
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t) {
                sm.q.template cols<8>(32 * sb, 32 * (t >> 1) + 4 * (t & 1), lane, qt[t]);
                if constexpr (DELTA) sm.k.template cols<8>(32 * sb, 32 * (t >> 1) + 4 * (t & 1), lane, kt[t]);
            }
        };
        f32x4 hm[MT];
        if constexpr (DELTA) {
            b16x8 xv[SB][MT][3];
#pragma unroll
            for (int sb = 0; sb < SB; ++sb)
#pragma unroll
                for (int mt = 0; mt < 2 * sb + 2; ++mt)
                    sm.x.template cols<8>(sb, mt >> 1, 4 * (mt & 1), lane, xv[sb][mt]);
            fence();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) hm[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                float x[8];
                b16x8 yp[3];
                pair8(y[2 * sb], y[2 * sb + 1], x);
                split8(x, yp);
                if (sb == 0) mma_all<2>(xv[0], yp, hm);
                else mma_all<MT>(xv[SB - 1], yp, hm);
            }
            fence();
        } else {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) hm[mt] = y[mt];
        }
        if (more) fetch(2, ch - 1, next);
        turned(0);
        fence();
        {
            float *h0 = w.Hm + cu * w.dvp * C;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) store4(h0 + (uint32_t)(col * C + token_of(mt, 4 * g)), hm[mt]);
        }
        if (more) fetch(3, ch - 1, next);
        const float ge = sm.g.gam[C - 1];
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t) st[t] *= ge;
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
            float x[8], v[8];
            pair8(d[2 * sb], d[2 * sb + 1], x);
            pair8(hm[2 * sb], hm[2 * sb + 1], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int tk = 32 * sb + 8 * g + i;
                x[i] *= sm.g.gam[tk];
                v[i] *= -(sm.g.be[tk] * sm.g.gam[tk]);
            }
            b16x8 xp[3], vp[3];
            split8(x, xp);
            mma_all<2 * KS>(qt, xp, st);
            if constexpr (DELTA) {
                split8(v, vp);
                mma_all<2 * KS>(kt, vp, st);
            }
            if (sb + 1 < SB) {
                fence();
                turned(sb + 1);
            }
        }
        }
        if (ch) {
            if constexpr (NS == 1) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) fetch(i, ch - 1, lds[0]);
            }
            place(ch - 1, next);
            arrived();
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

template <typename IN, int DKP, bool DELTA, bool FAST, bool VEC, int NW>
hipError_t go(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const int groups = (a.dv + 16 * NW - 1) / (16 * NW);
    const dim3 grid = grid_of(((int64_t)a.B * a.H + 7) / 8 * 8 * groups);
    lores_scan_back_kernel<IN, DKP, DELTA, FAST, VEC, NW><<<grid, 64 * NW, 0, s>>>(a, w, groups);
    return hipGetLastError();
}

template <typename IN, int DKP, bool DELTA>
hipError_t by_rows(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (!a.vec) return go<IN, DKP, DELTA, false, false, 4>(a, w, s);
    if (!a.vec_v) return go<IN, DKP, DELTA, true, false, 4>(a, w, s);
    // With delta, fp32 operands of 128 keys leave too few registers for eight
    // (256 units x 512 tokens, all kernels: 947 us by eight, 818 by four;
    // without delta 567 and 619)
    if constexpr (DKP <= (sizeof(IN) == 4 && DELTA ? 64 : 128))
        if (scan_waves(a) == 8) return go<IN, DKP, DELTA, true, true, 8>(a, w, s);
    return go<IN, DKP, DELTA, true, true, 4>(a, w, s);
}

template <typename IN, bool DELTA>
hipError_t by_width(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (a.dk <= 64) return by_rows<IN, 64, DELTA>(a, w, s);
    if (a.dk <= 128) return by_rows<IN, 128, DELTA>(a, w, s);
    return by_rows<IN, 256, DELTA>(a, w, s);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_back(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (a.delta) return in_bf16 ? scan::by_width<uint16_t, true>(a, w, s) : scan::by_width<float, true>(a, w, s);
    return in_bf16 ? scan::by_width<uint16_t, false>(a, w, s) : scan::by_width<float, false>(a, w, s);
}

}  // namespace lores
