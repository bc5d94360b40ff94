// The inputs' gradients of every chunk (lores_scan_backward), all chunks at
// once.  With S the chunk's first state, dS the gradient of its last, U and H
// from the passes over the chunks, dP = dO U^T (i >= j), Z = H U^T (i > j):
//   dv_i    = beta_i h_i
//   dq      = gamma S^T dO + (dP.D) k
//   dk_j    = (dP.D)^T q + D_Cj dS^T u_j
//             - delta [beta gamma S^T h + (beta Z.D) k + (beta Z.D)^T k]
//   dbeta_i = h_i . v_i - delta [gamma_i k_i . S^T h_i + sum_j (k_i.k_j) D_ij Z_ij]
//   dalpha_t = sum_{i >= t > j} D_it A_ij D_(t-1)j
// where A holds what token i reads of token j without any decay,
//   A_ij = dP_ij q_i.k_j - delta beta_i Z_ij k_i.k_j,
// bordered by the entering state (j = 0: q_i . S^T dO_i - delta beta_i k_i .
// S^T h_i), the leaving one (i = C + 1: k_j . dS^T u_j) and <S, dS>.  The
// double sum runs as two recurrences, along j and along i, without the
// quotient by alpha_t that a sum of decayed products would need: alpha_t = 0
// has the gradient it should have.
//
// A work-group takes one chunk and key head and loops over the value heads
// that share it, so dq and dk are summed in registers in head order.  The
// value columns go by in blocks of 32: dO and the planes of S, dS, U and H, which
// the passes over the chunks have left in operand form, come to LDS directly,
// a block ahead where two fit.  A wavefront owns 16 tokens' rows of dP and Z and
// its share of 16-key strips of the products with S and dS.  That part is
// bound by the matrix instructions (of 16 cycles, one in five instructions
// is another's); dv, the decays and the two recurrences take about a third.
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

constexpr int VB = 32;                               // value columns of a block

template <typename IN, int DKP>
struct GradBlock {                                   // value columns v0 .. v0 + 31
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN;
    Planes<3, VB, DKP> s, ds;
    Planes<3, VB, C> u, h;
    Planes<NIN, C, VB> d;                            // dO
};

template <typename IN, int DKP>
struct GradRows {                                    // when they have all gone by
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NO = sizeof(IN) == 2 ? 2 : 3;
    Planes<NIN, C, DKP> k, q;
    Planes<NO, C, C> p, z;                           // dP.D and -beta Z.D
    float a[C + 1][C + 1];                           // A, row C and column 0 its borders
};

template <typename IN, int DKP>
struct GradLds {
    static constexpr int C = Cfg<IN>::C;
    static constexpr int NS = 2 * sizeof(GradBlock<IN, DKP>) <= 152 * 1024 ? 2 : 1;
    union {
        GradBlock<IN, DKP> b[NS];
        GradRows<IN, DKP> r;
    };
    float part[3][4][C];                             // per wavefront: q.S^T dO, k.S^T h, k.dS^T u
    float hv[C], mz[C], ss[4];
    Gates<C> g;
};

// GROUP: several value heads share the key head.
template <typename IN, int DKP, bool DELTA, bool GROUP>
__global__ void __launch_bounds__(Cfg<IN>::C * 4) lores_scan_grad_kernel(const ScanArgs a, const ScanWork w) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NT = C / 16, SB = C / 32, NW = C / 16, TH = 64 * NW;
    constexpr int ST = DKP / 16 / NT;                // 16-key strips of a wavefront
    constexpr int NO = sizeof(IN) == 2 ? 2 : 3;      // planes of what ends in the inputs' type
    typedef GradLds<IN, DKP> Lds;
    constexpr int NS = Lds::NS;
    __shared__ __attribute__((aligned(16))) Lds sm;
    const int tid = threadIdx.x, lane = tid & 63, mt = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int chunk = blockIdx.x % w.chunks;
    const int bk = blockIdx.x / w.chunks, b = bk / a.Hk, hk = bk - b * a.Hk, G = GROUP ? a.H / a.Hk : 1;
    int len = a.T;
    if (a.lengths) len = min(max(a.lengths[b], 0), a.T);
    const int t0 = chunk * C, n = min(max(len - t0, 0), C), nT = min(a.T - t0, C);
    IN *dqp = (IN *)a.dq + (((int64_t)b * a.T + t0) * a.Hk + hk) * a.dk;
    IN *dkp = (IN *)a.dkey + (((int64_t)b * a.T + t0) * a.Hk + hk) * a.dk;
    if (n == 0) {                                    // behind the sequence's end
        for (int x = tid; x < nT * a.dk; x += TH) {
            const int64_t at = (int64_t)(x / a.dk) * a.Hk * a.dk + x % a.dk;
            put1(dqp + at, 0.0f);
            put1(dkp + at, 0.0f);
        }
        for (int gi = 0; gi < G; ++gi) {
            const int h = hk * G + gi;
            for (int x = tid; x < nT * a.dv; x += TH)
                put1((IN *)a.dvalue + (((int64_t)b * a.T + t0 + x / a.dv) * a.H + h) * a.dv + x % a.dv, 0.0f);
            for (int x = tid; x < nT; x += TH) {
                a.dalpha[((int64_t)b * a.T + t0 + x) * a.H + h] = 0.0f;
                a.dbeta[((int64_t)b * a.T + t0 + x) * a.H + h] = 0.0f;
            }
        }
        return;
    }
    const IN *kc = (const IN *)a.k + b * a.ks[0] + t0 * a.ks[1] + hk * a.ks[2];
    const IN *qc = (const IN *)a.q + b * a.qs[0] + t0 * a.qs[1] + hk * a.qs[2];
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 dqa[NT][GROUP ? ST : 1], dka[NT][GROUP ? ST : 1];   // sums over the heads
    if constexpr (GROUP) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int s = 0; s < ST; ++s) dqa[t][s] = dka[t][s] = zero;
    }
    for (int gi = 0; gi < G; ++gi) {
        const int h = hk * G + gi;
        const int64_t cu = ((int64_t)b * a.H + h) * w.chunks + chunk;
        const int64_t tok = ((int64_t)b * a.T + t0) * a.H + h;   // of the chunk's first token
        const int64_t os = (int64_t)a.H * a.dv;
        const IN *dc = (const IN *)a.dout + tok * a.dv;
        const uint16_t *Sp = w.S + cu * 3 * w.dvp * a.dk, *dSp = w.dS + cu * 3 * w.dvp * a.dk;
        const uint16_t *Up = w.U + cu * 3 * w.dvp * C, *Hp = w.Hm + cu * 3 * w.dvp * C;
        auto fetch = [&](int v0, GradBlock<IN, DKP> &to) {
            const int rows = min(w.dvp - v0, VB);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                direct_rows<VB, DKP, NW>(to.s.x[i], Sp + (i * w.dvp + v0) * a.dk, a.dk, rows, a.dk, mt, lane);
                direct_rows<VB, DKP, NW>(to.ds.x[i], dSp + (i * w.dvp + v0) * a.dk, a.dk, rows, a.dk, mt, lane);
                direct_rows<VB, C, NW>(to.u.x[i], Up + (i * w.dvp + v0) * C, C, rows, C, mt, lane);
                direct_rows<VB, C, NW>(to.h.x[i], Hp + (i * w.dvp + v0) * C, C, rows, C, mt, lane);
            }
            if constexpr (NIN == 1) {
                if (a.vec_v) direct_rows<C, VB, NW>(to.d.x[0], (const uint16_t *)dc + v0, os, n, a.dv - v0, mt, lane);
            }
        };
        // dO rows that do not come directly
        auto place = [&](int v0, GradBlock<IN, DKP> &to) {
            if (NIN == 3 || !a.vec_v) stage_rows(to.d, dc + v0, os, n, a.dv - v0, a.vec_v, tid, TH);
        };
        __syncthreads();                             // the last head's arrays have been read
        if (tid < 4 * C) (&sm.g.al[0])[tid] = w.G[cu * (4 * C) + tid];
        f32x4 dp[NT], z[NT], sdo[NT][ST], sh[NT][ST], dsu[NT][ST];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dp[t] = z[t] = zero;
#pragma unroll
            for (int s = 0; s < ST; ++s) sdo[t][s] = sh[t][s] = dsu[t][s] = zero;
        }
        float ss = 0.0f, hv = 0.0f;                  // <S, dS>; h_i . v_i of token 16 mt + m
        fetch(0, sm.b[0]);
        place(0, sm.b[0]);
        arrived();
        for (int v0 = 0; v0 < a.dv; v0 += VB) {
            GradBlock<IN, DKP> &bl = sm.b[NS == 2 ? v0 / VB & 1 : 0];
            __syncthreads();                         // this block is there, the other has been read
            if (NS == 2 && v0 + VB < a.dv) fetch(v0 + VB, sm.b[(v0 / VB & 1) ^ 1]);
            const int row = 16 * mt + m, c = v0 + 8 * g;          // the lane's token and its 8 columns
            // h of the wavefront's tokens: dv and h . v
            b16x8 ha[3];
            bl.h.template cols<4>(0, 16 * mt, lane, ha);
            float h8[8], v8[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) h8[e] = (float)ha[0][e] + (float)ha[1][e] + (float)ha[2][e];
            const IN *vp = (const IN *)a.v + b * a.vs[0] + (t0 + min(row, n - 1)) * a.vs[1] + h * a.vs[2] + c;
            if constexpr (NIN == 1) {
                b16x8 t[1];
                get_planes(vp, row < n ? a.dv - c : 0, a.vec_v, t);
#pragma unroll
                for (int e = 0; e < 8; ++e) v8[e] = (float)t[0][e];
            } else {
                get8(vp, row < n ? a.dv - c : 0, a.vec_v, v8);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) hv = fmaf(h8[e], v8[e], hv);
            if (row < nT) {
                IN *op = (IN *)a.dvalue + tok * a.dv + row * os + c;
                const float be = sm.g.be[row];
#pragma unroll
                for (int e = 0; e < 8; ++e) h8[e] *= be;
                if (a.vec_v && c + 8 <= a.dv) {
                    if constexpr (NIN == 1) {
                        b16x8 t[1];
                        split8(h8, t);
                        store4((float *)op, __builtin_bit_cast(f32x4, t[0]));
                    } else {
                        store4((float *)op, f32x4{h8[0], h8[1], h8[2], h8[3]});
                        store4((float *)op + 4, f32x4{h8[4], h8[5], h8[6], h8[7]});
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (c + e < a.dv) put1(op + e, h8[e]);
                }
            }
            // <S, dS>: every thread its share of the block
            for (int x = tid; x < VB * (DKP / 8); x += TH) {
                const int r8 = x / (DKP / 8), c8 = (x % (DKP / 8)) * 8;
                b16x8 s3[3], d3[3];
                bl.s.rows(r8, c8, s3);
                bl.ds.rows(r8, c8, d3);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    ss = fmaf((float)s3[0][e] + (float)s3[1][e] + (float)s3[2][e],
                              (float)d3[0][e] + (float)d3[1][e] + (float)d3[2][e], ss);
            }
            // dP and Z, the wavefront's rows
            {
                b16x8 da[NIN];
                bl.d.rows(row, 8 * g, da);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt <= mt) {
                        b16x8 ub[3];
                        bl.u.template cols<4>(0, 16 * nt, lane, ub);
                        dp[nt] = mma<3>(da, ub, dp[nt]);
                        if constexpr (DELTA) z[nt] = mma<3>(ha, ub, z[nt]);
                    }
            }
            // S^T dO, S^T h and dS^T u, the wavefront's strips
            b16x8 sf[ST][3], ef[ST][3];
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                bl.s.template cols<4>(0, 16 * (mt + NT * s), lane, sf[s]);
                bl.ds.template cols<4>(0, 16 * (mt + NT * s), lane, ef[s]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                b16x8 x1[NIN], xh[3], xu[3];
                bl.d.rows(16 * t + m, 8 * g, x1);
                if constexpr (DELTA) bl.h.template cols<4>(0, 16 * t, lane, xh);
                bl.u.template cols<4>(0, 16 * t, lane, xu);
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    sdo[t][s] = mma<3>(x1, sf[s], sdo[t][s]);
                    if constexpr (DELTA) sh[t][s] = mma<3>(xh, sf[s], sh[t][s]);
                    dsu[t][s] = mma<3>(xu, ef[s], dsu[t][s]);
                }
            }
            if (v0 + VB < a.dv) {
                if constexpr (NS == 1) {
                    __syncthreads();
                    fetch(v0 + VB, sm.b[0]);
                }
                place(v0 + VB, sm.b[NS == 2 ? (v0 / VB & 1) ^ 1 : 0]);
                arrived();
            }
        }
        __syncthreads();                             // the blocks have been read: the rows take their place
        if constexpr (NIN == 1) {
            if (a.vec) {
                direct_rows<C, DKP, NW>(sm.r.k.x[0], (const uint16_t *)kc, a.ks[1], n, a.dk, mt, lane);
                direct_rows<C, DKP, NW>(sm.r.q.x[0], (const uint16_t *)qc, a.qs[1], n, a.dk, mt, lane);
            }
        }
        if (NIN == 3 || !a.vec) {
            stage_rows(sm.r.k, kc, a.ks[1], n, a.dk, a.vec, tid, TH);
            stage_rows(sm.r.q, qc, a.qs[1], n, a.dk, a.vec, tid, TH);
        }
        hv += __shfl_xor(hv, 16);
        hv += __shfl_xor(hv, 32);
        if (g == 0) sm.hv[16 * mt + m] = hv;
        ss = sum16(ss);
        ss += __shfl_xor(ss, 16);
        ss += __shfl_xor(ss, 32);
        if (lane == 0) sm.ss[mt] = ss;
        arrived();
        __syncthreads();
        // dots with the rows of q and k over the wavefront's strips; then sdo
        // becomes dq, dsu dk
        {
            float x[NT][4], y[NT][4], e[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) x[t][r] = y[t][r] = e[t][r] = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const f32x4 gm = *(const f32x4 *)&sm.g.gam[16 * t + 4 * g], be = *(const f32x4 *)&sm.g.be[16 * t + 4 * g];
                const f32x4 en = *(const f32x4 *)&sm.g.end[16 * t + 4 * g];
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    const f32x4 kv = sm.r.k.tile(16 * t, 16 * (mt + NT * s), lane);
                    const f32x4 qv = sm.r.q.tile(16 * t, 16 * (mt + NT * s), lane);
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        x[t][r] = fmaf(qv[r], sdo[t][s][r], x[t][r]);
                        if constexpr (DELTA) y[t][r] = fmaf(kv[r], sh[t][s][r], y[t][r]);
                        e[t][r] = fmaf(kv[r], dsu[t][s][r], e[t][r]);
                        sdo[t][s][r] *= gm[r];
                        dsu[t][s][r] *= en[r];
                        if constexpr (DELTA) dsu[t][s][r] = fmaf(-be[r] * gm[r], sh[t][s][r], dsu[t][s][r]);
                    }
                }
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x[t][r] = sum16(x[t][r]);
                    if constexpr (DELTA) y[t][r] = sum16(y[t][r]);
                    e[t][r] = sum16(e[t][r]);
                    if (m == 0) {
                        sm.part[0][mt][16 * t + 4 * g + r] = x[t][r];
                        sm.part[1][mt][16 * t + 4 * g + r] = y[t][r];
                        sm.part[2][mt][16 * t + 4 * g + r] = e[t][r];
                    }
                }
        }
        // A without its borders, dP.D and -beta Z.D
        {
            f32x4 qk[NT], kk[NT];                    // the wavefront's rows of q k^T and k k^T
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) qk[nt] = kk[nt] = zero;
#pragma unroll
            for (int ks = 0; ks < DKP / 32; ++ks) {
                b16x8 qa[NIN], ka[NIN];
                sm.r.q.rows(16 * mt + m, 32 * ks + 8 * g, qa);
                if constexpr (DELTA) sm.r.k.rows(16 * mt + m, 32 * ks + 8 * g, ka);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt <= mt) {
                        b16x8 kb[NIN];
                        sm.r.k.rows(16 * nt + m, 32 * ks + 8 * g, kb);
                        qk[nt] = mma<3>(qa, kb, qk[nt]);
                        if constexpr (DELTA) kk[nt] = mma<3>(ka, kb, kk[nt]);
                    }
            }
            float mz[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            const f32x4 be = *(const f32x4 *)&sm.g.be[16 * mt + 4 * g];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                if (nt > (mt | 1)) continue;
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                if (nt <= mt) decay_tile(sm.g, mt, nt, lane, d);
                const int colj = 16 * nt + m;
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int row = 16 * mt + 4 * g + r;
                    float zr = 0.0f;
                    if constexpr (DELTA) {
                        zr = row > colj ? z[nt][r] : 0.0f;
                        mz[r] = fmaf(kk[nt][r] * d[r], zr, mz[r]);
                        zr *= -be[r];
                        sm.r.z.put(row, colj, zr * d[r]);
                    }
                    sm.r.p.put(row, colj, dp[nt][r] * d[r]);
                    if (row >= colj) sm.r.a[row][colj + 1] = fmaf(dp[nt][r], qk[nt][r], zr * kk[nt][r]);
                }
            }
            if constexpr (DELTA) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    mz[r] = sum16(mz[r]);
                    if (m == 0) sm.mz[16 * mt + 4 * g + r] = mz[r];
                }
            }
        }
        __syncthreads();
        if (tid < C) {
            float x = 0.0f, y = 0.0f, e = 0.0f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                x += sm.part[0][i][tid];
                y += sm.part[1][i][tid];
                e += sm.part[2][i][tid];
            }
            sm.r.a[tid][0] = DELTA ? x - sm.g.be[tid] * y : x;
            sm.r.a[C][tid + 1] = e;
            if (tid == 0) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NT; ++i) s += sm.ss[i];
                sm.r.a[C][0] = s;
            }
            if (tid < nT)
                a.dbeta[tok + (int64_t)tid * a.H] =
                    tid < n ? (DELTA ? sm.hv[tid] - sm.g.gam[tid] * y - sm.mz[tid] : sm.hv[tid]) : 0.0f;
        }
        __syncthreads();
        // along j: what row i has read of everything before token t, decayed to
        // t - 1, kept in place; column t of A holds token t - 1.  Row C goes to
        // the second wavefront.
        if (tid <= C) {
            float u = 0.0f;
#pragma unroll
            for (int t = 0; t < C; t += 8) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = sm.r.a[tid][t + e];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    // what stands right of token i is not read below
                    u = t + e ? fmaf(sm.g.al[t + e - 1], u, x[e]) : x[e];
                    sm.r.a[tid][t + e] = u;
                }
            }
        }
        __syncthreads();
        // along i: those rows decayed back from i to t
        if (tid < C) {
            float s = 0.0f, d = 1.0f;
#pragma unroll
            for (int i0 = 0; i0 < C; i0 += 8) {
                float x[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = sm.r.a[i0 + e][tid];
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (i0 + e > tid) d *= sm.g.al[i0 + e];
                    if (i0 + e >= tid) s = fmaf(d, x[e], s);
                }
            }
            s = fmaf(d, sm.r.a[C][tid], s);
            if (tid < nT) a.dalpha[tok + (int64_t)tid * a.H] = tid < n ? s : 0.0f;
        }
        // dq += (dP.D) k;  dk += (dP.D)^T q + (-beta Z.D) k + (-beta Z.D)^T k
#pragma unroll
        for (int sb = 0; sb < SB; ++sb) {
            b16x8 kv[ST][NIN], qv[ST][NIN];
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                sm.r.k.template cols<4>(32 * sb, 16 * (mt + NT * s), lane, kv[s]);
                sm.r.q.template cols<4>(32 * sb, 16 * (mt + NT * s), lane, qv[s]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                b16x8 x[NO], y[NO];
                if (t >= 2 * sb) {                   // rows t read tokens of block sb
                    sm.r.p.rows(16 * t + m, 32 * sb + 8 * g, x);
                    if constexpr (DELTA) sm.r.z.rows(16 * t + m, 32 * sb + 8 * g, y);
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        sdo[t][s] = mma<NO>(x, kv[s], sdo[t][s]);
                        if constexpr (DELTA) dsu[t][s] = mma<NO>(y, kv[s], dsu[t][s]);
                    }
                }
                if (t < 2 * sb + 2) {                // tokens t are read by rows of block sb
                    sm.r.p.template cols<4>(32 * sb, 16 * t, lane, x);
                    if constexpr (DELTA) sm.r.z.template cols<4>(32 * sb, 16 * t, lane, y);
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        dsu[t][s] = mma<NO>(x, qv[s], dsu[t][s]);
                        if constexpr (DELTA) dsu[t][s] = mma<NO>(y, kv[s], dsu[t][s]);
                    }
                }
            }
        }
        if constexpr (GROUP) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    dqa[t][s] += sdo[t][s];
                    dka[t][s] += dsu[t][s];
                }
        }
        if (!GROUP || gi + 1 == G) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int s = 0; s < ST; ++s)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int row = 16 * t + 4 * g + r, key = 16 * (mt + NT * s) + m;
                        if (row < nT && key < a.dk) {
                            const int64_t at = (int64_t)row * a.Hk * a.dk + key;
                            put1(dqp + at, GROUP ? dqa[t][GROUP ? s : 0][r] : sdo[t][s][r]);
                            put1(dkp + at, GROUP ? dka[t][GROUP ? s : 0][r] : dsu[t][s][r]);
                        }
                    }
        }
    }
}

template <typename IN, int DKP>
hipError_t go(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.B * a.Hk * w.chunks));
    constexpr int TH = Cfg<IN>::C * 4;
    if (a.H > a.Hk) {
        if (a.delta) lores_scan_grad_kernel<IN, DKP, true, true><<<grid, TH, 0, s>>>(a, w);
        else lores_scan_grad_kernel<IN, DKP, false, true><<<grid, TH, 0, s>>>(a, w);
    } else {
        if (a.delta) lores_scan_grad_kernel<IN, DKP, true, false><<<grid, TH, 0, s>>>(a, w);
        else lores_scan_grad_kernel<IN, DKP, false, false><<<grid, TH, 0, s>>>(a, w);
    }
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

hipError_t launch_scan_grad(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    return in_bf16 ? scan::by_width<uint16_t>(a, w, s) : scan::by_width<float>(a, w, s);
}

}  // namespace lores
