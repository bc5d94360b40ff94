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
// value columns go by in blocks of 32: S, dS, U and H become planes in LDS on
// the way from registers, where the next block's arrive while one is worked
// on.  All results are made turned over (a lane holds four neighbours of one
// token's row, see the prep kernel), which also leaves the sums over keys to
// two lane exchanges.  A wavefront owns strips of 16 keys of the products with
// S and dS, and a share of 16 tokens' rows of dP and Z.
//
// Measured (bf16, d_k = d_v = 128, delta): 128 units x 2048 tokens 464 us, 1.3
// GB (0.8 of it S, dS, U and H) at 2.8 TB/s, matrix instructions busy for 19 %
// of the time.  Two thirds of a chunk go to the value columns, bound by the
// loads and the planes' way through LDS; the last third is the double sum of
// dalpha and the products with q and k, short steps between barriers with two
// wavefronts per SIMD.  At d_k > 128 a wavefront holds two strips and spills (84
// to 684 bytes a lane at bf16, 156 at fp32 with delta and shared heads).
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
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN;
    Planes<NIN, C, DKP> k, q;
    Tri<3, C> p, z;                                  // dP.D and -beta Z.D
    float a[C + 1][C + 1];                           // A, row C and column 0 its borders
};

// The sums over the heads of a group: a wavefront's own results, kept in LDS
// where they fit beside the rest (they would not leave enough registers).
template <typename IN, int DKP, int NW>
constexpr bool group_in_lds() {
    return (sizeof(GradBlock<IN, DKP>) > sizeof(GradRows<IN, DKP>) ? sizeof(GradBlock<IN, DKP>) : sizeof(GradRows<IN, DKP>)) +
               Cfg<IN>::C * DKP * 8 <= 152 * 1024;
}

template <typename IN, int DKP, int NW, bool GROUP>
struct GradLds {
    static constexpr int C = Cfg<IN>::C;
    f32x4 acc[GROUP && group_in_lds<IN, DKP, NW>() ? C * DKP / 2 : 1];
    union {
        GradBlock<IN, DKP> b;
        GradRows<IN, DKP> r;
    };
    float part[3][NW][C];                            // per wavefront: q.S^T dO, k.S^T h, k.dS^T u
    float hv[2][C], mz[2][C], ss[NW];
    Gates<C> g;
};

// Wavefronts: a strip each where d_k has that many, two to a 16-token row.
template <typename IN, int DKP>
constexpr int grad_waves() { return Cfg<IN>::C / 16 * (DKP > 64 ? 2 : 1); }

// GROUP: several value heads share the key head.
template <typename IN, int DKP, bool DELTA, bool GROUP>
__global__ void __launch_bounds__((64 * grad_waves<IN, DKP>())) lores_scan_grad_kernel(const ScanArgs a, const ScanWork w) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NT = C / 16, SB = C / 32, NW = grad_waves<IN, DKP>(), TH = 64 * NW;
    constexpr int ST = DKP / 16 / NW, RW = NW / NT;  // strips of a wavefront, wavefronts of a row
    __shared__ __attribute__((aligned(16))) GradLds<IN, DKP, NW, GROUP> sm;
    constexpr bool ACC = GROUP && group_in_lds<IN, DKP, NW>();
    const int tid0 = threadIdx.x, wv = __builtin_amdgcn_readfirstlane(tid0 >> 6);
    const int mt = wv / RW, half = wv % RW;          // the wavefront's row of tiles, its share of it
    int b, hk, chunk;
    if (!chunk_of((int)block_at(blockIdx.x, blockIdx.y), a, w, &b, &hk, &chunk)) return;
    const int G = GROUP ? a.H / a.Hk : 1;
    int len = a.T;
    if (a.lengths) len = min(max(a.lengths[b], 0), a.T);
    const int t0 = chunk * C, n = min(max(len - t0, 0), C), nT = min(a.T - t0, C);
    IN *dqp = (IN *)a.dq + (((int64_t)b * a.T + t0) * a.Hk + hk) * a.dk;
    IN *dkp = (IN *)a.dkey + (((int64_t)b * a.T + t0) * a.Hk + hk) * a.dk;
    if (n == 0) {                                    // behind the sequence's end
        for (int x = tid0; x < nT * a.dk; x += TH) {
            const int64_t at = (int64_t)(x / a.dk) * a.Hk * a.dk + x % a.dk;
            put1(dqp + at, 0.0f);
            put1(dkp + at, 0.0f);
        }
        for (int gi = 0; gi < G; ++gi) {
            const int h = hk * G + gi;
            for (int x = tid0; x < nT * a.dv; x += TH)
                put1((IN *)a.dvalue + (((int64_t)b * a.T + t0 + x / a.dv) * a.H + h) * a.dv + x % a.dv, 0.0f);
            for (int x = tid0; x < nT; x += TH) {
                a.dalpha[((int64_t)b * a.T + t0 + x) * a.H + h] = 0.0f;
                a.dbeta[((int64_t)b * a.T + t0 + x) * a.H + h] = 0.0f;
            }
        }
        return;
    }
    const IN *kc = (const IN *)a.k + b * a.ks[0] + t0 * a.ks[1] + hk * a.ks[2];
    const IN *qc = (const IN *)a.q + b * a.qs[0] + t0 * a.qs[1] + hk * a.qs[2];
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 dqa[NT][GROUP && !ACC ? ST : 1], dka[NT][GROUP && !ACC ? ST : 1];   // sums over the heads
    if constexpr (GROUP && !ACC) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int s = 0; s < ST; ++s) dqa[t][s] = dka[t][s] = zero;
    }
    for (int gi = 0; gi < G; ++gi) {
        // the lane's addresses are made anew for every head: kept over the loop they
        // would take more registers than there are
        int lane = tid0 & 63;
        if constexpr (GROUP) asm volatile("" : "+v"(lane));
        const int tid = wv * 64 + lane, m = lane & 15, g = lane >> 4;
        const int h = hk * G + gi;
        const int64_t cu = ((int64_t)b * a.H + h) * w.chunks + chunk;
        const int64_t tok = ((int64_t)b * a.T + t0) * a.H + h;   // of the chunk's first token
        const int64_t os = (int64_t)a.H * a.dv;
        const IN *dc = (const IN *)a.dout + tok * a.dv;
        // a block's pieces of 8: S and dS, U and H, dO
        constexpr int NSP = (VB * (DKP / 8) + TH - 1) / TH, NUP = (2 * VB * (C / 8) + TH - 1) / TH;
        constexpr int NDP = (C * (VB / 8) + TH - 1) / TH;
        f32x4 fs[NSP][2], fe[NSP][2], fu[NUP][2];
        b16x8 fd[NDP][NIN];
        const float *Sp = w.S + cu * w.dvp * a.dk, *dSp = w.dS + cu * w.dvp * a.dk;
        const float *Up = w.U + cu * w.dvp * C, *Hp = w.Hm + cu * w.dvp * C;
        // In parts that the products are interleaved with: 0 S, 1 dS, 2 U and H,
        // 3 dO.
        auto fetch = [&](int part, int v0) {
            const int last = w.dvp - v0 - 1;         // rows behind it are blanked in place()
            if (part < 2) {
#pragma unroll
                for (int i = 0; i < NSP; ++i) {
                    const int x = tid + i * TH, r = min(x / (DKP / 8), last), c = (x % (DKP / 8)) * 8;
                    const uint32_t at = (uint32_t)((v0 + r) * a.dk + (c < a.dk ? c : 0));
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        if (part == 0) fs[i][j] = *(const f32x4 *)(Sp + at + 4 * j);
                        else fe[i][j] = *(const f32x4 *)(dSp + at + 4 * j);
                    }
                }
            } else if (part == 2) {
#pragma unroll
                for (int i = 0; i < NUP; ++i) {
                    const int x = tid + i * TH, y = x % (VB * (C / 8)), r = min(y / (C / 8), last), c = (y % (C / 8)) * 8;
                    const float *p = (x < VB * (C / 8) ? Up : Hp) + (uint32_t)((v0 + r) * C + c);
#pragma unroll
                    for (int j = 0; j < 2; ++j) fu[i][j] = *(const f32x4 *)(p + 4 * j);
                }
            } else {
#pragma unroll
                for (int i = 0; i < NDP; ++i) {
                    const int x = tid + i * TH, r = x / (VB / 8), c = (x % (VB / 8)) * 8;
                    get_planes(dc + (int64_t)r * os + v0 + c, x < C * (VB / 8) && r < n ? a.dv - v0 - c : 0, a.vec_v, fd[i]);
                }
            }
        };
        float ss = 0.0f, hv = 0.0f;                  // <S, dS>; h_i . v_i of token 16 mt + m
        auto place = [&](int v0) {
            const int rows = w.dvp - v0;
#pragma unroll
            for (int i = 0; i < NSP; ++i) {
                const int x = tid + i * TH, r = x / (DKP / 8), c = (x % (DKP / 8)) * 8;
                if (VB * (DKP / 8) % TH != 0 && x >= VB * (DKP / 8)) continue;
                float s8[8], e8[8];
                pair8(fs[i][0], fs[i][1], s8);
                pair8(fe[i][0], fe[i][1], e8);
                if (r >= rows || c >= a.dk) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) s8[e] = e8[e] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) ss = fmaf(s8[e], e8[e], ss);
                b16x8 p[3];
                split8(s8, p);
                sm.b.s.put8(r, c, p);
                split8(e8, p);
                sm.b.ds.put8(r, c, p);
            }
#pragma unroll
            for (int i = 0; i < NUP; ++i) {
                const int x = tid + i * TH, y = x % (VB * (C / 8)), r = y / (C / 8), c = (y % (C / 8)) * 8;
                if (2 * VB * (C / 8) % TH != 0 && x >= 2 * VB * (C / 8)) continue;
                float u8[8];
                pair8(fu[i][0], fu[i][1], u8);
                if (r >= rows) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) u8[e] = 0.0f;
                }
                b16x8 p[3];
                split8(u8, p);
                if (x < VB * (C / 8)) sm.b.u.put8(r, c, p);
                else sm.b.h.put8(r, c, p);
            }
#pragma unroll
            for (int i = 0; i < NDP; ++i) {
                const int x = tid + i * TH;
                if (x < C * (VB / 8)) sm.b.d.put8(x / (VB / 8), (x % (VB / 8)) * 8, fd[i]);
            }
        };
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch(i, 0);
        __syncthreads();                             // the last head's arrays have been read
        for (int i = tid; i < 6 * C; i += TH) (&sm.g.al[0])[i] = w.G[cu * (6 * C) + i];
        // turned over: the lane's token is the column, its rows four neighbours
        f32x4 dp[NT], z[NT], sdo[NT][ST], sh[NT][ST], dsu[NT][ST];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dp[t] = z[t] = zero;
#pragma unroll
            for (int s = 0; s < ST; ++s) sdo[t][s] = sh[t][s] = dsu[t][s] = zero;
        }
        for (int v0 = 0; v0 < a.dv; v0 += VB) {
            if (v0) __syncthreads();                 // the last block has been read
            place(v0);
            __syncthreads();
            const bool more = v0 + VB < a.dv;
            const int row = 16 * mt + m, c = v0 + 8 * g;          // the lane's token and its 8 columns
            // S^T dO, S^T h and dS^T u, the wavefront's strips
            b16x8 sf[ST][3], ef[ST][3];
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                sm.b.s.template cols<4>(0, 16 * (wv + NW * s), lane, sf[s]);
                sm.b.ds.template cols<4>(0, 16 * (wv + NW * s), lane, ef[s]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (more) {
                    fetch(t * 4 / NT, v0 + VB);
                    if (NT == 2) fetch(t * 4 / NT + 1, v0 + VB);
                }
                b16x8 x1[NIN], xh[3], xu[3];
                sm.b.d.rows(16 * t + m, 8 * g, x1);
                if constexpr (DELTA) sm.b.h.template cols<4>(0, 16 * t, lane, xh);
                sm.b.u.template cols<4>(0, 16 * t, lane, xu);
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    sdo[t][s] = mma(sf[s], x1, sdo[t][s]);
                    if constexpr (DELTA) sh[t][s] = mma(sf[s], xh, sh[t][s]);
                    dsu[t][s] = mma(ef[s], xu, dsu[t][s]);
                }
            }
            // dP and Z, the wavefront's tiles
            b16x8 ha[3];
            sm.b.h.template cols<4>(0, 16 * mt, lane, ha);
            {
                b16x8 da[NIN];
                sm.b.d.rows(row, 8 * g, da);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t <= mt && t % RW == half) {
                        b16x8 ub[3];
                        sm.b.u.template cols<4>(0, 16 * t, lane, ub);
                        dp[t] = mma(ub, da, dp[t]);
                        if constexpr (DELTA) z[t] = mma(ub, ha, z[t]);
                    }
            }
            // h of the row's tokens: dv and h . v
            if (v0 / VB % RW == half) {
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
            }
        }
        __syncthreads();                             // the blocks have been read: the rows take their place
        if constexpr (NIN == 1) {
            if (a.vec) {
                direct_rows<C, DKP, NW>(sm.r.k.x[0], (const uint16_t *)kc, a.ks[1], n, a.dk, wv, lane);
                direct_rows<C, DKP, NW>(sm.r.q.x[0], (const uint16_t *)qc, a.qs[1], n, a.dk, wv, lane);
            }
        }
        if (NIN == 3 || !a.vec) {
            stage_rows(sm.r.k, kc, a.ks[1], n, a.dk, a.vec, tid, TH);
            stage_rows(sm.r.q, qc, a.qs[1], n, a.dk, a.vec, tid, TH);
        }
        hv += __shfl_xor(hv, 16);
        hv += __shfl_xor(hv, 32);
        if (g == 0) sm.hv[half][16 * mt + m] = hv;
        ss = sum16(ss);
        ss += __shfl_xor(ss, 16);
        ss += __shfl_xor(ss, 32);
        if (lane == 0) sm.ss[wv] = ss;
        arrived();
        __syncthreads();
        // dots with the rows of q and k over the wavefront's strips; then sdo
        // becomes dq, dsu dk
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int tk = 16 * t + m;
            const float gm = sm.g.gam[tk], bg = sm.g.be[tk] * gm, en = sm.g.end[tk];
            float x = 0.0f, y = 0.0f, e = 0.0f;
#pragma unroll
            for (int s = 0; s < ST; ++s) {
                const f32x4 kv = sm.r.k.get4(tk, 16 * (wv + NW * s) + 4 * g);
                const f32x4 qv = sm.r.q.get4(tk, 16 * (wv + NW * s) + 4 * g);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    x = fmaf(qv[r], sdo[t][s][r], x);
                    if constexpr (DELTA) y = fmaf(kv[r], sh[t][s][r], y);
                    e = fmaf(kv[r], dsu[t][s][r], e);
                    sdo[t][s][r] *= gm;
                    dsu[t][s][r] *= en;
                    if constexpr (DELTA) dsu[t][s][r] = fmaf(-bg, sh[t][s][r], dsu[t][s][r]);
                }
            }
            x += __shfl_xor(x, 16);
            x += __shfl_xor(x, 32);
            if constexpr (DELTA) {
                y += __shfl_xor(y, 16);
                y += __shfl_xor(y, 32);
            }
            e += __shfl_xor(e, 16);
            e += __shfl_xor(e, 32);
            if (g == 0) {
                sm.part[0][wv][tk] = x;
                sm.part[1][wv][tk] = y;
                sm.part[2][wv][tk] = e;
            }
        }
        // A without its borders, dP.D and -beta Z.D: the wavefront's tiles
        {
            f32x4 qk[NT], kk[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) qk[t] = kk[t] = zero;
#pragma unroll
            for (int ks = 0; ks < DKP / 32; ++ks) {
                b16x8 qa[NIN], ka[NIN];
                sm.r.q.rows(16 * mt + m, 32 * ks + 8 * g, qa);
                if constexpr (DELTA) sm.r.k.rows(16 * mt + m, 32 * ks + 8 * g, ka);
#pragma unroll
                for (int t = 0; t < NT; ++t)
                    if (t <= mt && t % RW == half) {
                        b16x8 kb[NIN];
                        sm.r.k.rows(16 * t + m, 32 * ks + 8 * g, kb);
                        qk[t] = mma(kb, qa, qk[t]);
                        if constexpr (DELTA) kk[t] = mma(kb, ka, kk[t]);
                    }
            }
            const int i = 16 * mt + m;               // the lane's row; its columns j = 16 t + 4 g + r
            const float be = sm.g.be[i];
            float mz = 0.0f;
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                if (t > (mt | 1) || t % RW != half) continue;
                float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, pv[4], zv[4];
                if (t <= mt) decay_turned(sm.g, mt, t, lane, d);
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int j = 16 * t + 4 * g + r;
                    float zr = 0.0f;
                    if constexpr (DELTA) {
                        zr = i > j ? z[t][r] : 0.0f;
                        mz = fmaf(kk[t][r] * d[r], zr, mz);
                        zr *= -be;
                        zv[r] = zr * d[r];
                    }
                    pv[r] = dp[t][r] * d[r];
                    if (i >= j) sm.r.a[i][j + 1] = fmaf(dp[t][r], qk[t][r], zr * kk[t][r]);
                }
                sm.r.p.put4(mt >> 1, t >> 1, 16 * (mt & 1) + m, 16 * (t & 1) + 4 * g, pv);
                if constexpr (DELTA) sm.r.z.put4(mt >> 1, t >> 1, 16 * (mt & 1) + m, 16 * (t & 1) + 4 * g, zv);
            }
            if constexpr (DELTA) {
                mz += __shfl_xor(mz, 16);
                mz += __shfl_xor(mz, 32);
                if (g == 0) sm.mz[half][i] = mz;
            }
        }
        __syncthreads();
        if (tid < C) {
            float x = 0.0f, y = 0.0f, e = 0.0f, hvs = 0.0f, mzs = 0.0f;
#pragma unroll
            for (int i = 0; i < NW; ++i) {
                x += sm.part[0][i][tid];
                y += sm.part[1][i][tid];
                e += sm.part[2][i][tid];
            }
#pragma unroll
            for (int i = 0; i < RW; ++i) {
                hvs += sm.hv[i][tid];
                if constexpr (DELTA) mzs += sm.mz[i][tid];
            }
            sm.r.a[tid][0] = DELTA ? x - sm.g.be[tid] * y : x;
            sm.r.a[C][tid + 1] = e;
            if (tid == 0) {
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NW; ++i) s += sm.ss[i];
                sm.r.a[C][0] = s;
            }
            if (tid < nT)
                a.dbeta[tok + (int64_t)tid * a.H] =
                    tid < n ? (DELTA ? hvs - sm.g.gam[tid] * y - mzs : hvs) : 0.0f;
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
                sm.r.k.template cols<4>(32 * sb, 16 * (wv + NW * s), lane, kv[s]);
                sm.r.q.template cols<4>(32 * sb, 16 * (wv + NW * s), lane, qv[s]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                b16x8 x[3], y[3];
                if (t >= 2 * sb) {                   // rows t read tokens of block sb
                    sm.r.p.rows(t >> 1, sb, 16 * (t & 1) + m, g, x);
                    if constexpr (DELTA) sm.r.z.rows(t >> 1, sb, 16 * (t & 1) + m, g, y);
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        sdo[t][s] = mma(kv[s], x, sdo[t][s]);
                        if constexpr (DELTA) dsu[t][s] = mma(kv[s], y, dsu[t][s]);
                    }
                }
                if (t < 2 * sb + 2) {                // tokens t are read by rows of block sb
                    sm.r.p.template cols<4>(sb, t >> 1, 16 * (t & 1), lane, x);
                    if constexpr (DELTA) sm.r.z.template cols<4>(sb, t >> 1, 16 * (t & 1), lane, y);
#pragma unroll
                    for (int s = 0; s < ST; ++s) {
                        dsu[t][s] = mma(qv[s], x, dsu[t][s]);
                        if constexpr (DELTA) dsu[t][s] = mma(kv[s], y, dsu[t][s]);
                    }
                }
            }
        }
        if constexpr (GROUP) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    if constexpr (ACC) {
                        f32x4 *at = &sm.acc[((wv * NT + t) * ST + s) * 128 + lane];
                        if (gi) {
                            sdo[t][s] += at[0];
                            dsu[t][s] += at[64];
                        }
                        at[0] = sdo[t][s];
                        at[64] = dsu[t][s];
                    } else {
                        sdo[t][s] = dqa[t][s] += sdo[t][s];
                        dsu[t][s] = dka[t][s] += dsu[t][s];
                    }
                }
        }
        if (!GROUP || gi + 1 == G) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    const int row = 16 * t + m, key = 16 * (wv + NW * s) + 4 * g;
                    if (row < nT && key < a.dk) {
                        const int64_t at = (int64_t)row * a.Hk * a.dk + key;
                        put4(dqp + at, sdo[t][s], a.vec_g);
                        put4(dkp + at, dsu[t][s], a.vec_g);
                    }
                }
        }
    }
}

template <typename IN, int DKP>
hipError_t go(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const dim3 grid = chunk_grid(a, w);
    constexpr int TH = 64 * grad_waves<IN, DKP>();
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
