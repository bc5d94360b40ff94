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
// that share it, so dq and dk are summed in registers in head order.  A
// wavefront owns 16 tokens' rows of dP and Z, and its share of 16-key strips
// of the products with S and dS: their fragments come straight from memory
// (each is read by one wavefront only), dO, U and H are staged in LDS in
// blocks of 64 value columns.
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

constexpr int VB = 64;                               // value columns of a block

template <typename IN, int DKP>
struct GradLds {
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN;
    Planes<NIN, C, DKP> k, q;
    Planes<NIN, C, VB> d;                            // dO
    union {
        struct { Planes<3, C, VB> u, h; } v;
        struct { Planes<3, C, C> p, z; } m;          // dP.D and -beta Z.D
    };
    float a[C + 1][C + 3];                           // A, row C and column 0 its borders
    float part[3][4][C];                             // per wavefront: q.S^T dO, k.S^T h, k.dS^T u
    float hv[C], mz[C], ss[4];
    Gates<C> g;
};

__device__ __forceinline__ float sum16(float x) {
    x += __shfl_xor(x, 1);
    x += __shfl_xor(x, 2);
    x += __shfl_xor(x, 4);
    return x + __shfl_xor(x, 8);
}

template <typename IN, int DKP, bool DELTA>
__global__ void __launch_bounds__(Cfg<IN>::C * 4) lores_scan_grad_kernel(const ScanArgs a, const ScanWork w) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NT = C / 16, SB = C / 32, TH = C * 4;
    constexpr int ST = DKP / 16 / NT;                // 16-key strips of a wavefront
    constexpr int NO = sizeof(IN) == 2 ? 2 : 3;      // planes of what ends in the inputs' type
    __shared__ __attribute__((aligned(16))) GradLds<IN, DKP> sm;
    const int tid = threadIdx.x, lane = tid & 63, mt = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int chunk = blockIdx.x % w.chunks;
    const int bk = blockIdx.x / w.chunks, b = bk / a.Hk, hk = bk - b * a.Hk, G = a.H / a.Hk;
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
    stage_rows(sm.k, (const IN *)a.k + b * a.ks[0] + t0 * a.ks[1] + hk * a.ks[2], a.ks[1], n, a.dk, a.vec, tid, TH);
    stage_rows(sm.q, (const IN *)a.q + b * a.qs[0] + t0 * a.qs[1] + hk * a.qs[2], a.qs[1], n, a.dk, a.vec, tid, TH);
    __syncthreads();
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 qk[NT], kk[NT];                            // the wavefront's rows of q k^T and k k^T
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) qk[nt] = kk[nt] = zero;
#pragma unroll
    for (int ks = 0; ks < DKP / 32; ++ks) {
        b16x8 qa[NIN], ka[NIN];
        sm.q.rows(16 * mt + m, 32 * ks + 8 * g, qa);
        sm.k.rows(16 * mt + m, 32 * ks + 8 * g, ka);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            if (nt <= mt) {
                b16x8 kb[NIN];
                sm.k.rows(16 * nt + m, 32 * ks + 8 * g, kb);
                qk[nt] = mma<3>(qa, kb, qk[nt]);
                if constexpr (DELTA) kk[nt] = mma<3>(ka, kb, kk[nt]);
            }
    }
    f32x4 dq[NT][ST], dk[NT][ST];                    // token rows 16 t + 4 g + r, key strips mt + NT s
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < ST; ++s) dq[t][s] = dk[t][s] = zero;
    for (int gi = 0; gi < G; ++gi) {
        const int h = hk * G + gi;
        const int64_t cu = ((int64_t)b * a.H + h) * w.chunks + chunk;
        const int64_t tok = ((int64_t)b * a.T + t0) * a.H + h;   // of the chunk's first token
        __syncthreads();                             // the last head's arrays have been read
        if (mt == 0) sm.g.load(a.alpha + tok, a.beta + tok, a.H, n, lane);
        if (tid < C) sm.hv[tid] = 0.0f;
        f32x4 dp[NT], z[NT], sdo[NT][ST], sh[NT][ST], dsu[NT][ST];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            dp[t] = z[t] = zero;
#pragma unroll
            for (int s = 0; s < ST; ++s) sdo[t][s] = sh[t][s] = dsu[t][s] = zero;
        }
        float ss = 0.0f;                             // <S, dS>
        for (int v0 = 0; v0 < a.dv; v0 += VB) {
            __syncthreads();                         // the last block has been read; gates are there
            for (int x = tid; x < C * (VB / 8); x += TH) {
                const int row = x / (VB / 8), c = (x % (VB / 8)) * 8, left = a.dv - v0 - c;
                const int64_t in = (tok + (int64_t)row * a.H) * a.dv + v0 + c;
                b16x8 p[NIN];
                get_planes((const IN *)a.dout + in, row < n ? left : 0, false, p);
                sm.d.put8(row, c, p);
                float u8[8], h8[8];
                const int64_t at = (cu * C + row) * w.dvp + v0 + c;
                // dvp is a multiple of 16: whole groups of 8 (columns from dv on hold zeros)
                get8(w.U + at, w.dvp - v0 - c, true, u8);
                get8(w.Hm + at, w.dvp - v0 - c, true, h8);
                b16x8 u3[3], h3[3];
                split8(u8, u3);
                sm.v.u.put8(row, c, u3);
                if constexpr (DELTA) {
                    split8(h8, h3);
                    sm.v.h.put8(row, c, h3);
                }
                float s = 0.0f;
                if (row < n) {
                    const IN *vp = (const IN *)a.v + b * a.vs[0] + (t0 + row) * a.vs[1] + h * a.vs[2] + v0 + c;
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < left) s = fmaf(h8[e], get1(vp + e), s);
                }
                if (row < nT) {
                    IN *op = (IN *)a.dvalue + in;
                    const float be = sm.g.be[row];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        if (e < left) put1(op + e, be * h8[e]);
                }
                // 8 neighbouring threads hold the row's 64 columns
                s += __shfl_xor(s, 1);
                s += __shfl_xor(s, 2);
                s += __shfl_xor(s, 4);
                if ((x & 7) == 0) sm.hv[row] += s;
            }
            __syncthreads();
#pragma unroll
            for (int ks = 0; ks < VB / 32; ++ks) {
                const int c = 32 * ks + 8 * g;
                b16x8 da[NIN], ha[3];
                sm.d.rows(16 * mt + m, c, da);
                if constexpr (DELTA) sm.v.h.rows(16 * mt + m, c, ha);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt <= mt) {
                        b16x8 ub[3];
                        sm.v.u.rows(16 * nt + m, c, ub);
                        dp[nt] = mma<3>(da, ub, dp[nt]);
                        if constexpr (DELTA) z[nt] = mma<3>(ha, ub, z[nt]);
                    }
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    const int key = 16 * (mt + NT * s) + m, left = key < a.dk ? w.dvp - v0 - c : 0;
                    const int64_t at = (cu * a.dk + key) * w.dvp + v0 + c;
                    float s8[8], e8[8];
                    get8(w.S + at, left, true, s8);
                    get8(w.dS + at, left, true, e8);
#pragma unroll
                    for (int e = 0; e < 8; ++e) ss = fmaf(s8[e], e8[e], ss);
                    b16x8 sb[3], eb[3];
                    split8(s8, sb);
                    split8(e8, eb);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        b16x8 x1[NIN], x3[3];
                        sm.d.rows(16 * t + m, c, x1);
                        sdo[t][s] = mma<3>(x1, sb, sdo[t][s]);
                        if constexpr (DELTA) {
                            sm.v.h.rows(16 * t + m, c, x3);
                            sh[t][s] = mma<3>(x3, sb, sh[t][s]);
                        }
                        sm.v.u.rows(16 * t + m, c, x3);
                        dsu[t][s] = mma<3>(x3, eb, dsu[t][s]);
                    }
                }
            }
        }
        __syncthreads();                             // u and h have been read: their place is p's and z's
        // dots with the rows of q and k, over the wavefront's strips
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * t + 4 * g + r;
                float x = 0.0f, y = 0.0f, e = 0.0f;
#pragma unroll
                for (int s = 0; s < ST; ++s) {
                    const int key = 16 * (mt + NT * s) + m;
                    const float kv = sm.k.at(row, key);
                    x = fmaf(sm.q.at(row, key), sdo[t][s][r], x);
                    if constexpr (DELTA) y = fmaf(kv, sh[t][s][r], y);
                    e = fmaf(kv, dsu[t][s][r], e);
                    // their shares of dq and dk
                    dq[t][s][r] = fmaf(sm.g.gam[row], sdo[t][s][r], dq[t][s][r]);
                    dk[t][s][r] = fmaf(sm.g.end[row], dsu[t][s][r], dk[t][s][r]);
                    if constexpr (DELTA)
                        dk[t][s][r] = fmaf(-sm.g.be[row] * sm.g.gam[row], sh[t][s][r], dk[t][s][r]);
                }
                x = sum16(x);
                if constexpr (DELTA) y = sum16(y);
                e = sum16(e);
                if (m == 0) {
                    sm.part[0][mt][row] = x;
                    sm.part[1][mt][row] = y;
                    sm.part[2][mt][row] = e;
                }
            }
        ss = sum16(ss);
        ss += __shfl_xor(ss, 16);
        ss += __shfl_xor(ss, 32);
        if (lane == 0) sm.ss[mt] = ss;
        // A without its borders, dP.D and -beta Z.D
        {
            float mz[4] = {0.0f, 0.0f, 0.0f, 0.0f};
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
                        zr *= -sm.g.be[row];
                        sm.m.z.put(row, colj, zr * d[r]);
                    }
                    sm.m.p.put(row, colj, dp[nt][r] * d[r]);
                    if (row >= colj) sm.a[row][colj + 1] = fmaf(dp[nt][r], qk[nt][r], zr * kk[nt][r]);
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
            for (int i = 0; i < NT; ++i) {
                x += sm.part[0][i][tid];
                y += sm.part[1][i][tid];
                e += sm.part[2][i][tid];
            }
            sm.a[tid][0] = DELTA ? x - sm.g.be[tid] * y : x;
            sm.a[C][tid + 1] = e;
            if (tid == 0) {
                float s = 0.0f;
                for (int i = 0; i < NT; ++i) s += sm.ss[i];
                sm.a[C][0] = s;
            }
            if (tid < nT)
                a.dbeta[tok + (int64_t)tid * a.H] =
                    tid < n ? (DELTA ? sm.hv[tid] - sm.g.gam[tid] * y - sm.mz[tid] : sm.hv[tid]) : 0.0f;
        }
        __syncthreads();
        // along j: what row i has read of everything before token t, decayed to
        // t - 1; column t of A holds token t - 1
        for (int i = tid; i <= C; i += TH) {
            float u = 0.0f;
            const int last = i < C ? i : C - 1;
            for (int t = 0; t <= last; ++t) {
                const float x = sm.a[i][t];
                u = t ? fmaf(sm.g.al[t - 1], u, x) : x;
                sm.a[i][t] = u;
            }
        }
        __syncthreads();
        // along i: those rows decayed back from i to t
        if (tid < nT) {
            float s = 0.0f, d = 1.0f;
            for (int i = tid; i < C; ++i) {
                if (i > tid) d *= sm.g.al[i];
                s = fmaf(d, sm.a[i][tid], s);
            }
            s = fmaf(d, sm.a[C][tid], s);
            a.dalpha[tok + (int64_t)tid * a.H] = tid < n ? s : 0.0f;
        }
        // dq += (dP.D) k;  dk += (dP.D)^T q + (-beta Z.D) k + (-beta Z.D)^T k
#pragma unroll
        for (int s = 0; s < ST; ++s) {
            const int c0 = 16 * (mt + NT * s);
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) {
                b16x8 kv[NIN], qv[NIN];
                sm.k.template cols<4>(32 * sb, c0, lane, kv);
                sm.q.template cols<4>(32 * sb, c0, lane, qv);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    b16x8 x[NO];
                    if (t >= 2 * sb) {               // rows t read tokens of block sb
                        sm.m.p.rows(16 * t + m, 32 * sb + 8 * g, x);
                        dq[t][s] = mma<NO>(x, kv, dq[t][s]);
                        if constexpr (DELTA) {
                            sm.m.z.rows(16 * t + m, 32 * sb + 8 * g, x);
                            dk[t][s] = mma<NO>(x, kv, dk[t][s]);
                        }
                    }
                    if (t < 2 * sb + 2) {            // tokens t are read by rows of block sb
                        sm.m.p.template cols<4>(32 * sb, 16 * t, lane, x);
                        dk[t][s] = mma<NO>(x, qv, dk[t][s]);
                        if constexpr (DELTA) {
                            sm.m.z.template cols<4>(32 * sb, 16 * t, lane, x);
                            dk[t][s] = mma<NO>(x, kv, dk[t][s]);
                        }
                    }
                }
            }
        }
    }
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int s = 0; s < ST; ++s)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * t + 4 * g + r, key = 16 * (mt + NT * s) + m;
                if (row < nT && key < a.dk) {
                    put1(dqp + (int64_t)row * a.Hk * a.dk + key, dq[t][s][r]);
                    put1(dkp + (int64_t)row * a.Hk * a.dk + key, dk[t][s][r]);
                }
            }
}

template <typename IN, int DKP>
hipError_t go(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.B * a.Hk * w.chunks));
    if (a.delta) lores_scan_grad_kernel<IN, DKP, true><<<grid, Cfg<IN>::C * 4, 0, s>>>(a, w);
    else lores_scan_grad_kernel<IN, DKP, false><<<grid, Cfg<IN>::C * 4, 0, s>>>(a, w);
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
