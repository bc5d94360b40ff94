// X and P of every chunk (lores_scan, lores_scan_backward): what a chunk's
// tokens do to one another, which depends on q, k, alpha and beta alone and
// so is computed for all chunks at once.
//
// A work-group takes one chunk of one sequence and key head, a wavefront 16
// rows of it.  q k^T and k k^T are formed once for all value heads that share
// them.  All tiles are made turned over (operands exchanged), so that a lane
// holds four neighbours of one row: planes then go to LDS 8 bytes at a time
// and to memory 16 (2-byte stores of the tiles as they come out took three
// quarters of this kernel's time).  X = (I + N)^-1 with N = diag(beta) M
// strictly lower: the 16 x 16 diagonal blocks by forward substitution (a lane
// per column), the blocks left of them by X_IJ = -(sum_{K>J} X_IK N_KJ) X_JJ
// on the fp32 matrix instructions, a wavefront per block row.  Substitution
// follows the recurrence itself, so X stays as bounded as the tokens'
// transition products are.
//
// Measured (bf16, d_k = 128, delta): 256 units x 4096 tokens 220 us, 1.07 GB at
// 4.9 TB/s, close to a copy: bound by reading q and k and by writing X and P.
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

// P as the passes behind read it: in fp32 or as planes
template <int C, bool WORDS> struct PrepP : TriWords<C> {};
template <int C> struct PrepP<C, false> : Tri<3, C> {};

template <typename IN, int DKP, bool WORDS>
struct PrepLds {
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NT = C / 16;
    Gates<C> g;
    union {
        struct { Planes<NIN, C, DKP> k, q; } r;      // until the tiles of q k^T and k k^T are made
        struct {
            float nt[NT * (NT - 1) / 2 + 1][16][20]; // N_KJ turned over (rows j), tile K (K - 1) / 2 + J
            float nd[NT][16][20];                    // N_II, then X_II
            Tri<3, C> x;
            PrepP<C, WORDS> p;
        } t;
    };
};

// WORDS: P in fp32 instead of planes.  Two work-groups share a compute unit; asking for registers
// for three is the same within 1 % (8 x 4096 tokens x 32 heads with the pass
// behind: 721 and 724 us).
template <typename IN, int DKP, bool WORDS, bool DELTA>
__global__ void __launch_bounds__(Cfg<IN>::C * 4, (sizeof(IN) == 2 && DKP <= 128 ? 2 : 1)) lores_scan_prep_kernel(const ScanArgs a, const ScanWork w) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NT = C / 16, NB = tri_blocks(C), NW = NT, TH = 64 * NW;
    __shared__ __attribute__((aligned(16))) PrepLds<IN, DKP, WORDS> sm;
    const int tid = threadIdx.x, lane = tid & 63, mt = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    int b, hk, chunk;
    if (!chunk_of((int)block_at(blockIdx.x, blockIdx.y), a, w, &b, &hk, &chunk)) return;
    const int G = a.H / a.Hk;
    int len = a.T;
    if (a.lengths) len = min(max(a.lengths[b], 0), a.T);
    const int t0 = chunk * C, n = min(len - t0, C);
    if (n <= 0) return;
    const IN *kp = (const IN *)a.k + b * a.ks[0] + t0 * a.ks[1] + hk * a.ks[2];
    const IN *qp = (const IN *)a.q + b * a.qs[0] + t0 * a.qs[1] + hk * a.qs[2];
    const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
    f32x4 qk[NT], kk[NT];                            // rows j = 16 nt + 4 g + r of column i = 16 mt + m
#pragma unroll
    for (int t = 0; t < NT; ++t) qk[t] = kk[t] = zero;
    // the first head's gates are on their way with the rows
    const int l = lane & (C - 1);
    const int64_t gate0 = ((int64_t)b * a.T + t0) * a.H + hk * G + (int64_t)min(l, n - 1) * a.H;
    float al = a.alpha[gate0], bt = a.beta[gate0];
    if constexpr (NIN == 1) {
        if (a.vec) {
            direct_rows<C, DKP, NW>(sm.r.k.x[0], (const uint16_t *)kp, a.ks[1], n, a.dk, mt, lane);
            direct_rows<C, DKP, NW>(sm.r.q.x[0], (const uint16_t *)qp, a.qs[1], n, a.dk, mt, lane);
        }
    }
    if (NIN == 3 || !a.vec) {
        stage_rows(sm.r.k, kp, a.ks[1], n, a.dk, a.vec, tid, TH);
        stage_rows(sm.r.q, qp, a.qs[1], n, a.dk, a.vec, tid, TH);
    }
    arrived();
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < DKP / 32; ++ks) {
        b16x8 qv[NIN], ko[NIN], kv[NT][NIN];
        sm.r.q.rows(16 * mt + m, 32 * ks + 8 * g, qv);
        if constexpr (DELTA) sm.r.k.rows(16 * mt + m, 32 * ks + 8 * g, ko);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t <= mt) sm.r.k.rows(16 * t + m, 32 * ks + 8 * g, kv[t]);
#pragma unroll
        for (int t = 0; t < NT; ++t)
            if (t <= mt) {
                qk[t] = mma(kv[t], qv, qk[t]);
                if constexpr (DELTA) kk[t] = mma(kv[t], ko, kk[t]);
            }
    }
    for (int gi = 0; gi < G; ++gi) {
        const int h = hk * G + gi;
        const int64_t unit = ((int64_t)b * a.H + h) * w.chunks + chunk;
        __syncthreads();                             // the rows, or the last head's arrays, have been read
#pragma unroll
        for (int q = 0; q < 4; q += NW) make_gates(sm.g, q + mt, l < n ? al : 1.0f, l < n ? bt : 0.0f, lane);
        if (gi + 1 < G) {
            al = a.alpha[gate0 + gi + 1];
            bt = a.beta[gate0 + gi + 1];
        }
        __syncthreads();
        const float be = sm.g.be[16 * mt + m];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t > (mt | 1)) continue;              // blocks of 32 tokens above the diagonal are not read
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f}, v[4];
            if (t <= mt) decay_turned(sm.g, mt, t, lane, d);
#pragma unroll
            for (int r = 0; r < 4; ++r) v[r] = qk[t][r] * d[r];
            sm.t.p.put4(mt >> 1, t >> 1, 16 * (mt & 1) + m, 16 * (t & 1) + 4 * g, v);
            if constexpr (DELTA) {
                if (t > mt) continue;
#pragma unroll
                for (int r = 0; r < 4; ++r) v[r] = t < mt || 4 * g + r < m ? be * (kk[t][r] * d[r]) : 0.0f;
                if (t < mt) {
#pragma unroll
                    for (int r = 0; r < 4; ++r) sm.t.nt[mt * (mt - 1) / 2 + t][4 * g + r][m] = v[r];
                } else {
                    *(f32x4 *)&sm.t.nd[mt][m][4 * g] = f32x4{v[0], v[1], v[2], v[3]};
                }
            }
        }
        if constexpr (DELTA) {
            // the wavefront's diagonal block, written and read by it alone:
            // column m by the lanes of every group
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == m ? 1.0f : 0.0f;
#pragma unroll
                for (int l = 0; l < i; l += 4) {
                    const f32x4 nr = *(const f32x4 *)&sm.t.nd[mt][i][l];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (l + e < i) s = fmaf(-nr[e], x[l + e], s);
                }
                x[i] = s;
            }
            if (g == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) sm.t.nd[mt][i][m] = x[i];
            }
        }
        __syncthreads();
        // what is done goes to memory while X is made
        for (int i = tid; i < 6 * C / 4; i += TH) ((f32x4 *)(w.G + unit * 6 * C))[i] = ((const f32x4 *)&sm.g.al[0])[i];
        for (int i = tid; i < (int)sizeof(sm.t.p) / 16; i += TH)
            ((u32x4 *)((uint8_t *)w.P + unit * sizeof(sm.t.p)))[i] = ((const u32x4 *)&sm.t.p.x[0])[i];
        if constexpr (!DELTA) continue;
        f32x4 xt[NT];                                // X_IJ of block row I = mt: rows j, column i
#pragma unroll
        for (int J = NT - 1; J >= 0; --J) {
            xt[J] = zero;
            if (J > mt) continue;
            if (J == mt) {
                xt[J] = *(const f32x4 *)&sm.t.nd[mt][m][4 * g];
            } else {
                f32x4 s = zero;
#pragma unroll
                for (int K = 0; K < NT; ++K)
                    if (K > J && K <= mt) {
                        const f32x4 nr = *(const f32x4 *)&sm.t.nt[K * (K - 1) / 2 + J][m][4 * g];
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            s = __builtin_amdgcn_mfma_f32_16x16x4f32(nr[r], xt[K][r], s, 0, 0, 0);
                    }
                f32x4 y = zero;
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    y = __builtin_amdgcn_mfma_f32_16x16x4f32(sm.t.nd[J][4 * g + r][m], s[r], y, 0, 0, 0);
                xt[J] = -y;
            }
        }
#pragma unroll
        for (int J = 0; J < NT; ++J) {
            if (J > (mt | 1)) continue;
            const float v[4] = {xt[J][0], xt[J][1], xt[J][2], xt[J][3]};
            sm.t.x.put4(mt >> 1, J >> 1, 16 * (mt & 1) + m, 16 * (J & 1) + 4 * g, v);
        }
        __syncthreads();
        for (int i = tid; i < 3 * NB * 128; i += TH)
            ((u32x4 *)(w.X + unit * 3 * NB * 1024))[i] = ((const u32x4 *)&sm.t.x.x[0])[i];
    }
}

template <typename IN, int DKP, bool WORDS>
hipError_t go(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const dim3 grid = chunk_grid(a, w);
    if (a.delta) lores_scan_prep_kernel<IN, DKP, WORDS, true><<<grid, Cfg<IN>::C * 4, 0, s>>>(a, w);
    else lores_scan_prep_kernel<IN, DKP, WORDS, false><<<grid, Cfg<IN>::C * 4, 0, s>>>(a, w);
    return hipGetLastError();
}

template <typename IN, bool WORDS>
hipError_t by_width(const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (a.dk <= 64) return go<IN, 64, WORDS>(a, w, s);
    if (a.dk <= 128) return go<IN, 128, WORDS>(a, w, s);
    return go<IN, 256, WORDS>(a, w, s);
}

}  // namespace
}  // namespace scan

uint64_t plan_scan_work(bool in_bf16, bool backward, const ScanArgs &a, void *base, ScanWork *w) {
    const uint64_t C = scan_chunk(in_bf16);
    w->chunks = (int32_t)((a.T + C - 1) / C);
    w->p_words = !backward && in_bf16;
    w->dvp = (a.dv + 15) / 16 * 16;
    const uint64_t units = (uint64_t)a.B * a.H * w->chunks;
    uint64_t off = 0;
    auto cut = [&](uint64_t bytes) {
        uint8_t *p = base ? (uint8_t *)base + off : nullptr;
        off += (bytes + 255) / 256 * 256;
        return p;
    };
    const uint64_t tri = scan::tri_blocks((int)C) * 2048;       // bytes of a plane
    w->X = (uint16_t *)(a.delta ? cut(units * 3 * tri) : nullptr);
    w->P = (uint16_t *)cut(units * (w->p_words ? 2 : 3) * tri);
    w->G = (float *)cut(units * 6 * C * 4);
    w->S = w->dS = w->U = w->Hm = nullptr;
    if (backward) {
        w->S = (float *)cut(units * a.dk * w->dvp * 4);
        w->dS = (float *)cut(units * a.dk * w->dvp * 4);
        w->U = (float *)cut(units * C * w->dvp * 4);
        w->Hm = (float *)cut(units * C * w->dvp * 4);
    }
    return off;
}

hipError_t launch_scan_prep(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (!in_bf16) return scan::by_width<float, false>(a, w, s);
    return w.p_words ? scan::by_width<uint16_t, true>(a, w, s) : scan::by_width<uint16_t, false>(a, w, s);
}

}  // namespace lores
