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
//
// Measured (bf16, d_k = d_v = 128, delta): 256 units x 4096 tokens 494 us, 1.6
// GB at 3.3 TB/s with the matrix instructions busy for 46 % of the time, two
// wavefronts per SIMD taking turns between them and the splitting into planes.
// 32 units x 4096 tokens 321 us, 5.0 us for each of 64 chunks: one wavefront
// on a quarter of the SIMDs, bound by the chain of a chunk's five products.
// Storing S and U for the backward pass, 128 units x 2048 tokens take 149 us
// (0.62 GB, 4.1 TB/s).
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

// P: planes of fp32 inputs, fp32 of bf16 ones
template <typename IN, bool BACK> struct StateP : TriWords<Cfg<IN>::C> {};
template <> struct StateP<float, false> : Tri<3, Cfg<float>::C> {};
template <typename IN> struct alignas(16) StateP<IN, true> {};   // is not read

template <typename IN, int DKP, bool BACK, int NW>
struct StateLds {
    static constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN;
    Planes<NIN, C, DKP> k;
    Planes<NIN, BACK ? 1 : C, DKP> q;
    Tri<3, C> x;
    StateP<IN, BACK> p;
    Gates<C> g;
    Tile<IN, C> v[NW];
};

// Two chunks' rows where they fit: the next chunk's arrive while one is
// worked on.
template <typename L> __host__ __device__ constexpr int stages() { return 2 * sizeof(L) <= 160 * 1024 ? 2 : 1; }

// BACK: store every chunk's first state and U instead of outputs.  FAST: q and
// k rows that can be read 16 bytes at a time (a.vec); VEC: v and o rows (a.vec_v).
// Others take the same steps with narrower loads.  NW: wavefronts of a
// work-group.
template <typename IN, int DKP, bool DELTA, bool BACK, bool FAST, bool VEC, int NW>
__global__ void __launch_bounds__(64 * NW) lores_scan_state_kernel(const ScanArgs a, const ScanWork w, const int groups) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, MT = C / 16, SB = C / 32, KS = DKP / 32, TH = 64 * NW;
    constexpr bool IN16 = sizeof(IN) == 2;
    typedef StateLds<IN, DKP, BACK, NW> Lds;
    constexpr int NS = stages<Lds>();
    __shared__ __attribute__((aligned(16))) Lds lds[NS];
    const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int m = lane & 15, g = lane >> 4;
    int unit, grp;
    if (!unit_of((int)block_at(blockIdx.x, blockIdx.y), groups, a.B * a.H, &unit, &grp)) return;
    const int b = unit / a.H, h = unit - b * a.H, hk = h / (a.H / a.Hk);
    const int col0 = (grp * NW + wv) * 16, col = col0 + m;   // the wavefront's value rows of S, the lane's
    const bool mine = col0 < a.dv, ok = col < a.dv;
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
    const IN *vb = (const IN *)a.v + b * a.vs[0] + h * a.vs[2] + (mine ? col0 : 0);
    const int64_t os = (int64_t)a.H * a.dv;
    IN *ob = (IN *)a.o + ((int64_t)b * a.T * a.H + h) * a.dv + col0;
    const int chunks = (len + C - 1) / C;
    RowFetch<C, IN16 ? 8 : DKP, TH> kf, qf;          // fp32 only
    IN vf[VEC ? 1 : MT][4];
    // A chunk's rows to stage `to`, in parts that the compute steps below are
    // interleaved with: part 0 k, 1 q, 2 what the tokens do to one another,
    // 3 the values.
    auto fetch = [&](int part, int ch, Lds &to) {
        const int t0 = ch * C, n = min(len - t0, C);
        const int64_t cu = (int64_t)unit * w.chunks + ch;
        if (part == 0) {
            if constexpr (FAST && IN16) direct_rows<C, DKP, NW>(to.k.x[0], kb + t0 * a.ks[1], a.ks[1], n, a.dk, wv, lane);
            else if constexpr (FAST) kf.load(kb + t0 * a.ks[1], a.ks[1], n, a.dk, tid);
        } else if (part == 1) {
            if constexpr (!BACK && FAST && IN16) direct_rows<C, DKP, NW>(to.q.x[0], qb + t0 * a.qs[1], a.qs[1], n, a.dk, wv, lane);
            else if constexpr (!BACK && FAST) qf.load(qb + t0 * a.qs[1], a.qs[1], n, a.dk, tid);
        } else if (part == 2) {
            if constexpr (!BACK) direct_block<sizeof(to.p), NW>((const uint8_t *)w.P + cu * (int64_t)sizeof(to.p), &to.p, wv, lane);
            if constexpr (DELTA) direct_block<sizeof(to.x), NW>(w.X + cu * (3 * Tri<1, C>::NB * 1024), &to.x, wv, lane);
            direct_block<sizeof(to.g), NW>(w.G + cu * (6 * C), &to.g, wv, lane);
        } else if (mine) {
            if constexpr (VEC) {
                to.v[wv].fetch(vb + t0 * a.vs[1], a.vs[1], n, a.dv - col0, lane);
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        vf[mt][r] = vb[(t0 + token_of(mt, r) + min(8 * g, n - 1 - token_of(mt, r))) * a.vs[1] + (ok ? m : 0)];
            }
        }
    };
    // fp32 rows, and rows at odd addresses, through registers
    auto place = [&](int ch, Lds &to) {
        const int t0 = ch * C, n = min(len - t0, C);
        if constexpr (!FAST) {
            stage_rows(to.k, kb + t0 * a.ks[1], a.ks[1], n, a.dk, false, tid, TH);
            if constexpr (!BACK) stage_rows(to.q, qb + t0 * a.qs[1], a.qs[1], n, a.dk, false, tid, TH);
        } else if constexpr (!IN16) {
            kf.store(to.k, n, a.dk, tid);
            if constexpr (!BACK) qf.store(to.q, n, a.dk, tid);
        }
    };
    if (chunks) {
#pragma unroll
        for (int i = 0; i < 4; ++i) fetch(i, 0, lds[0]);
        place(0, lds[0]);
        arrived();
    }
    for (int ch = 0; ch < chunks; ++ch) {
        const int t0 = ch * C, n = min(len - t0, C);
        const int64_t cu = (int64_t)unit * w.chunks + ch;
        Lds &sm = lds[NS == 2 ? ch & 1 : 0];
        Lds &next = lds[NS == 2 ? (ch & 1) ^ 1 : 0];
        const bool more = NS == 2 && ch + 1 < chunks;
        f32x4 u[MT];                                 // V, then beta E, then U: tokens token_of(mt, 4 g + r)
        if constexpr (!VEC) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) u[mt][r] = get1(&vf[mt][r]);
        }
        __syncthreads();                             // this chunk is there, the other stage has been read
        if (!mine) {                                 // a wavefront without value rows only helps to fetch
            if (more) {
#pragma unroll
                for (int i = 0; i < 4; ++i) fetch(i, ch + 1, next);
            }
        } else {
        if constexpr (VEC) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float x[4];
                sm.v[wv].get(mt, lane, x);
#pragma unroll
                for (int r = 0; r < 4; ++r) u[mt][r] = x[r];
            }
        }
        if (more) fetch(0, ch + 1, next);
        f32x4 o[MT], e[MT], gm[MT], be[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) e[mt] = o[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        b16x8 sp[KS][3], rv[2][MT][NIN], xv[MT][3];
        auto split = [&](int ks) {
            float x[8];
            pair8(st[2 * ks], st[2 * ks + 1], x);
            split8(x, sp[ks]);
        };
        auto gates = [&]() {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                gm[mt] = *(const f32x4 *)&sm.g.gam[token_of(mt, 4 * g)];
                be[mt] = *(const f32x4 *)&sm.g.be[token_of(mt, 4 * g)];
            }
        };
        auto x_first = [&]() {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) sm.x.rows(mt >> 1, 0, token_of(mt, m) & 31, g, xv[mt]);
        };
        // K S^T; S is split one block of 32 keys ahead
        if constexpr (DELTA) {
            auto rows = [&](int ks) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sm.k.rows(token_of(mt, m), 32 * ks + 8 * g, rv[ks & 1][mt]);
            };
            rows(0);
            split(0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                fence();
                if (ks + 1 < KS) rows(ks + 1);
                else gates();
                fence();
                if (ks + 1 < KS) split(ks + 1);
                mma_all<MT>(rv[ks & 1], sp[ks], e);
                mix<(NIN == 1 ? 3 : 6) * MT, 4>();
            }
            fence();
        } else {
            gates();
        }
        if (more) fetch(1, ch + 1, next);
        if constexpr (BACK) {
            float *sp0 = w.S + cu * w.dvp * a.dk;
            const uint32_t at = (uint32_t)col * (uint32_t)a.dk + 8 * g;
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t)
                if (32 * (t >> 1) < a.dk) store4(sp0 + (at + 32 * (t >> 1) + 4 * (t & 1)), st[t]);
        }
        // Q S^T, and beside it E and its planes
        b16x8 ep[SB][3];
        // nothing behind the sequence's end or d_v counts, whatever stands there
        if (n < C || col0 + 16 > a.dv) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r) u[mt][r] = ok && 8 * g < n - token_of(mt, r) ? u[mt][r] : 0.0f;
        }
        auto finish_e = [&](int sb) {
#pragma unroll
            for (int mt = 2 * sb; mt < 2 * sb + 2; ++mt)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    u[mt][r] = be[mt][r] * (DELTA ? fmaf(-gm[mt][r], e[mt][r], u[mt][r]) : u[mt][r]);
            if constexpr (DELTA) {
                float x[8];
                pair8(u[2 * sb], u[2 * sb + 1], x);
                split8(x, ep[sb]);
            }
        };
        if constexpr (!BACK) {
            auto rows = [&](int ks) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sm.q.rows(token_of(mt, m), 32 * ks + 8 * g, rv[ks & 1][mt]);
            };
            rows(0);
            if constexpr (!DELTA) split(0);
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                fence();
                if (ks + 1 < KS) rows(ks + 1);
                else if constexpr (DELTA) x_first();
                fence();
                if constexpr (!DELTA) {
                    if (ks + 1 < KS) split(ks + 1);
                }
                if (ks < SB) finish_e(ks);
                mma_all<MT>(rv[ks & 1], sp[ks], o);
                mix<(NIN == 1 ? 3 : 6) * MT, 4>();
            }
            fence();
        } else {
            if constexpr (DELTA) x_first();
            fence();
#pragma unroll
            for (int sb = 0; sb < SB; ++sb) finish_e(sb);
        }
        if (more) fetch(2, ch + 1, next);
        // the last products' left operands come while U is made
        b16x8 kt[2 * KS][NIN], pv[BACK ? 1 : MT][3], ut[SB][3], up[SB][3];
        f32x4 pw[IN16 && !BACK ? MT : 1][2];         // P before it becomes planes
        f32x4 en[MT];
        auto turned = [&](int sb) {
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t)
                sm.k.template cols<8>(32 * sb, 32 * (t >> 1) + 4 * (t & 1), lane, kt[t]);
            if constexpr (!BACK) {
#pragma unroll
                for (int mt = 2 * sb; mt < MT; ++mt) {
                    if constexpr (IN16) sm.p.rows(mt >> 1, sb, token_of(mt, m) & 31, g, pw[mt]);
                    else sm.p.rows(mt >> 1, sb, token_of(mt, m) & 31, g, pv[mt]);
                }
            }
        };
        auto split_p = [&](int mt0) {
            if constexpr (IN16 && !BACK) {
#pragma unroll
                for (int mt = mt0; mt < MT; ++mt) {
                    float x[8];
                    pair8(pw[mt][0], pw[mt][1], x);
                    split8(x, pv[mt]);
                }
            }
        };
        // U = X beta E, one block of 32 tokens after the other
        if constexpr (DELTA) {
            b16x8 xn[MT][3];
            if constexpr (SB > 1) {
#pragma unroll
                for (int mt = 2; mt < MT; ++mt) sm.x.rows(mt >> 1, 1, token_of(mt, m) & 31, g, xn[mt]);
            }
            fence();
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) e[mt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            mma_all<MT>(xv, ep[0], e);
            if constexpr (!BACK) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) o[mt] *= gm[mt];
            }
            fence();
            turned(0);
            fence();
            if constexpr (SB > 1) mma_all<MT - 2>(xn + 2, ep[SB - 1], e + 2);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) u[mt] = e[mt];
        } else {
            turned(0);
            if constexpr (!BACK) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) o[mt] *= gm[mt];
            }
        }
        // S_C = gamma_C S + K^T (D_C U), and O += P U beside it
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) en[mt] = *(const f32x4 *)&sm.g.end[token_of(mt, 4 * g)];
        const float ge = sm.g.gam[C - 1];
        auto split_u = [&](int sb) {
            float x[8];
            pair8(u[2 * sb], u[2 * sb + 1], x);
            if constexpr (!BACK) split8(x, up[sb]);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] *= i < 4 ? en[2 * sb][i] : en[2 * sb + 1][i - 4];
            split8(x, ut[sb]);
        };
#pragma unroll
        for (int t = 0; t < 2 * KS; ++t) st[t] *= ge;
        split_u(0);
        fence();
        if (more) fetch(3, ch + 1, next);
        if constexpr (SB > 1) split_u(SB - 1);
        split_p(0);
        mma_all<2 * KS>(kt, ut[0], st);
        if constexpr (!BACK) mma_all<MT>(pv, up[0], o);
        mix<(NIN == 1 ? 3 : 6) * 2 * KS + (BACK ? 0 : 6 * MT), 3>();
        fence();
        if constexpr (SB > 1) {
            turned(1);
            fence();
            split_p(2);
            mma_all<2 * KS>(kt, ut[SB - 1], st);
            if constexpr (!BACK) mma_all<MT - 2>(pv + 2, up[SB - 1], o + 2);
            mix<3 * 2 * KS + (BACK ? 0 : 6 * (MT - 2)), 2>();
        }
        if constexpr (BACK) {
            float *u0 = w.U + cu * w.dvp * C;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) store4(u0 + (uint32_t)(col * C + token_of(mt, 4 * g)), u[mt]);
        } else {
            const int nT = min(a.T - t0, C);
            IN *oc = ob + t0 * os;
            if constexpr (VEC) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sm.v[wv].put(mt, lane, o[mt]);
                sm.v[wv].store(oc, os, nT, a.dv - col0, lane);
            } else {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (ok && 8 * g < nT - token_of(mt, r))
                            put1(oc + (token_of(mt, r) + 8 * g) * os + m, o[mt][r]);
            }
        }
        }
        if (ch + 1 < chunks) {
            if constexpr (NS == 1) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < 4; ++i) fetch(i, ch + 1, lds[0]);
            }
            place(ch + 1, next);
            arrived();
        }
    }
    if constexpr (!BACK) {
        // whole chunks behind the sequence's end
        if (ok)
            for (int t = chunks * C + g; t < a.T; t += 4) put1(ob + t * os + m, 0.0f);
        if (a.S && ok) {
#pragma unroll
            for (int t = 0; t < 2 * KS; ++t) {
                const int key = 32 * (t >> 1) + 8 * g + 4 * (t & 1);
                if (key < a.dk) store4(a.S + ((int64_t)unit * a.dv + col) * a.dk + key, st[t]);
            }
        }
    }
}

template <typename IN, int DKP, bool FAST, bool VEC, int NW>
hipError_t go(bool backward, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const int groups = (a.dv + 16 * NW - 1) / (16 * NW);
    const dim3 grid = grid_of(((int64_t)a.B * a.H + 7) / 8 * 8 * groups);
    if (backward) {
        if (a.delta) lores_scan_state_kernel<IN, DKP, true, true, FAST, VEC, NW><<<grid, 64 * NW, 0, s>>>(a, w, groups);
        else lores_scan_state_kernel<IN, DKP, false, true, FAST, VEC, NW><<<grid, 64 * NW, 0, s>>>(a, w, groups);
    } else {
        if (a.delta) lores_scan_state_kernel<IN, DKP, true, false, FAST, VEC, NW><<<grid, 64 * NW, 0, s>>>(a, w, groups);
        else lores_scan_state_kernel<IN, DKP, false, false, FAST, VEC, NW><<<grid, 64 * NW, 0, s>>>(a, w, groups);
    }
    return hipGetLastError();
}

template <typename IN, int DKP>
hipError_t by_rows(bool backward, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (!a.vec) return go<IN, DKP, false, false, 4>(backward, a, w, s);
    if (!a.vec_v) return go<IN, DKP, true, false, 4>(backward, a, w, s);
    if constexpr (DKP <= 128)
        if (scan_waves(a) == 8) return go<IN, DKP, true, true, 8>(backward, a, w, s);
    return go<IN, DKP, true, true, 4>(backward, a, w, s);
}

template <typename IN>
hipError_t by_width(bool backward, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    if (a.dk <= 64) return by_rows<IN, 64>(backward, a, w, s);
    if (a.dk <= 128) return by_rows<IN, 128>(backward, a, w, s);
    return by_rows<IN, 256>(backward, a, w, s);
}

}  // namespace
}  // namespace scan

hipError_t launch_scan_state(bool in_bf16, bool backward, const ScanArgs &a, const ScanWork &w,
                             hipStream_t s) {
    return in_bf16 ? scan::by_width<uint16_t>(backward, a, w, s) : scan::by_width<float>(backward, a, w, s);
}

}  // namespace lores
