// X and P of every chunk (lores_scan, lores_scan_backward): what a chunk's
// tokens do to one another, which depends on q, k, alpha and beta alone and
// so is computed for all chunks at once.
//
// A work-group takes one chunk of one sequence and key head, a wavefront 16
// rows of it.  q k^T and k k^T are formed once for all value heads that share
// them.  X = (I + N)^-1 with N = diag(beta) M strictly lower: the 16 x 16
// diagonal blocks by forward substitution (a lane per column), the blocks
// below by X_IJ = -X_II sum_K N_IK X_KJ on the fp32 matrix instructions, one
// wavefront per block column J.  Substitution follows the recurrence itself,
// so X stays as bounded as the tokens' transition products are.
#include "lores_scan_impl.h"

namespace lores {
namespace scan {
namespace {

template <typename IN>
__global__ void __launch_bounds__(Cfg<IN>::C * 4) lores_scan_prep_kernel(const ScanArgs a, const ScanWork w) {
    constexpr int C = Cfg<IN>::C, NIN = Cfg<IN>::NIN, NT = C / 16, NB = tri_blocks(C);
    __shared__ Gates<C> gt;
    __shared__ __attribute__((aligned(16))) float nm[C][C + 4];      // N, rows of 16-byte multiples
    __shared__ __attribute__((aligned(16))) float xd[NT][16][20];    // inverses of the diagonal blocks
    const int lane = threadIdx.x & 63, mt = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int m = lane & 15, g = lane >> 4;
    const int chunk = blockIdx.x % w.chunks;
    const int bk = blockIdx.x / w.chunks, b = bk / a.Hk, hk = bk - b * a.Hk, G = a.H / a.Hk;
    int len = a.T;
    if (a.lengths) len = min(max(a.lengths[b], 0), a.T);
    const int t0 = chunk * C, n = min(len - t0, C);
    if (n <= 0) return;
    const IN *kp = (const IN *)a.k + b * a.ks[0] + t0 * a.ks[1] + hk * a.ks[2];
    const IN *qp = (const IN *)a.q + b * a.qs[0] + t0 * a.qs[1] + hk * a.qs[2];
    f32x4 qk[NT], kk[NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) qk[nt] = kk[nt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for (int ks = 0; ks < a.dk; ks += 32) {
        const int row = 16 * mt + m, c = ks + 8 * g;
        b16x8 qa[NIN], ka[NIN];
        get_planes(qp + row * a.qs[1] + c, row < n ? 8 : 0, a.vec, qa);
        get_planes(kp + row * a.ks[1] + c, row < n ? 8 : 0, a.vec, ka);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
            if (nt <= mt) {
                const int col = 16 * nt + m;
                b16x8 kb[NIN];
                get_planes(kp + col * a.ks[1] + c, col < n ? 8 : 0, a.vec, kb);
                qk[nt] = mma<3>(qa, kb, qk[nt]);
                if (a.delta) kk[nt] = mma<3>(ka, kb, kk[nt]);
            }
    }
    for (int gi = 0; gi < G; ++gi) {
        const int h = hk * G + gi;
        const int64_t gate = ((int64_t)b * a.T + t0) * a.H + h;
        const int64_t unit = ((int64_t)b * a.H + h) * w.chunks + chunk;
        if (gi) __syncthreads();                     // the last head's arrays have been read
        if (mt == 0) gt.load(a.alpha + gate, a.beta + gate, a.H, n, lane);
        __syncthreads();
        w.G[unit * 4 * C + threadIdx.x] = (&gt.al[0])[threadIdx.x];
        uint16_t *Pp = w.P + unit * w.p_planes * NB * 1024;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (nt > (mt | 1)) continue;             // blocks of 32 tokens above the diagonal are not read
            float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (nt <= mt) decay_tile(gt, mt, nt, lane, d);
            const int col = 16 * nt + m;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int row = 16 * mt + 4 * g + r;
                float x = qk[nt][r] * d[r];
                for (int pl = 0; pl < w.p_planes; ++pl) {
                    const uint16_t bits = f2bf(x);
                    Pp[((pl * NB + tri_block(mt >> 1, nt >> 1)) * 32 + (row & 31)) * 32 + (col & 31)] = bits;
                    x -= bf2f(bits);
                }
                if (a.delta) nm[row][col] = row > col ? gt.be[row] * (kk[nt][r] * d[r]) : 0.0f;
            }
        }
        if (!a.delta) continue;
        __syncthreads();
        // the wavefront's diagonal block, column m by the lanes of every group
        {
            float x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float s = i == m ? 1.0f : 0.0f;
#pragma unroll
                for (int l = 0; l < i; ++l) s = fmaf(-nm[16 * mt + i][16 * mt + l], x[l], s);
                x[i] = s;
            }
            if (g == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) xd[mt][i][m] = x[i];
            }
        }
        __syncthreads();
        uint16_t *Xp = w.X + unit * 3 * NB * 1024;
        f32x4 x[NT];                                 // block column J = mt, rows 4 g + r of block I
#pragma unroll
        for (int I = 0; I < NT; ++I) {
            if (I < mt) {
                x[I] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                continue;
            }
            if (I == mt) {
#pragma unroll
                for (int r = 0; r < 4; ++r) x[I][r] = xd[mt][4 * g + r][m];
                continue;
            }
            f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int K = 0; K < I; ++K)
                if (K >= mt) {
                    const f32x4 nr = *(const f32x4 *)&nm[16 * I + m][16 * K + 4 * g];
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        s = __builtin_amdgcn_mfma_f32_16x16x4f32(nr[r], x[K][r], s, 0, 0, 0);
                }
            const f32x4 xr = *(const f32x4 *)&xd[I][m][4 * g];
            f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int r = 0; r < 4; ++r)
                y = __builtin_amdgcn_mfma_f32_16x16x4f32(xr[r], s[r], y, 0, 0, 0);
            x[I] = -y;
        }
#pragma unroll
        for (int I = 0; I < NT; ++I) {
            if (mt > (I | 1)) continue;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                float v = x[I][r];
#pragma unroll
                for (int pl = 0; pl < 3; ++pl) {
                    const uint16_t bits = f2bf(v);
                    Xp[((pl * NB + tri_block(I >> 1, mt >> 1)) * 32 + 16 * (I & 1) + 4 * g + r) * 32 + 16 * (mt & 1) + m] = bits;
                    v -= bf2f(bits);
                }
            }
        }
    }
}

}  // namespace
}  // namespace scan

uint64_t plan_scan_work(bool in_bf16, bool backward, const ScanArgs &a, void *base, ScanWork *w) {
    const uint64_t C = scan_chunk(in_bf16);
    w->chunks = (int32_t)((a.T + C - 1) / C);
    w->p_planes = backward || !in_bf16 ? 3 : 2;
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
    w->P = (uint16_t *)cut(units * w->p_planes * tri);
    w->G = (float *)cut(units * 4 * C * 4);
    w->S = w->dS = w->U = w->Hm = nullptr;
    if (backward) {
        w->S = (uint16_t *)cut(units * 3 * a.dk * w->dvp * 2);
        w->dS = (uint16_t *)cut(units * 3 * a.dk * w->dvp * 2);
        w->U = (uint16_t *)cut(units * 3 * C * w->dvp * 2);
        w->Hm = (uint16_t *)cut(units * 3 * C * w->dvp * 2);
    }
    return off;
}

hipError_t launch_scan_prep(bool in_bf16, const ScanArgs &a, const ScanWork &w, hipStream_t s) {
    const dim3 grid((unsigned)((int64_t)a.B * a.Hk * w.chunks));
    if (in_bf16) scan::lores_scan_prep_kernel<uint16_t><<<grid, 256, 0, s>>>(a, w);
    else scan::lores_scan_prep_kernel<float><<<grid, 128, 0, s>>>(a, w);
    return hipGetLastError();
}

}  // namespace lores
