// Projection on 4-bit weights (lores_mx_matmul): out[m][j] = sum_k a[m][k] w[j][k].
//
// The scaled matrix instruction 16 x 16 x 128 takes a lane's 32 neighbours of a
// row as they lie in memory, with the block's scale in a register: lane l
// holds block l / 16 of row l % 16.  Weights are its first operand, so a lane
// ends with 4 neighbouring outputs of one row.  E4M3 rows lie otherwise: lane l
// holds 16 neighbours from 16 (l / 16) and 16 from 64 + 16 (l / 16); their one
// factor per row is multiplied in at the end.
#include <type_traits>

#include "lores_direct.h"
#include "lores_layer.h"

namespace lores {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint16_t to_bf16(float f) {
    const __bf16 b = (__bf16)f;
    return __builtin_bit_cast(uint16_t, b);
}

template <bool FP8>
__device__ __forceinline__ f32x4 product(const i32x8 &w, const i32x8 &a, f32x4 c, int ws, int as) {
    // format 4: E2M1, 0: E4M3
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, a, c, 4, FP8 ? 0 : 4, 0, ws, 0, as);
}

template <bool BF16>
__device__ __forceinline__ void put4(const MxProduct &p, int64_t at, f32x4 c) {
    if constexpr (BF16) *(u16x4 *)((uint16_t *)p.out + at) = u16x4{to_bf16(c[0]), to_bf16(c[1]), to_bf16(c[2]), to_bf16(c[3])};
    else *(f32x4 *)((float *)p.out + at) = c;
}

// 4 outputs of row m from column j on, as far as there are any
template <bool FP8, bool BF16>
__device__ __forceinline__ void put(const MxProduct &p, int64_t m, int j, f32x4 c) {
    if (m >= p.M) return;
    if constexpr (FP8) c *= p.a_rows[m];
    const int64_t at = m * p.N + j;
    if ((p.N & 3) == 0 && j + 3 < p.N) {
        put4<BF16>(p, at, c);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (j + i < p.N) {
            if constexpr (BF16) ((uint16_t *)p.out)[at + i] = to_bf16(c[i]);
            else ((float *)p.out)[at + i] = c[i];
        }
}

// Few rows: a work-group has 16 columns and 16 MT rows, its wavefronts share k.
template <bool FP8, bool BF16, int MT, int W>
__global__ void __launch_bounds__(64 * W) lores_mx_few_kernel(const MxProduct p) {
    __shared__ f32x4 sm[W][MT][64];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int tiles = (p.N + 15) / 16;
    const int64_t b = block_at(blockIdx.x, blockIdx.y), mb = b / tiles;
    const int j0 = (int)(b - mb * tiles) * 16;
    const int64_t m0 = mb * (16 * MT);
    if (m0 >= p.M) return;
    const int blocks = p.K / 32, per = mx_scale_stride(p.K), steps = (p.K + 127) / 128;
    const int64_t wr = min(j0 + r, p.N - 1);
    const uint8_t *wc = p.w + wr * (p.K / 2), *wsc = p.w_scales + wr * per;
    int64_t ar[MT];
#pragma unroll
    for (int i = 0; i < MT; ++i) ar[i] = min(m0 + 16 * i + r, p.M - 1);
    f32x4 c[MT] = {};
    for (int k = wv; k < steps; k += W) {
        const int blk = 4 * k + g;
        const bool in = blk < blocks;
        i32x8 w = {};
        int ws = 0;
        if (in) {
            const i32x4 x = *(const i32x4 *)(wc + blk * 16);
            w = i32x8{x[0], x[1], x[2], x[3], 0, 0, 0, 0};
            ws = wsc[blk];
        }
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            i32x8 a = {};
            int as = 127;
            if constexpr (FP8) {
                const uint8_t *q = p.a + ar[i] * p.K;
                const int at = k * 128 + 16 * g;
                i32x4 x = {}, y = {};
                if (at < p.K) x = *(const i32x4 *)(q + at);
                if (at + 64 < p.K) y = *(const i32x4 *)(q + at + 64);
                a = i32x8{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
            } else if (in) {
                const i32x4 x = *(const i32x4 *)(p.a + ar[i] * (p.K / 2) + blk * 16);
                a = i32x8{x[0], x[1], x[2], x[3], 0, 0, 0, 0};
                as = p.a_scales[ar[i] * per + blk];
            }
            c[i] = product<FP8>(w, a, c[i], ws, as);
        }
    }
#pragma unroll
    for (int i = 0; i < MT; ++i) sm[wv][i][lane] = c[i];
    __syncthreads();
    for (int i = wv; i < MT; i += W) {               // the wavefronts' sums in their order
        f32x4 s = sm[0][i][lane];
#pragma unroll
        for (int v = 1; v < W; ++v) s += sm[v][i][lane];
        put<FP8, BF16>(p, m0 + 16 * i + r, j0 + 4 * g, s);
    }
}

template <bool FP8, bool BF16, int MT>
hipError_t go_few(const MxProduct &p, hipStream_t s) {
    const int64_t groups = (p.M + 16 * MT - 1) / (16 * MT) * ((p.N + 15) / 16);
    lores_mx_few_kernel<FP8, BF16, MT, 8><<<grid_of(groups), 512, 0, s>>>(p);
    return hipGetLastError();
}

// ------------------------------------------------------------ many rows
//
// A work-group has WM x WN wavefronts, each with 16 MI rows and 16 NI columns in
// registers.  Steps of 128 k go from memory straight to LDS, S steps deep; a
// wavefront reads the next step's operands while it multiplies this one's.
// A 4-bit row of a step is 64 bytes: pieces of 16 bytes, whose places are turned by
// the row so that 8 neighbouring rows read their like pieces from different banks;
// an E4M3 row is 128 bytes of 8 pieces, turned alike.
template <bool FP8, int TM, int TN>
struct Stage {
    uint8_t w[TN * 64], a[TM * (FP8 ? 128 : 64)];
};
// The scales of 4 steps, 16 bytes a row: the columns', the rows' behind them.  (4 bytes
// a step and row would be as many requests to the cache as the codes are.)
template <bool FP8, int TM, int TN>
struct Scales {
    uint8_t s[TN * 16 + (FP8 ? 0 : TM * 16)];
};

// A wavefront's operands of a step: its rows, and a part of its columns at a time.
template <bool FP8, int MI>
struct Rows {
    i32x4 x[MI][FP8 ? 2 : 1];
    int s[MI];
};
template <int NH>
struct Columns {
    i32x4 x[NH];
    int s[NH];
};

// The work-group's tile: each of the 8 XCDs (work-groups go to them in turn) takes a
// run of tiles, and a run goes over 8 rows of tiles before the next column.
__device__ __forceinline__ void tile_of(int64_t b, int64_t tiles_m, int64_t tiles_n, int64_t &m, int64_t &n) {
    const int64_t all = tiles_m * tiles_n, each = all / 8, more = all % 8, x = b % 8;
    const int64_t t = x * each + (x < more ? x : more) + b / 8;
    const int64_t band = t / (8 * tiles_n), first = band * 8;
    const int64_t high = tiles_m - first < 8 ? tiles_m - first : 8, in = t - band * 8 * tiles_n;
    m = first + in % high;
    n = in / high;
}

template <bool FP8, bool BF16, int MI, int NI, int WM, int WN, int S>
__global__ void __launch_bounds__(64 * WM * WN) lores_mx_tile_kernel(const MxProduct p) {
    constexpr int TM = 16 * MI * WM, TN = 16 * NI * WN, NW = WM * WN;
    constexpr int AB = FP8 ? 128 : 64, AR = 1024 / AB;          // bytes of a row, rows of a load
    constexpr int LW = TN / 16 / NW, LA = TM / AR / NW;         // a wavefront's loads of a step
    constexpr int PW = TN / 64, PA = FP8 ? 0 : TM / 64;         // scales: 64 rows a load
    constexpr int LS = (PW + PA + NW - 1) / NW;
    constexpr int L = LW + LA;
    static_assert(LW * NW * 16 == TN && LA * NW * AR == TM && TN % 64 == 0 && TM % 64 == 0, "loads");
    __shared__ __attribute__((aligned(1024))) Stage<FP8, TM, TN> st[S];
    __shared__ __attribute__((aligned(1024))) Scales<FP8, TM, TN> sc[2];
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
    const int wm = wv % WM, wn = wv / WM;
    int64_t tm, tn;
    tile_of(block_at(blockIdx.x, blockIdx.y), (p.M + TM - 1) / TM, (p.N + TN - 1) / TN, tm, tn);
    const int64_t m0 = tm * TM, n0 = tn * TN;
    if (m0 >= p.M || n0 >= p.N) return;
    const int steps = (p.K + 127) / 128, per = mx_scale_stride(p.K);
    const int64_t wrow = p.K / 2, arow = FP8 ? p.K : p.K / 2;
    const int last_m = (int)min(p.M - 1 - m0, (int64_t)TM - 1), last_n = (int)min(p.N - 1 - n0, (int64_t)TN - 1);
    const uint8_t *wb = p.w + n0 * wrow, *ab = p.a + m0 * arow;
    const uint8_t *wsb = p.w_scales + n0 * per, *asb = FP8 ? nullptr : p.a_scales + m0 * per;
    // a lane's piece of its row, the same in all its loads; rows behind the end are the last one
    const int wpiece = (lane & 3) ^ ((lane >> 3) & 3), apiece = FP8 ? (lane & 7) ^ ((lane >> 3) & 7) : wpiece;
    uint32_t wat[LW], aat[LA], sat[LS];
#pragma unroll
    for (int i = 0; i < LW; ++i)
        wat[i] = (uint32_t)min((wv + i * NW) * 16 + (lane >> 2), last_n) * (uint32_t)wrow + wpiece * 16;
#pragma unroll
    for (int i = 0; i < LA; ++i)
        aat[i] = (uint32_t)min((wv + i * NW) * AR + lane / (AB / 16), last_m) * (uint32_t)arow + apiece * 16;
    int spart[LS];
    const uint8_t *sbase[LS];
#pragma unroll
    for (int i = 0; i < LS; ++i) {                   // (a wavefront without a part of its own repeats another's)
        spart[i] = __builtin_amdgcn_readfirstlane((wv + i * NW) % (PW + PA));
        sat[i] = spart[i] < PW ? (uint32_t)min(spart[i] * 64 + lane, last_n) * (uint32_t)per
                               : (uint32_t)min((spart[i] - PW) * 64 + lane, last_m) * (uint32_t)per;
        sbase[i] = spart[i] < PW ? wsb : asb;
    }
    const int wv_ = __builtin_amdgcn_readfirstlane(wv);
    // (whole: no k of the step lies behind the rows' end; the others get zeros there)
    auto load = [&](int k, auto whole) {
        Stage<FP8, TM, TN> &s = st[k % S];
        const bool win = whole || 128 * k + 32 * wpiece < p.K;
        const bool ain = whole || (FP8 ? 128 * k + 16 * apiece < p.K : win);
        const i32x4 zero = {};
#pragma unroll
        for (int i = 0; i < LW; ++i) {
            uint8_t *to = s.w + (wv_ + i * NW) * 1024;
            if (win) direct16(wb + (int64_t)k * 64, wat[i], to);
            else *(i32x4 *)(to + lane * 16) = zero;
        }
#pragma unroll
        for (int i = 0; i < LA; ++i) {
            uint8_t *to = s.a + (wv_ + i * NW) * 1024;
            if (ain) direct16(ab + (int64_t)k * AB, aat[i], to);
            else *(i32x4 *)(to + lane * 16) = zero;
        }
    };
    // the scales of steps 4 b .. 4 b + 3; the last 16 bytes of a row where it ends before
    auto scales_from = [&](int b) { return min(16 * b, max(per - 16, 0)); };
    auto load_scales = [&](int b) {
        uint8_t *to = sc[b & 1].s;
        const int from = scales_from(b);
        if (per >= 16) {
#pragma unroll
            for (int i = 0; i < LS; ++i) direct16(sbase[i] + from, sat[i], to + spart[i] * 1024);
        } else {
#pragma unroll
            for (int i = 0; i < LS; ++i)
                for (int j = 0; j < per; j += 4)
                    *(uint32_t *)(to + spart[i] * 1024 + lane * 16 + j) = *(const uint32_t *)(sbase[i] + sat[i] + j);
        }
    };
    // places in a stage, but for constants: like pieces of rows 16 apart are turned alike
    const int wplace = (wn * NI * 16 + r) * 64 + (g ^ ((r >> 1) & 3)) * 16, wsplace = (wn * NI * 16 + r) * 16 + g;
    const int aplace = FP8 ? (wm * MI * 16 + r) * 128 + (g ^ (r & 7)) * 16 : (wm * MI * 16 + r) * 64 + (g ^ ((r >> 1) & 3)) * 16;
    const int aplace2 = (wm * MI * 16 + r) * 128 + ((4 + g) ^ (r & 7)) * 16, asplace = (TN + wm * MI * 16 + r) * 16 + g;
    // columns are taken in parts, E4M3 rows with their wider operands in smaller ones
    constexpr int PARTS = FP8 && NI == 8 ? 4 : 2, NH = NI / PARTS;
    auto scales_at = [&](int k) { return sc[(k >> 2) & 1].s + (4 * k - scales_from(k >> 2)); };
    auto read_rows = [&](int k, Rows<FP8, MI> &o) {
        const Stage<FP8, TM, TN> &s = st[k % S];
        const uint8_t *q = scales_at(k);
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            o.x[i][0] = *(const i32x4 *)(s.a + aplace + i * 16 * AB);
            if constexpr (FP8) o.x[i][1] = *(const i32x4 *)(s.a + aplace2 + i * 16 * AB);
            o.s[i] = FP8 ? 127 : q[asplace + i * 256];
        }
    };
    auto read_columns = [&](int k, int part, Columns<NH> &o) {
        const Stage<FP8, TM, TN> &s = st[k % S];
        const uint8_t *q = scales_at(k);
#pragma unroll
        for (int i = 0; i < NH; ++i) {
            o.x[i] = *(const i32x4 *)(s.w + wplace + (part * NH + i) * 1024);
            o.s[i] = q[wsplace + (part * NH + i) * 256];
        }
    };
    f32x4 c[MI][NI] = {};
    auto multiply = [&](const Rows<FP8, MI> &a, const Columns<NH> &w, int part) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            i32x8 x = {a.x[i][0][0], a.x[i][0][1], a.x[i][0][2], a.x[i][0][3], 0, 0, 0, 0};
            if constexpr (FP8)
                x = i32x8{a.x[i][0][0], a.x[i][0][1], a.x[i][0][2], a.x[i][0][3],
                          a.x[i][1][0], a.x[i][1][1], a.x[i][1][2], a.x[i][1][3]};
#pragma unroll
            for (int j = 0; j < NH; ++j) {
                const i32x8 y = {w.x[j][0], w.x[j][1], w.x[j][2], w.x[j][3], 0, 0, 0, 0};
                c[i][part * NH + j] = product<FP8>(y, x, c[i][part * NH + j], w.s[j], a.s[i]);
            }
        }
    };
    const int ahead = min(S, steps), wholes = p.K / 128;
    load_scales(0);
    for (int k = 0; k < ahead; ++k) load(k, false);
    if (steps >= S) arrived_but<L * (S - 1)>();
    else arrived();
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    Rows<FP8, MI> a[2];
    Columns<NH> w[2];
    read_rows(0, a[0]);
    read_columns(0, 0, w[0]);
    // one step: a part's products run while the next part's operands are read.  Before
    // the last part this wavefront's reads of step k are done and its loads of step
    // k + 1 have landed; behind the barrier that holds for all wavefronts, so step k's
    // place takes step k + S.  Every fourth step (Q = k % 4 = 0) loads the next four's
    // scales first, into the place of those that step k - 1 has read; the loads that
    // may still be on their way are those of steps k + 2 .. k + S - 1, and scales that
    // were asked for among them.
    auto fence = [] { __builtin_amdgcn_sched_barrier(0); };
    auto step = [&](int k, auto Q, const Rows<FP8, MI> &now, Rows<FP8, MI> &next) {
#pragma unroll
        for (int q = 0; q < PARTS - 1; ++q) {
            read_columns(k, q + 1, w[(q + 1) & 1]);
            fence();
            multiply(now, w[q & 1], q);
            fence();
        }
        constexpr bool among = Q() >= 1 && Q() <= S - 2;
        arrived_but<L * (S - 2) + (among ? LS : 0)>();
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (Q() == 0) load_scales((k >> 2) + 1);
        load(k + S, std::true_type());
        read_rows(k + 1, next);
        read_columns(k + 1, 0, w[0]);
        fence();
        multiply(now, w[1], PARTS - 1);
        fence();
    };
    // the steps at the end, where loads run out
    auto last = [&](int k, const Rows<FP8, MI> &now, Rows<FP8, MI> &next) {
#pragma unroll
        for (int q = 0; q < PARTS - 1; ++q) {
            read_columns(k, q + 1, w[(q + 1) & 1]);
            multiply(now, w[q & 1], q);
        }
        if (k + 1 < steps) {
            if (S >= 4 && k + 4 <= steps) arrived_but<2 * L>();
            else if (k + 3 <= steps) arrived_but<L>();
            else arrived();
            asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
            if (k % 4 == 0 && k + 4 < steps) load_scales((k >> 2) + 1);
            if (k + S < steps) load(k + S, false);
            read_rows(k + 1, next);
            read_columns(k + 1, 0, w[0]);
        }
        multiply(now, w[1], PARTS - 1);
    };
    static_assert(S == 3 || S == 4, "the waits");
    int k = 0;
    for (; k + 3 + S < wholes; k += 4) {
        step(k, std::integral_constant<int, 0>(), a[0], a[1]);
        step(k + 1, std::integral_constant<int, 1>(), a[1], a[0]);
        step(k + 2, std::integral_constant<int, 2>(), a[0], a[1]);
        step(k + 3, std::integral_constant<int, 3>(), a[1], a[0]);
    }
    for (; k < steps; k += 2) {
        last(k, a[0], a[1]);
        if (k + 1 < steps) last(k + 1, a[1], a[0]);
    }
    const int64_t m = m0 + wm * MI * 16 + r;
    const int n = (int)n0 + wn * NI * 16 + 4 * g;
    if (last_m == TM - 1 && last_n == TN - 1 && (p.N & 3) == 0) {
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            const float f = FP8 ? p.a_rows[m + 16 * i] : 1.0f;
#pragma unroll
            for (int j = 0; j < NI; ++j) put4<BF16>(p, (m + 16 * i) * p.N + n + 16 * j, FP8 ? c[i][j] * f : c[i][j]);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < NI; ++j) put<FP8, BF16>(p, m + 16 * i, n + 16 * j, c[i][j]);
}

template <bool FP8, bool BF16, int MI, int NI, int WM, int WN, int S>
hipError_t go_tile(const MxProduct &p, hipStream_t s) {
    constexpr int TM = 16 * MI * WM, TN = 16 * NI * WN;
    const int64_t groups = (p.M + TM - 1) / TM * ((p.N + TN - 1) / TN);
    lores_mx_tile_kernel<FP8, BF16, MI, NI, WM, WN, S><<<grid_of(groups), 64 * WM * WN, 0, s>>>(p);
    return hipGetLastError();
}

template <bool FP8, bool BF16>
hipError_t go(const MxProduct &p, hipStream_t s) {
    if (p.M <= 16) return go_few<FP8, BF16, 1>(p, s);
    if (p.M <= 64) return go_few<FP8, BF16, 4>(p, s);
    if (p.M * p.N >= (int64_t)256 * 256 * 128) return go_tile<FP8, BF16, 4, 8, 4, 2, FP8 ? 3 : 4>(p, s);
    return go_tile<FP8, BF16, 4, 4, 2, 2, 3>(p, s);
}

}  // namespace

hipError_t launch_mx_product(bool a_fp8, bool out_bf16, const MxProduct &p, hipStream_t s) {
    if (a_fp8) return go<true, true>(p, s);
    return out_bf16 ? go<false, true>(p, s) : go<false, false>(p, s);
}

}  // namespace lores
