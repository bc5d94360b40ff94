/*
 * lores.h - C ABI of the LoReS quantized recurrent-state decode step for
 * AMD Instinct MI355X (gfx950).
 *
 * The method: "Quantizing Recurrent Language Models Is Easier Than You Think"
 * (structured summary page).  Each (sequence, head) unit keeps a recurrent
 * state S in R^{d_v x d_k} that every decode step updates in place:
 *
 *   S_t = S_{t-1} diag(alpha_t) (I - delta beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *   o_t = S_t q_t
 *
 * (section "Introduction and Theoretical Foundation", general recurrence form)
 * while the state is stored quantized, dequantized, updated and requantized
 * every step (section "Intra-State Quantization Approach", property 3), with
 * one scale per value row (section "Intra-State Quantization (Section 4)",
 * scale grouping and Proposition 1), stochastic rounding (same section,
 * Rounding and Proposition 3) and a per-head precision chosen from the decay
 * rate (same section, decay-based mixed precision).
 *
 * Conventions for every entry point:
 *   - Return value: LORES_OK (0) or a negative LORES_E* code.  On error,
 *     lores_last_error() (thread-local) describes it.  No C++ exception
 *     crosses this boundary.  Validation happens before any GPU work, so a
 *     call that fails validation launches nothing.
 *   - "device" pointers point to HIP device memory owned by the caller; the
 *     library never allocates or frees device memory.  "host" pointers point
 *     to ordinary host memory, read or written synchronously.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Device work is enqueued asynchronously on it; inputs must stay alive
 *     and unmodified until that work has run.
 *   - Calls on one lores_state handle are not re-entrant across streams.
 *   - LORES_EHIP reports that a launch of this call failed.  Before each of
 *     its launches the library consumes any HIP error left on the calling
 *     thread by earlier work, so such an error is never reported as this
 *     call's (and is no longer visible to the caller afterwards).
 */
#ifndef LORES_H
#define LORES_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define LORES_SPEC_VERSION 8

/* Per-head state precision. */
enum {
    LORES_FP32 = 0, /* unquantized fp32 state (the full-precision reference path) */
    LORES_BF16 = 1, /* bfloat16 state, stochastic rounding from fp32               */
    LORES_INT8 = 2, /* int8 codes in [-127, 127] + one fp32 scale per value row     */
    LORES_INT4 = 3, /* int4 codes in [-7, 7]     + one fp32 scale per value row     */
    LORES_INT6 = 4, /* int6 codes in [-31, 31]   + one fp32 scale per value row     */
    LORES_FP8 = 5   /* E4M3 (OCP fp8) values     + one fp32 scale per value row     */
};
#define LORES_NUM_PREC 6
/* An output or operand of the layer operators, not a state: rows of E2M1 values
 * with one power of two per 32 neighbours (see lores_mx_quant). */
#define LORES_MXFP4 16

/* What a gate z is put through: z, z / (1 + e^-z), 1 / (1 + e^-z). */
enum { LORES_ACT_NONE = 0, LORES_ACT_SILU = 1, LORES_ACT_SIGMOID = 2 };

/* Rounding of the requantization (per state; lores_state_set_rounding). */
enum {
    LORES_ROUND_STOCHASTIC = 0, /* default: the counter-based draw n below              */
    LORES_ROUND_NEAREST = 1     /* the same quantizer with the draw fixed at n = 2^15 */
};

/* Scale grouping of the scaled classes (int8, int4, int6, fp8), fixed when
 * the state is allocated (lores_state_alloc_axis).  The pages compare one
 * scale per value row with one per key column ("Intra-State Quantization
 * (Section 4)", Scale Grouping and Proposition 1); value rows are their
 * choice and the default here. */
enum {
    LORES_SCALE_VALUE = 0, /* one fp32 scale per value row: s_i = max_j |S_ij| / r  */
    LORES_SCALE_KEY = 1    /* one fp32 scale per key column: s_j = max_i |S_ij| / r */
};

/* Status codes. */
enum {
    LORES_OK = 0,
    LORES_EINVAL = -1,      /* invalid argument (NULL, misaligned, out of range)  */
    LORES_EUNSUPPORTED = -2,/* valid but not built (kept for the ABI; no current case) */
    LORES_ESIZE = -3,       /* buffer too small                                     */
    LORES_EHIP = -4,        /* a HIP runtime call failed                           */
    LORES_ENOMEM = -5       /* host allocation failed                              */
};

/* Limits. */
#define LORES_MAX_HEADS 512 /* heads per state                                   */
#define LORES_MAX_DV 256    /* value rows per head                               */
#define LORES_ROW_BLOCK 64  /* value rows per stored row block (one wavefront)   */
#define LORES_MAX_WINDOW 16 /* steps per requantization window                   */

/* Opaque host handle: dimensions, per-head precision, layout and the bound
 * device buffer.  Created by lores_state_alloc, released by lores_state_free. */
typedef struct lores_state lores_state;

/*
 * Packed state layout (version LORES_SPEC_VERSION), for inspection, tests and
 * checkpointing.  The buffer holds one segment pair per precision class that
 * has at least one head, in class order fp32, bf16, int8, int4, int6, fp8,
 * each segment starting on a 256-byte boundary:
 *
 *   codes  [B][H_c][n_chunk][d_v_pad][16 bytes]
 *   scales [B][H_c][d_v_pad] fp32                 (int8, int4, int6, fp8 classes)
 *          [B][H_c][d_k] fp32                     (the same, key-column scales)
 *   window [B][H_c][unit_window_bytes]            (scaled classes of a windowed
 *                                                  state, window W > 1)
 *
 * H_c = heads of class c, ordered by head index (head_slot below).
 * d_v_pad = d_v rounded up to LORES_ROW_BLOCK; padding rows are never read
 * or written by a step.  A row is cut into 16-byte chunks of E elements
 * (E = 4 fp32, 8 bf16, 16 int8, 32 int4; n_chunk = d_k / E), stored
 * chunk-major so one wavefront's 64 rows of a chunk are 1 KiB contiguous.
 * Within a chunk, element e is:
 *   fp32: word e, IEEE binary32        bf16: halfword e, bfloat16 bits
 *   int8: byte e  = 128 + s code       (offset binary, 1..255)
 *   fp8:  byte e  = E4M3 byte (OCP: sign, 4 exponent bits with bias 7,
 *         3 mantissa bits; never the NaN pattern), value scale * E4M3 value
 *   int4: byte e/2, low nibble for even e, high nibble for odd e,
 *         nibble = 8 + s code          (offset binary, 1..15)
 * int6 rows are a little-endian bit stream over the row's chunks (chunk c
 * holds row bytes 16c .. 16c + 15): element j is bits 6j .. 6j + 5, value
 * 32 + s code (offset binary, 1..63); n_chunk = ceil(6 d_k / 128), the bits
 * after the last element are zero.
 * s = +1 in the even columns of a row and -1 in the odd ones: an int row
 * holds the codes of its odd columns negated (a column pair shares one
 * rounding draw, and the odd column is requantized as -U; see
 * lores_decode_step).
 * A row of d_k > 128 is stored as two half rows of d_k / 2 columns, each laid
 * out as above from its own first chunk (n_chunk = 2 n_chunk(d_k / 2): an
 * int4 or int6 half that ends inside a chunk is zero-padded to its end).
 * The value of an int element is scale[row] * code (scale[column] * code
 * with key-column scales).  A row of all-zero bytes with scale 0 also reads
 * as zero, so a zero-filled buffer is S = 0.
 * A unit's window block holds W - 1 token slots: g [W-1][d_v_pad] fp32 (the
 * write vector of the token), then k [W-1][d_k] fp32, then alpha [W-1][d_k]
 * fp32 (the token's decay per key channel; a scalar decay in element 0, the
 * others unused), the whole block padded to 16 bytes.  Slot tau - 1 holds
 * token tau of the current window (lores_state_alloc_window).
 */
typedef struct {
    int32_t B, H, d_k, d_v, d_v_pad;
    int32_t n_class[LORES_NUM_PREC];        /* heads per precision class        */
    int64_t codes_offset[LORES_NUM_PREC];   /* byte offset of class codes, -1   */
    int64_t scales_offset[LORES_NUM_PREC];  /* byte offset of class scales, -1  */
    int64_t unit_code_bytes[LORES_NUM_PREC];/* code bytes per (sequence, head)  */
    uint64_t total_bytes;      /* bytes the caller's buffer must hold           */
    int32_t scale_axis;        /* LORES_SCALE_VALUE or LORES_SCALE_KEY          */
    int32_t unit_scales;       /* fp32 scales per (sequence, head): d_v_pad or d_k */
    int32_t window;            /* W: steps per requantization (1: every step)   */
    int32_t window_fill;       /* tokens of the current window in the buffer    */
    int64_t window_offset[LORES_NUM_PREC];    /* byte offset of class windows, -1 */
    int64_t unit_window_bytes[LORES_NUM_PREC];/* window bytes per unit, 0       */
} lores_layout;

/*
 * lores_state_alloc - plan the packed layout and bind a caller-owned buffer.
 * The state of every (sequence, head) unit is S in R^{d_v x d_k} of the
 * general recurrence ("Introduction and Theoretical Foundation"), held in
 * the precision head_prec assigns to its head (decay-based mixed precision,
 * "Intra-State Quantization (Section 4)") with one scale per value row (the
 * same section, scale grouping), starting from S_0 = 0.
 *   B, H        sequences and heads (1 <= B <= 65535, 1 <= H <= LORES_MAX_HEADS)
 *   d_k, d_v    key and value dimensions; d_k a multiple of 32, at most 256
 *               (LORES_EINVAL otherwise), 1 <= d_v <= LORES_MAX_DV.
 *   head_prec   host [H] precision per head (LORES_FP32 .. LORES_FP8)
 *   d_buf       device buffer, 256-byte aligned, >= *bytes; or NULL
 *   bytes       host in/out.  d_buf == NULL: size query, writes the size and
 *               returns LORES_OK without creating a handle.  Otherwise *bytes
 *               is the buffer size (LORES_ESIZE if too small).
 *   stream      the buffer is cleared to S_0 = 0 asynchronously on it
 *   out         host out: the new handle (owned by the caller; free it with
 *               lores_state_free, which never touches device memory)
 */
int lores_state_alloc(int32_t B, int32_t H, int32_t d_k, int32_t d_v,
                      const uint8_t *head_prec, void *d_buf, size_t *bytes,
                      void *stream, lores_state **out);

/*
 * lores_state_alloc_axis - lores_state_alloc with a choice of scale grouping
 * for every scaled head (int8, int4, int6, fp8): LORES_SCALE_VALUE is
 * lores_state_alloc itself; LORES_SCALE_KEY keeps one scale per key column,
 * s_j = fl(m_j / r) with m_j the maximum of |S_ij| over the unit's d_v rows,
 * and the same codes, rounding and draws otherwise (the comparison grouping
 * of "Intra-State Quantization (Section 4)", Scale Grouping and Proposition
 * 1).  A step then dequantizes S'_ij = fl(c_ij * fl(s_j * alpha_j)).
 * LORES_SCALE_KEY is built for every d_k and d_v that lores_state_alloc
 * accepts.  A key-column state runs one launch per precision class (no
 * fused pairs).  LORES_EINVAL for any other scale_axis.
 */
int lores_state_alloc_axis(int32_t B, int32_t H, int32_t d_k, int32_t d_v,
                           const uint8_t *head_prec, int32_t scale_axis, void *d_buf,
                           size_t *bytes, void *stream, lores_state **out);

/*
 * lores_state_alloc_window - lores_state_alloc_axis for a state whose scaled
 * heads (int8, int4, int6, fp8) are requantized once per window of W steps
 * instead of every step, the window's tokens being kept at fp32
 * in a per-unit buffer (the reading of the PACE and LeapQuant abstracts:
 * rounding once every few tokens, with the tokens in between buffered, cuts
 * the error that accumulates in the state).  Windows are the steps
 * t = kW + 1 .. (k + 1) W.  Inside a window the stored state is the state at
 * the window start, X_0, and is not written; step t at position
 * p = (t - 1) mod W + 1 < W computes g, o from X_0 and the buffered tokens
 * and appends (g, k, alpha) to the buffer; the step at p = W rebuilds the
 * state by the fp32 recurrence (S'_1 = fl(c fl(s alpha_1)), then
 * U_tau = fma(g_tau, k_tau, S'_tau), S'_tau = fl(U_{tau-1} alpha_tau), with a
 * decay per key channel taken column by column), steps it and requantizes
 * it as lores_decode_step does.  W = 1 is
 * lores_state_alloc_axis.  fp32 and bf16 heads step every token as usual.
 * With key-column scales (PACE shares scales within a column), s_i above is
 * the column's s_j and the window's end takes the column maxima.
 *   scale_axis  LORES_SCALE_VALUE or LORES_SCALE_KEY (as lores_state_alloc_axis)
 *   window      W, 1 <= W <= LORES_MAX_WINDOW
 * Built for every d_k and d_v that lores_state_alloc_axis accepts.
 * Steps on a windowed state must come in order (t = 1, 2, ... from the
 * allocation or a lores_quant_state; the handle counts the buffered tokens
 * and lores_decode_step returns LORES_EINVAL for a step t whose window
 * position does not follow them).  The decay may be a scalar per head or
 * one value per key channel (alpha_per_channel), the same kind for every
 * token of a window: a step inside a window whose kind differs from the
 * buffered tokens' returns LORES_EINVAL.  Each scaled class runs one launch
 * per step.
 * The count is kept on the host: a captured graph of steps on a windowed
 * state replays correctly when it covers whole windows.
 */
int lores_state_alloc_window(int32_t B, int32_t H, int32_t d_k, int32_t d_v,
                             const uint8_t *head_prec, int32_t scale_axis, int32_t window,
                             void *d_buf, size_t *bytes, void *stream, lores_state **out);

void lores_state_free(lores_state *st);

/* Copy the layout of `st` into host struct *out. */
int lores_state_layout(const lores_state *st, lores_layout *out);

/*
 * lores_state_set_rounding - rounding of every later requantization of `st`
 * (host only; takes effect for calls enqueued afterwards).
 *   LORES_ROUND_STOCHASTIC  stochastic rounding (the default), as described
 *                           at lores_decode_step
 *   LORES_ROUND_NEAREST     the same formula with u = 1/2 (n = 2^15): codes
 *                           s (floor(fl(s U * inv + bias + 1/2)) - bias), i.e.
 *                           round to nearest, ties upward in even and downward
 *                           in odd columns, after the fp32 rounding of the
 *                           sum; bf16 heads keep the high half of
 *                           f32bits(U) + 2^15 (nearest, ties away from zero)
 * Round-to-nearest is the deterministic baseline the stochastic rounding is
 * compared with ("Intra-State Quantization (Section 4)", Rounding and
 * Proposition 3).  LORES_EINVAL for any other mode.
 */
int lores_state_set_rounding(lores_state *st, int32_t mode);

/* Host arrays [H]: precision and slot (index among heads of that class). */
int lores_state_head_map(const lores_state *st, uint8_t *prec_out, int32_t *slot_out);

/*
 * lores_decay_stat - decay statistic per head for precision assignment:
 * stat[h] = mean over n rows and `width` channels of log(alpha), computed in
 * double.  Larger (closer to 0) means slower decay.
 *   alpha  host [n][H][width] fp32, every value > 0
 *   stat   host out [H] double
 * (Decay-based mixed precision: section "Intra-State Quantization (Section 4)".)
 */
int lores_decay_stat(const float *alpha, int64_t n, int32_t H, int32_t width,
                     double *stat);

/*
 * lores_assign_precision - decay-based mixed precision (same section): heads
 * are ranked slowest-decaying first (larger stat first, ties to the lower head
 * index) and dealt into tiers listed slowest first.  Tier k takes
 * floor(tier_frac[k] * H + 0.5) heads (never more than remain); the last tier
 * takes every remaining head.
 *   stat       host [H] double (e.g. from lores_decay_stat)
 *   tier_frac  host [n_tiers] double, each >= 0
 *   tier_prec  host [n_tiers] precision codes
 *   head_prec  host out [H]
 * Host only and synchronous.
 */
int lores_assign_precision(const double *stat, int32_t H, const double *tier_frac,
                           const uint8_t *tier_prec, int32_t n_tiers, uint8_t *head_prec);

/*
 * lores_decode_step - one decode step t for all B x H units, in place: the
 * general recurrence S_t = S_{t-1} diag(alpha_t)(I - delta beta_t k_t k_t^T)
 * + beta_t v_t k_t^T and the readout o_t = S_t q_t ("Introduction and
 * Theoretical Foundation"), on a state that is dequantized, updated and
 * requantized each step ("Intra-State Quantization Approach", property 3)
 * with a fresh scale per value row and stochastic rounding ("Intra-State
 * Quantization (Section 4)": scale grouping, Proposition 1, Rounding,
 * Proposition 3).
 *   q, k        device [B][H][d_k]; fp32, or bfloat16 if in_bf16 != 0
 *   v           device [B][H][d_v]; same dtype as q and k
 *   alpha       device fp32 decay: [B][H] (scalar per head) or, if
 *               alpha_per_channel != 0, [B][H][d_k] (one per key channel)
 *   beta        device [B][H] fp32 write gate
 *   delta       0 (no correction) or 1 (delta rule)
 *   seed, t     key the stochastic rounding; t >= 1 (S_{t-1} -> S_t)
 *   seq_base,   added to the local sequence and head index before keying the
 *   head_base   rounding, so a shard of a larger batch reproduces the
 *               unsharded result bit for bit
 *   o           device out [B][H][d_v] fp32, the readout S_t q_t taken from
 *               the updated state before requantization
 * q, k, alpha, beta and o must be 4-byte aligned and v aligned to its
 * element size (LORES_EINVAL otherwise).  Caller preconditions not
 * checked: |q| = |k| = 1, decay in (0, 1], beta in (0, 2) when delta = 1,
 * finite inputs.  Per element of an int head, with U the updated fp32 row:
 *   scale' = fl(m / r), m = max|U_row|, r = 127 (int8), 31 (int6) or 7 (int4);
 *   code'  = s (floor(fl(s U * inv + bias + u)) - bias), inv = the largest
 *            fp32 not above r / m (0 if m = 0), bias = 128 (int8), 160 (int6)
 *            or 136 (int4), s = +1 in even and -1 in odd columns, and the
 *            columns 2m, 2m + 1 of a row share one draw u (so the odd column
 *            rounds U with the antithetic draw 1 - u: still unbiased),
 * fp8 heads: scale' = fl(m / 448), y = fl(U * inv) with inv the largest fp32
 *            not above 448 / m; the E4M3 byte of y is the sign and the top
 *            7 magnitude bits of f32bits(fl(y * 2^-120)) + (n << 4), which
 *            rounds stochastically on the E4M3 grid (subnormals included),
 *            u = n * 2^-16 and n a 16-bit counter-based draw keyed on
 *            (seed, t, sequence, head, row, column) (int heads: on the
 *            column pair).
 */
int lores_decode_step(lores_state *st, const void *q, const void *k, const void *v,
                      int32_t in_bf16, const float *alpha, int32_t alpha_per_channel,
                      const float *beta, int32_t delta, uint64_t seed, uint64_t t,
                      int64_t seq_base, int64_t head_base, float *o, void *stream);

/*
 * lores_step_launches - kernel launches one lores_decode_step on `st`
 * enqueues (host out *n): one per precision class present, except that the
 * pairs (int8, int4), (int4, int6), (bf16, int8) and (bf16, int4) share a
 * single launch when the state keeps value-row scales.
 */
int lores_step_launches(const lores_state *st, int32_t *n);

/*
 * lores_dequant_state - packed state -> device out [B][H][d_v][d_k] fp32: the
 * dequantization step of "Intra-State Quantization Approach" (the state read
 * back at full precision between steps; for inspection, checkpoints and the
 * error measurements of "Intra-State Quantization (Section 4)"),
 * value = scale * code for int heads (the row's or the column's scale), the
 * stored value for bf16 / fp32 heads.  For a windowed state with buffered
 * tokens: the current state, the stored state followed by the buffered
 * tokens' fp32 recurrence (as lores_state_alloc_window describes).
 */
int lores_dequant_state(const lores_state *st, float *out, void *stream);

/*
 * lores_quant_state - fp32 state -> packed state of `st`, in place of its
 * contents: the requantization of lores_decode_step applied to X itself
 * (int heads: fresh row scale and codes; bf16 heads: rounded; fp32 heads:
 * copied; key-column states take the column maxima of X), with the state's
 * rounding mode and draws keyed on step index 0,
 * which lores_decode_step never uses (t >= 1).  This hands a state built
 * elsewhere (a prefill, a checkpoint) to decoding: S_0 = Q(X).
 * ("Intra-State Quantization Approach": the state is held quantized between
 * steps; "Intra-State Quantization (Section 4)", scale grouping and Rounding.)
 *   X          device [B][H][d_v][d_k] fp32, 16-byte aligned (the layout
 *              lores_dequant_state writes), finite
 *   seed, seq_base, head_base   as for lores_decode_step
 * LORES_EINVAL on a NULL or misaligned X or out-of-range bases; nothing is
 * launched then.  On a windowed state it also empties the window buffer: the
 * next step is a window's first (t = 1, W + 1, ...).
 */
int lores_quant_state(lores_state *st, const float *X, uint64_t seed, int64_t seq_base,
                      int64_t head_base, void *stream);

/*
 * ------------------------------------------------------------------------
 * Sequence operators: the same recurrence over whole sequences at full
 * precision (prompts, training), and the norm next to it.
 * ------------------------------------------------------------------------
 */

/* Shapes of a scan.  Strides are in elements, between sequences, tokens and
 * heads; the last dimension is contiguous.  Any stride >= 0 will do (0
 * broadcasts); 16-byte aligned q and k rows are read faster. */
typedef struct {
    int32_t B, T;              /* sequences (1 .. 65535), tokens (0 .. 2^28); the heads'
                                  chunks, H (B (T / 32 + 9) + 8), number at most
                                  2^31 - 2^21 - 1                                      */
    int32_t H, H_k;            /* value heads (as lores_state_alloc), and query / key
                                  heads: H_k divides H, and value head h reads
                                  query / key head h / (H / H_k)                       */
    int32_t d_k, d_v;          /* as lores_state_alloc                                  */
    int32_t in_bf16;           /* q, k, v, o and their gradients: bf16 (1) or fp32 (0)  */
    int32_t delta;             /* 0 or 1 (delta rule)                                   */
    int64_t q_stride[3], k_stride[3], v_stride[3];
} lores_scan_dims;

/* Bytes of device workspace a lores_scan (backward = 0) or a
 * lores_scan_backward (1) of these shapes needs (host out; may be 0). */
int lores_scan_workspace(const lores_scan_dims *dims, int32_t backward, size_t *bytes);

/*
 * lores_scan - the general recurrence over T tokens without quantization,
 *   S_t = S_{t-1} alpha_t (I - delta beta_t k_t k_t^T) + beta_t v_t k_t^T,
 *   o_t = S_t q_t
 * ("Introduction and Theoretical Foundation", scalar decay per head): the
 * prompt of a layer whose decoding lores_decode_step runs.  S_last has the
 * layout that lores_quant_state takes.
 *   q, k       device [B][T][H_k][d_k] by strides
 *   v          device [B][T][H][d_v] by strides
 *   alpha      device [B][T][H] fp32 decay in [0, 1] (0 forgets everything)
 *   beta       device [B][T][H] fp32 write gate
 *   lengths    device [B] int32, or NULL: sequence b has lengths[b] tokens
 *              (values outside [0, T] are taken as 0 and T); nothing behind
 *              them is read, and o is 0 there
 *   S_first    device [B][H][d_v][d_k] fp32, 16-byte aligned, or NULL: zero
 *   o          device out [B][T][H][d_v] contiguous, the inputs' type
 *   S_last     device out [B][H][d_v][d_k] fp32, 16-byte aligned, or NULL;
 *              may be S_first
 *   work       device workspace, 256-byte aligned, of at least
 *              lores_scan_workspace bytes (NULL if that is 0); its contents
 *              do not matter before or after
 * The state and every sum are held to fp32 accuracy for either input type;
 * bf16 outputs are rounded once.  Caller preconditions not checked: finite
 * inputs, and for delta = 1 |k| = 1 and beta in (0, 2).  Nothing is launched
 * on an error.
 */
int lores_scan(const lores_scan_dims *dims, const void *q, const void *k, const void *v,
               const float *alpha, const float *beta, const int32_t *lengths,
               const float *S_first, void *o, float *S_last, void *work, size_t work_bytes,
               void *stream);

/*
 * lores_scan_backward - gradients of lores_scan's inputs from those of its
 * outputs; the forward pass is recomputed from the inputs, nothing is kept
 * between the calls.
 *   q .. S_first  as given to lores_scan
 *   dout       device [B][T][H][d_v] contiguous, the inputs' type
 *   dS_last    device [B][H][d_v][d_k] fp32, 16-byte aligned, or NULL: zero
 *   dq, dk     device out [B][T][H_k][d_k] contiguous, the inputs' type
 *              (summed over the value heads that share them, in head order)
 *   dv         device out [B][T][H][d_v] contiguous, the inputs' type
 *   dalpha, dbeta  device out [B][T][H] fp32 (also where alpha is 0)
 *   dS_first   device out [B][H][d_v][d_k] fp32, 16-byte aligned, or NULL
 *   work       as for lores_scan, of lores_scan_workspace(dims, 1) bytes
 * Gradients of tokens behind lengths[b] are 0.  Results do not depend on
 * scheduling: the same call gives the same bits.
 */
int lores_scan_backward(const lores_scan_dims *dims, const void *q, const void *k, const void *v,
                        const float *alpha, const float *beta, const int32_t *lengths,
                        const float *S_first, const void *dout, const float *dS_last, void *dq,
                        void *dk, void *dv, float *dalpha, float *dbeta, float *dS_first,
                        void *work, size_t work_bytes, void *stream);

#define LORES_MAX_NORM 16384 /* columns of a normed row */

/*
 * lores_rmsnorm - root-mean-square norm of rows, with the residual's addition
 * and an output in 8 bits with one scale per row:
 *   h = rnd(x + residual) in the inputs' type (x itself without a residual),
 *   z_j = fl(h_j w_j),  r = (mean_j h_j^2 + eps)^(-1/2),  y_j = rnd(z_j r)
 *   out_prec LORES_INT8: m = max_j |z_j| (at least 2^-119), code_j =
 *     z_j fl(127 fl(1 / m)) rounded to nearest (ties to even),
 *     scale = fl(fl(m / 127) r): y_j ~ scale code_j
 *   out_prec LORES_FP8: the same with 448 and E4M3 values
 * A row whose z are all zero has the scale 0, also at eps = 0 (where its y of
 * the other outputs are 0 times an infinite r: NaN).  A row where an h_j or z_j
 * is not finite (a weight can make it so), or where the sum of the squares
 * leaves fp32's range, has the scale NaN and the codes 0.
 *   x          device [rows][n], in_bf16 ? bf16 : fp32, rows x_stride elements
 *              apart; 1 <= n <= LORES_MAX_NORM, 0 <= rows < 2^31
 *   residual   device [rows][n] of x's type, rows res_stride apart, or NULL
 *   weight     device [n], w_bf16 ? bf16 : fp32
 *   out_prec   LORES_FP32, LORES_BF16, LORES_INT8 or LORES_FP8
 *   y          device out [rows][n] contiguous (int8 codes, E4M3 bytes)
 *   scales     device out [rows] fp32 (8-bit outputs; else unused)
 *   h          device out [rows][n] contiguous, x's type (with a residual;
 *              else unused); may be x or residual if that is contiguous
 */
int lores_rmsnorm(const void *x, int64_t x_stride, const void *residual, int64_t res_stride,
                  const void *weight, int32_t w_bf16, int64_t rows, int32_t n, int32_t in_bf16,
                  float eps, int32_t out_prec, void *y, float *scales, void *h, void *stream);

/* Bytes of device workspace of a lores_rmsnorm_backward (host out). */
int lores_rmsnorm_workspace(int64_t rows, int32_t n, size_t *bytes);

/*
 * lores_rmsnorm_backward - gradients of y = h r w (LORES_FP32 / LORES_BF16
 * output, before its rounding):
 *   dx_j = r (w_j dy_j - h_j r^2 mean_i(w_i dy_i h_i)) + dresidual_j
 *   dw_j = sum over rows of dy_j h_j r
 *   h          device [rows][n] of in_bf16's type, rows h_stride apart: the
 *              sum that lores_rmsnorm stored (x without a residual)
 *   dy         device [rows][n] contiguous, h's type
 *   dresidual  device [rows][n] contiguous, h's type: the gradient that
 *              reaches h by other ways, or NULL
 *   dx         device out [rows][n] contiguous, h's type: the gradient of x
 *              and of the residual alike; may be dy or dresidual
 *   dw         device out [n] fp32
 *   work       device workspace of lores_rmsnorm_workspace bytes, 16-byte
 *              aligned
 * Results do not depend on scheduling.
 */
int lores_rmsnorm_backward(const void *h, int64_t h_stride, const void *weight, int32_t w_bf16,
                           const void *dy, const void *dresidual, int64_t rows, int32_t n,
                           int32_t in_bf16, float eps, void *dx, float *dw, void *work,
                           size_t work_bytes, void *stream);

/*
 * ------------------------------------------------------------------------
 * Layer operators: what a layer runs per token around the recurrence - the
 * norm behind it with its gate, the norms before and after a block with its
 * gate and residual scale, and projections on microscaled 4-bit rows.
 * ------------------------------------------------------------------------
 * Rows may have any length 1 .. LORES_MAX_NORM and any alignment of their type;
 * 16-byte aligned rows of a multiple of 8 elements are read faster.  Every row is
 * computed.  Sums are fp32, results are rounded once, and do not depend on
 * scheduling.  The gradients are those of the formula before its rounding.  At
 * eps = 0 a row of zeros has an infinite r, and its y are NaN (4-bit rows: 0).
 * No output may overlap an input or another output.
 */

/* Shapes of a gated norm: rows (token, head) of n elements.  Strides are in
 * elements, between tokens and heads (0 or more: 0 broadcasts); a row is contiguous. */
typedef struct {
    int64_t tokens;            /* 0 .. ; tokens x heads < 2^31                       */
    int32_t heads, n;          /* 1 .. LORES_MAX_HEADS, 1 .. LORES_MAX_NORM          */
    int32_t in_bf16, w_bf16;   /* bf16 (1) or fp32 (0): x, gate and gradients; weight */
    int32_t per_head;          /* weight [heads][n] (1) or [n] (0)                   */
    int32_t act, gate_first;   /* LORES_ACT_*; 1: the gate comes before the norm     */
    float eps;                 /* finite, >= 0                                       */
    int64_t x_stride[2], gate_stride[2];
} lores_gated_dims;

/*
 * lores_gated_norm - the norm of the recurrence's readout with its gate, per head:
 *   gate_first 0: y_j = x_j r w_j a(z_j),  r = (mean_j x_j^2 + eps)^(-1/2)
 *   gate_first 1: u_j = x_j a(z_j),  y_j = u_j r w_j,  r of u
 *   x, gate    device rows by dims' strides
 *   weight     device [n] or [heads][n]
 *   out_prec   LORES_FP32, LORES_BF16 or LORES_MXFP4 (n a multiple of 32; a row whose
 *              squares' sum is above fp32's range, or at eps = 0 below it without being a
 *              row of zeros, has NaN scales)
 *   y          device out [tokens][heads][n] contiguous; LORES_MXFP4: codes
 *              [tokens][heads n / 2], 16-byte aligned
 *   scales     device out [tokens][4 ceil(heads n / 128)] (LORES_MXFP4: a token's
 *              row as lores_mx_matmul reads it; else unused)
 */
int lores_gated_norm(const lores_gated_dims *dims, const void *x, const void *gate,
                     const void *weight, int32_t out_prec, void *y, uint8_t *scales, void *stream);

/* Bytes of device workspace of a lores_gated_norm_backward (host out). */
int lores_gated_norm_workspace(const lores_gated_dims *dims, size_t *bytes);

/*
 * lores_gated_norm_backward - gradients of lores_gated_norm's inputs from dy:
 *   dy         device [tokens][heads][n] contiguous, x's type
 *   dx, dgate  device out [tokens][heads][n] contiguous, x's type
 *   dw         device out [n] or [heads][n] fp32
 *   work       device workspace of lores_gated_norm_workspace bytes, 16-byte aligned
 */
int lores_gated_norm_backward(const lores_gated_dims *dims, const void *x, const void *gate,
                              const void *weight, const void *dy, void *dx, void *dgate, float *dw,
                              void *work, size_t work_bytes, void *stream);

/* Shapes of the norms around a block.  Strides in elements between rows, 0 or
 * at least n (0 broadcasts one row). */
typedef struct {
    int64_t rows;              /* 0 .. 2^31 - 1                                      */
    int32_t n;                 /* 1 .. LORES_MAX_NORM                                */
    int32_t in_bf16, w_bf16;   /* bf16 (1) or fp32 (0): rows; both weights           */
    int32_t act;               /* LORES_ACT_* of the gate                            */
    float eps, scale;          /* eps of both norms; the residual scale (finite)     */
    int64_t x_stride, res_stride, gate_stride;
} lores_block_dims;

/*
 * lores_block_norm - a block's output x into the residual stream, and the next
 * block's input:
 *   p_j = x_j r1 w_j with r1 = (mean_j x_j^2 + eps)^(-1/2)   (x_j without a weight)
 *   h_j = rnd(residual_j + scale a(gate_j) p_j)              (a = 1 without a gate)
 *   y_j = h_j r2 wn_j with r2 = (mean_j h_j^2 + eps)^(-1/2)
 *   x, residual, gate  device [rows][n] by dims' strides; residual and gate may be NULL
 *   weight      device [n], the norm after the block, or NULL: none
 *   weight_next device [n], the norm before the next one
 *   out_prec    LORES_FP32, LORES_BF16, LORES_INT8, LORES_FP8 (z_j = fl(h_j wn_j)
 *               coded as by lores_rmsnorm) or LORES_MXFP4 (n a multiple of 32; a row
 *               that is not finite, or whose squares' sum is above fp32's range, or at
 *               eps = 0 below it without being a row of zeros, has NaN scales)
 *   y           device out [rows][n] contiguous; LORES_MXFP4: codes [rows][n / 2],
 *               16-byte aligned
 *   scales      device out: 8 bits [rows] fp32; LORES_MXFP4 [rows][4 ceil(n / 128)] bytes
 *   h           device out [rows][n] contiguous, x's type
 */
int lores_block_norm(const lores_block_dims *dims, const void *x, const void *residual,
                     const void *gate, const void *weight, const void *weight_next,
                     int32_t out_prec, void *y, void *scales, void *h, void *stream);

/* Bytes of device workspace of a lores_block_norm_backward (host out). */
int lores_block_norm_workspace(const lores_block_dims *dims, size_t *bytes);

/*
 * lores_block_norm_backward - gradients of lores_block_norm's inputs:
 *   x, gate, weight, weight_next  as given to lores_block_norm
 *   h          device [rows][n] contiguous, the sum that it stored
 *   dy         device [rows][n] contiguous, x's type
 *   dh         device [rows][n] contiguous, x's type: the gradient that reaches h
 *              by other ways, or NULL
 *   dx, dresidual  device out [rows][n] contiguous, x's type
 *   dgate      device out [rows][n] contiguous, x's type (with a gate; else unused)
 *   dw         device out [n] fp32 (with a weight; else unused)
 *   dw_next    device out [n] fp32
 *   work       device workspace of lores_block_norm_workspace bytes, 16-byte aligned
 */
int lores_block_norm_backward(const lores_block_dims *dims, const void *x, const void *h,
                              const void *gate, const void *weight, const void *weight_next,
                              const void *dy, const void *dh, void *dx, void *dresidual,
                              void *dgate, float *dw, float *dw_next, void *work,
                              size_t work_bytes, void *stream);

/*
 * lores_mx_quant - rows to microscaled 4-bit blocks: 32 neighbours share the
 * scale 2^e, the smallest power of two (e >= -127) with max |x| < 7 2^e, and
 * each is x 2^-e rounded to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (ties to
 * the even code; the largest is rounded, never cut off).
 *   x       device [rows][n], in_bf16 ? bf16 : fp32, rows x_stride (0 or at least n)
 *           elements apart; n a multiple of 32 up to 2^24, 0 <= rows < 2^31, rows x n at most 2^38
 *   codes   device out [rows][n / 2], 16-byte aligned: code c of column j in bits
 *           4 (j & 1) .. of byte j / 2, its sign in bit 3
 *   scales  device out [rows][4 ceil(n / 128)]: e + 127 of block j / 32, 0 behind the
 *           last; 4-byte aligned
 * A block with a value that is not finite has the scale 255 (NaN) and codes of 0.
 */
int lores_mx_quant(const void *x, int64_t x_stride, int64_t rows, int32_t n, int32_t in_bf16,
                   uint8_t *codes, uint8_t *scales, void *stream);

/* lores_mx_dequant - the values of such rows, device out [rows][n] contiguous, bf16
 * or fp32, 16-byte aligned (values beyond the type's range become infinite; scale 255: NaN).  codes
 * and scales as lores_mx_quant writes them. */
int lores_mx_dequant(const uint8_t *codes, const uint8_t *scales, int64_t rows, int32_t n,
                     int32_t out_bf16, void *out, void *stream);

/*
 * lores_mx_matmul - a projection on 4-bit weights: out[m][j] = sum_k a[m][k] w[j][k].
 *   a, a_scales  a_prec LORES_MXFP4: device codes [M][K / 2] and scales
 *                [M][4 ceil(K / 128)]; LORES_FP8: device E4M3 [M][K] and one fp32
 *                factor per row [M] (the rows that lores_rmsnorm writes)
 *   w, w_scales  device codes [N][K / 2] and scales [N][4 ceil(K / 128)]
 *   M, N, K      0 <= M < 2^31, 1 <= N <= 2^24, M x N at most 2^38, K a multiple of 32
 *                in [32, 2^24]
 *   out_prec     LORES_BF16, or with LORES_MXFP4 rows LORES_FP32
 *   out          device out [M][N] contiguous, 16-byte aligned
 * Codes are 16-byte aligned, scales 4-byte aligned; bytes behind the last block of a
 * row's scales must be 0.  Products of 4-bit values are exact and summed in fp32, in an
 * order that M, N and K alone decide.
 * With E4M3 rows the matrix instruction adds 8 neighbours of k on a grid of 2^-13 of
 * the power of two of the largest of the 8 (whose own E4M3 rounding is up to 2^-4 of
 * it), and those sums in fp32; outputs are bf16 only for that.
 */
int lores_mx_matmul(const void *a, const void *a_scales, int32_t a_prec, const uint8_t *w,
                    const uint8_t *w_scales, int64_t M, int32_t N, int32_t K, int32_t out_prec,
                    void *out, void *stream);

/* Thread-local description of the last error (empty string if none). */
const char *lores_last_error(void);

/* LORES_SPEC_VERSION of the library. */
int lores_spec_version(void);

#ifdef __cplusplus
}
#endif

#endif /* LORES_H */
