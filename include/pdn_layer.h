/*
 * pdn_layer.h -- the operators around the gated delta rule (libpdn.so): q and k
 * out of a projection, the gated recurrence with a vector state, and the way
 * back to the model's layout, forward and backward.
 *
 * The conventions of pdn.h hold: plain device pointers, asynchronous on the
 * given stream of the current device, arguments validated before any launch,
 * its return codes, nothing allocated, kernels only (so that a call can be
 * captured into a HIP graph), and the caller's workspace where one is needed.
 * Every pointer is 16-byte aligned (PDN_EINVAL otherwise), those to positions and
 * inverse frequencies too: a slice of a longer buffer may have to be copied.
 */
#ifndef PDN_LAYER_H
#define PDN_LAYER_H

#include "pdn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of the structs and calls below (those of pdn.h have their own). */
#define PDN_LAYER_VERSION 1
int pdn_layer_version(void);

/* Tensors marked "strided" need only have their last dimension contiguous.
 * Their strides are given in elements, are >= 0, and keep every row 16-byte
 * aligned; the stride of a dimension of size 1 is not read.  Inputs may overlap
 * or repeat (stride 0); the rows of a strided output must not overlap each
 * other (PDN_EINVAL).  No output may overlap an input, another output or the
 * workspace, except where two arguments may be one buffer.
 * PDN_EUNSUPPORTED where B * T or B * D passes 2^30, or a launch's 2^32 threads
 * do not suffice (B * T past some 10^8; a scan of 2^23 or more tiles of 128
 * channels by PDN_SCAN_MARK tokens, B ceil(D / 128) ceil(T / PDN_SCAN_MARK)). */

/* Norm of a head's row x[0..d): r = (c sum x^2 + eps)^(-1/2), with c = 1/d
 * (RMS) or 1 (L2, which the delta rule's keys are commonly given). */
#define PDN_NORM_NONE 0
#define PDN_NORM_RMS 1
#define PDN_NORM_L2 2

/* Which elements of a head's first rot_dim a rotation pairs: i with
 * i + rot_dim/2, or 2i with 2i + 1. */
#define PDN_ROPE_HALF 0
#define PDN_ROPE_INTERLEAVED 1

/*
 * Norm of the queries and keys of each head, with the position rotation, from
 * the projection's layout to the recurrence's:
 *
 *   n_i = x_i r w_i scale           (scale: q_scale or k_scale)
 *   (n_i, n_j) -> rope_scale (n_i cos - n_j sin, n_j cos + n_i sin)
 *       for the pairs of the first rot_dim elements, by the angle
 *       position * inv_freq[pair], formed in 64 bits (positions of many
 *       millions keep their angles); the other elements stay
 *   out[b, h, t] = row of input head h / (H / Hx)    (a head group shares one)
 *
 *   B, T, H, d        sizes of the outputs; B, H >= 1; T >= 0; d in {64, 128}.
 *   Hq, Hk            heads of xq and xk; each divides H.
 *   dtype             PDN_F32 or PDN_BF16: xq, xk, q, k (and dxq, dxk).
 *   norm, eps         PDN_NORM_*; eps a normal fp32 number > 0 (not read
 *                     without a norm).  Sums are fp32: a row's sum of squares
 *                     must stay below its range.
 *   wq, wk            [d] fp32 weights; NULL = ones; NULL without a norm.
 *   rot_dim           0 = no rotation; else a multiple of 16, <= d.
 *   inv_freq          [rot_dim / 2] fp64 (device), radians per position.
 *   positions         [B,T] int64 (device); NULL = 0, 1, .. T - 1 in each
 *                     sequence.  Packed sequences count from their own starts
 *                     here; nothing else in this call couples tokens.
 *   xq, xk            strided [B,T,Hq,d], [B,T,Hk,d] (strides sb, st, sh).
 *   q, k              [B,H,T,d], contiguous.  With T == 1 they are the
 *                     [B,H,d] that pdn_decode_step takes.
 */
typedef struct pdn_qk_norm_args {
    int32_t B, T, H, Hq, Hk, d;
    int32_t dtype;
    int32_t norm;
    float eps;
    float q_scale, k_scale;
    int32_t rot_dim, rope_layout;
    float rope_scale;
    const double *inv_freq;
    const int64_t *positions;
    const float *wq;
    const float *wk;
    const void *xq;
    const void *xk;
    int64_t xq_sb, xq_st, xq_sh;
    int64_t xk_sb, xk_st, xk_sh;
    void *q;
    void *k;
} pdn_qk_norm_args;

/*
 * Its backward, from the fp32 gradients pdn_chunk_bwd leaves:
 *   fwd          the forward's arguments (q and k are not read).
 *   dq, dk       [B,H,T,d] fp32.
 *   dxq, dxk     strided [B,T,Hq,d], [B,T,Hk,d] in dtype; summed over the
 *                heads that share a row.
 *   dwq, dwk     [d] fp32, given exactly when the weight is.  Sums in a fixed
 *                order: the same call gives the same bits.
 */
typedef struct pdn_qk_norm_bwd_args {
    pdn_qk_norm_args fwd;
    const float *dq;
    const float *dk;
    void *dxq;
    void *dxk;
    int64_t dxq_sb, dxq_st, dxq_sh;
    int64_t dxk_sb, dxk_st, dxk_sh;
    float *dwq;
    float *dwk;
    void *workspace;
    size_t workspace_bytes;
} pdn_qk_norm_bwd_args;

/* Gate of the output norm: none, z sigmoid(z), or sigmoid(z). */
#define PDN_ACT_NONE 0
#define PDN_ACT_SILU 1
#define PDN_ACT_SIGMOID 2

/*
 * Gated norm of the recurrence's output, from its layout to the projection's:
 *
 *   y[b, t, h, i] = o[b, h, t, i] r w_i act(z[b, t, h, i])
 *   r = (mean_i o^2 + eps)^(-1/2)
 *
 *   B, H, T, dv       sizes; B, H >= 1; T >= 0; dv a multiple of 16, <= 256.
 *   o_dtype           PDN_F32 or PDN_BF16: o, [B,H,T,dv] contiguous (with
 *                     T == 1 pdn_decode_step's [B,H,dv]).
 *   dtype             PDN_F32 or PDN_BF16: z and y (and dy, dz).
 *   eps               as above.      w: [dv] fp32; NULL = ones.
 *   act, z            PDN_ACT_*; z strided [B,T,H,dv], NULL exactly when none.
 *   y                 strided [B,T,H,dv].
 */
typedef struct pdn_out_norm_args {
    int32_t B, H, T, dv;
    int32_t o_dtype, dtype;
    int32_t act;
    float eps;
    const void *o;
    const float *w;
    const void *z;
    int64_t z_sb, z_st, z_sh;
    void *y;
    int64_t y_sb, y_st, y_sh;
} pdn_out_norm_args;

/*
 * Its backward:
 *   fwd     the forward's arguments (y is not read).
 *   dy      strided [B,T,H,dv] in dtype.
 *   d_o     [B,H,T,dv] fp32, contiguous: the dO of pdn_chunk_bwd.
 *   dz      strided [B,T,H,dv] in dtype; NULL exactly when z is.
 *   dw      [dv] fp32, given exactly when w is; summed in a fixed order.
 */
typedef struct pdn_out_norm_bwd_args {
    pdn_out_norm_args fwd;
    const void *dy;
    int64_t dy_sb, dy_st, dy_sh;
    float *d_o;
    void *dz;
    int64_t dz_sb, dz_st, dz_sh;
    float *dw;
    void *workspace;
    size_t workspace_bytes;
} pdn_out_norm_bwd_args;

/* Gain of the scan's input by its decay a: 1, 1 - a, or sqrt(1 - a^2) (which
 * keeps the state's variance that of the input). */
#define PDN_GAIN_NONE 0
#define PDN_GAIN_COMPLEMENT 1
#define PDN_GAIN_NORM 2

/* Tokens between two of the scan's kept states (see marks). */
#define PDN_SCAN_MARK 96

/*
 * The gated linear recurrence with a vector state, per channel:
 *
 *   h_t = a_t h_{t-1} + g(a_t) x_t,   a_t = exp(log_a_t),   g by `gain`
 *
 * A decay that is zero in fp32 (log_a below about -87; -inf states it) drops
 * the state before it, whatever that holds, infinities and NaN included: so
 * a packed row starts each of its sequences.  Elsewhere infinities and NaN
 * in x or log_a stay in their channel at least until the decay since then
 * leaves fp32's range.
 *
 *   B, T, D           sizes; B, D >= 1; T >= 0 (hT = h0 then); D a multiple
 *                     of 8.
 *   dtype             PDN_F32 or PDN_BF16: x and h (and dh, dx).  The state is
 *                     fp32 throughout; h is rounded once, as it is written.
 *   log_dtype         PDN_F32, or PDN_BF16 where x is too: log_a (and dlog_a);
 *                     natural logarithms, <= 0.
 *   x, log_a          strided [B,T,D] (strides sb, st).   h: the same.
 *   h0                [B,D] fp32 state before the first token; NULL = zeros.
 *   hT                [B,D] fp32 state after the last; NULL = not written;
 *                     may be h0.
 *   marks             NULL, or [B, ceil(T / PDN_SCAN_MARK), D] fp32, written:
 *                     (pdn_scan_marks() of them) the states before tokens
 *                     0, PDN_SCAN_MARK, ..  A
 *                     backward that is given them need not scan forward again.
 *   workspace, workspace_bytes   at least pdn_scan_fwd_workspace_size() bytes
 *                     (0 where one workgroup's span covers T).  It holds
 *                     no state between calls; calls that overlap need one
 *                     each.
 * Results do not depend on timing or on the workspace's contents.
 */
typedef struct pdn_scan_args {
    int32_t B, T, D;
    int32_t dtype, log_dtype;
    int32_t gain;
    const void *x;
    int64_t x_sb, x_st;
    const void *log_a;
    int64_t log_a_sb, log_a_st;
    const float *h0;
    float *hT;
    void *h;
    int64_t h_sb, h_st;
    float *marks;
    void *workspace;
    size_t workspace_bytes;
} pdn_scan_args;

/*
 * Its backward: gradients of sum <dh, h> + <dhT, h_T>,
 *
 *   G_t = dh_t + a_{t+1} G_{t+1}  (dhT after the last token),
 *   dx_t = g(a_t) G_t,   dlog_a_t = (a_t h_{t-1} + g'(log_a_t) x_t) G_t,
 *   dh0 = a_1 G_1
 *
 *   fwd        the forward's arguments; h, hT, workspace and workspace_bytes
 *              are not read.  marks: as that forward wrote them (h0 is not
 *              read then), or NULL: they are formed here, in the workspace.
 *   dh         strided [B,T,D] in dtype.     dhT: [B,D] fp32; NULL = zeros.
 *   dx, dlog_a strided [B,T,D] in dtype and log_dtype.
 *   dh0        [B,D] fp32; NULL = not written; may be dhT.
 * PDN_GAIN_NORM's derivative tends to -inf as log_a tends to 0: tokens with
 * log_a = 0 (of either sign) give an infinity of the sign of -x_t G_t in dlog_a
 * (NaN where that is 0).
 */
typedef struct pdn_scan_bwd_args {
    pdn_scan_args fwd;
    const void *dh;
    int64_t dh_sb, dh_st;
    const float *dhT;
    void *dx;
    int64_t dx_sb, dx_st;
    void *dlog_a;
    int64_t dlog_a_sb, dlog_a_st;
    float *dh0;
    void *workspace;
    size_t workspace_bytes;
} pdn_scan_bwd_args;

/*
 * One token of the scan for every sequence:
 *   x, log_a, h     strided [B,D] (stride sb).
 *   h_prev, h_next  [B,D] fp32 states before and after; may be one buffer.
 */
typedef struct pdn_scan_step_args {
    int32_t B, D;
    int32_t dtype, log_dtype;
    int32_t gain;
    const void *x;
    int64_t x_sb;
    const void *log_a;
    int64_t log_a_sb;
    const float *h_prev;
    float *h_next;
    void *h;
    int64_t h_sb;
} pdn_scan_step_args;

/* Validate only (no HIP call, no launch), as pdn_chunk_fwd_check. */
int pdn_qk_norm_check(const pdn_qk_norm_args *args);
int pdn_qk_norm_bwd_check(const pdn_qk_norm_bwd_args *args);
int pdn_out_norm_check(const pdn_out_norm_args *args);
int pdn_out_norm_bwd_check(const pdn_out_norm_bwd_args *args);
int pdn_scan_check(const pdn_scan_args *args);
int pdn_scan_bwd_check(const pdn_scan_bwd_args *args);
int pdn_scan_step_check(const pdn_scan_step_args *args);

/* Device scratch bytes of the calls that take some (0 is valid). */
int pdn_qk_norm_bwd_workspace_size(const pdn_qk_norm_bwd_args *args, size_t *bytes);
int pdn_out_norm_bwd_workspace_size(const pdn_out_norm_bwd_args *args, size_t *bytes);
int pdn_scan_fwd_workspace_size(const pdn_scan_args *args, size_t *bytes);
int pdn_scan_bwd_workspace_size(const pdn_scan_bwd_args *args, size_t *bytes);

/* The calls themselves, on `stream`: PDN_OK, or a PDN_E* code before any
 * launch; PDN_EHIP if a launch fails. */
int pdn_qk_norm_fwd(const pdn_qk_norm_args *args, void *stream);
int pdn_qk_norm_bwd(const pdn_qk_norm_bwd_args *args, void *stream);
int pdn_out_norm_fwd(const pdn_out_norm_args *args, void *stream);
int pdn_out_norm_bwd(const pdn_out_norm_bwd_args *args, void *stream);
int pdn_scan_fwd(const pdn_scan_args *args, void *stream);
int pdn_scan_bwd(const pdn_scan_bwd_args *args, void *stream);
int pdn_scan_step(const pdn_scan_step_args *args, void *stream);

/* How many states `marks` holds for each sequence of T tokens:
 * ceil(T / PDN_SCAN_MARK), by the library's own spacing.  T < 0: PDN_EINVAL. */
int pdn_scan_marks(int32_t T);

/* How inverse frequencies are changed for contexts `factor` times as long as
 * the original one. */
#define PDN_ROPE_PLAIN 0     /* base^(-2i / rot_dim)                               */
#define PDN_ROPE_LINEAR 1    /* all divided by factor (positions interpolated)     */
#define PDN_ROPE_BASE 2      /* base raised by factor^(rot_dim / (rot_dim - 2)):
                                the slowest pair is divided by factor, the fastest
                                stays                                               */
#define PDN_ROPE_BY_PARTS 3  /* divided by factor where the original context holds
                                fewer than 1 turn, kept where it holds over 32, a
                                ramp over the turns between; rope_scale
                                0.1 ln(factor) + 1 ("YaRN: Efficient Context Window
                                Extension of Large Language Models", 3.2 and 3.4)   */

/* Inverse frequencies for inv_freq above, on the HOST: inv_freq [rot_dim / 2],
 * and *rope_scale (1 but for PDN_ROPE_BY_PARTS).  rot_dim even and >= 2 (>= 4
 * for PDN_ROPE_BASE), base > 1, factor >= 1, original_context >= 1 (read by
 * PDN_ROPE_BY_PARTS only).  PDN_OK, or PDN_EINVAL. */
int pdn_rope_freqs(int32_t rot_dim, double base, int32_t scaling, double factor,
                   int64_t original_context, double *inv_freq, float *rope_scale);

#ifdef __cplusplus
}
#endif

#endif /* PDN_LAYER_H */
