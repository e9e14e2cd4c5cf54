/*
 * pdn_block.h -- what a stack of delta-rule and attention layers needs besides
 * the recurrence (libpdn.so): the seam between two sublayers (dropout, residual,
 * norm, an output in 8 bits), softmax attention with its gradient, and the same
 * over a paged cache.
 *
 * The conventions of pdn.h and pdn_layer.h hold: plain device pointers,
 * asynchronous on the given stream of the current device, arguments validated
 * before any launch, their return codes, nothing allocated, kernels only (so that
 * a call can be captured into a HIP graph), the caller's workspace where one is
 * needed, every pointer 16-byte aligned (those to int32 and int64 numbers, to lse
 * and y_scale by the size of theirs), and "strided" as pdn_layer.h says: the last
 * dimension contiguous, strides in elements, >= 0, every row 16-byte aligned (8-byte
 * for PDN_E4M3), the rows of an output apart from each other.  No output may overlap
 * an input, another output or the workspace, except where two arguments may be one
 * buffer.
 *
 * A workspace holds no state between calls; calls that overlap need one each.
 * Results do not depend on timing or on a workspace's contents: the same call
 * gives the same bits.
 */
#ifndef PDN_BLOCK_H
#define PDN_BLOCK_H

#include "pdn_layer.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Version of the structs and calls below. */
#define PDN_BLOCK_VERSION 1
int pdn_block_version(void);

/* A type of y below: 8 bits, 4 of them exponent and 3 mantissa, no infinities,
 * largest 448. */
#define PDN_E4M3 2

/*
 * The seam between two sublayers, for each token's row of D channels:
 *
 *   s = res + keep x / (1 - p)      (held in s_dtype, rounded once)
 *   y = s r w,   r = (mean_i s_i^2 + eps)^(-1/2)        of s as it is held
 *
 * and, for PDN_E4M3, by groups of channels:
 *
 *   y_scale = top / 448,   y = nearest e4m3 of y (448 / top),   top = max(2^-64, max |y|)
 *
 * with each quotient and product rounded to fp32 (which of two neighbours a number next
 * to their middle becomes goes by that).
 *
 *   B, T, D           sizes; B >= 1; T >= 0; D a multiple of 8, <= 16384.
 *   dtype             PDN_F32 or PDN_BF16: x.
 *   s_dtype           PDN_F32, or PDN_BF16 where dtype is: res and s.
 *   y_dtype           PDN_F32, PDN_BF16 or PDN_E4M3.
 *   group             PDN_E4M3: channels of a scale: 0 = the row, or 32, 64, 128
 *                     (a divisor of D).  Otherwise 0.
 *   eps               a normal fp32 number > 0.   w: [D] fp32; NULL = ones.
 *   drop_p            0 <= p < 1: dropout of x.  round(65536 p) of 65536 values
 *                     drop an element (at most 65535), and the factor of those
 *                     kept is the inverse of their exact share.  A dropped
 *                     element counts as 0 whatever it holds.
 *   seed              [2] int64 (device), given exactly when drop_p > 0: the key,
 *                     and a number of the call.  The mask is never stored: 16 bits
 *                     for each element from Philox4x32-10 (Salmon et al., "Parallel
 *                     random numbers: as easy as 1, 2, 3"), key seed[0], counter
 *                     (n / 8, seed[1]) for element n = (b T + t) D + i, of whose
 *                     four words element n has half (n % 2) of word (n % 8) / 2.
 *   x                 strided [B,T,D] (strides sb, st).
 *   res               strided [B,T,D]; NULL = zeros.
 *   s                 strided [B,T,D]; NULL exactly when res is and drop_p is 0:
 *                     then s is x, in its type (s_dtype = dtype).  May be res (the
 *                     same strides), or x where res is NULL.
 *   y                 strided [B,T,D].
 *   y_scale           [B,T,D / group] (group 0: [B,T]) fp32, given exactly for
 *                     PDN_E4M3.
 * The sum of squares is fp32: a row in which it passes 3.4e38 has r = 0.  A row that
 * holds an infinity or NaN gives NaN where 0 times an infinity would; in 8 bits NaN
 * elements do not count for their group's scale, an infinity makes its group NaN.
 * PDN_EUNSUPPORTED where B * T reaches 2^23.
 */
typedef struct pdn_add_norm_args {
    int32_t B, T, D;
    int32_t dtype, s_dtype, y_dtype;
    int32_t group;
    float eps;
    float drop_p;
    const int64_t *seed;
    const float *w;
    const void *x;
    int64_t x_sb, x_st;
    const void *res;
    int64_t res_sb, res_st;
    void *s;
    int64_t s_sb, s_st;
    void *y;
    int64_t y_sb, y_st;
    float *y_scale;
} pdn_add_norm_args;

/*
 * Its backward; y's rounding to 8 bits counts as none:
 *
 *   dres = ds + r (g - s r^2 mean(g s)),  g = dy w
 *   dx = keep dres / (1 - p)   (of dres before its rounding)
 *   dw = sum over rows of dy s r, in a fixed order
 *
 *   B, T, D, eps, w, drop_p, seed   as in the forward.
 *   dtype             PDN_F32 or PDN_BF16: dx.
 *   s_dtype           PDN_F32, or PDN_BF16 where dtype is: s, ds, dres.
 *   y_dtype           PDN_F32 or PDN_BF16: dy.
 *   s                 strided [B,T,D] as the forward left it (x where it had none).
 *   dy                strided [B,T,D].
 *   ds                strided [B,T,D]: what reaches s otherwise; NULL = zeros.
 *   dres              strided [B,T,D]; may be ds (the same strides).
 *   dx                strided [B,T,D]; NULL = not written (without dropout dx is
 *                     dres, in dx's type).
 *   dw                [D] fp32, given exactly when w is.
 */
typedef struct pdn_add_norm_bwd_args {
    int32_t B, T, D;
    int32_t dtype, s_dtype, y_dtype;
    float eps;
    float drop_p;
    const int64_t *seed;
    const float *w;
    const void *s;
    int64_t s_sb, s_st;
    const void *dy;
    int64_t dy_sb, dy_st;
    const void *ds;
    int64_t ds_sb, ds_st;
    void *dres;
    int64_t dres_sb, dres_st;
    void *dx;
    int64_t dx_sb, dx_st;
    float *dw;
    void *workspace;
    size_t workspace_bytes;
} pdn_add_norm_bwd_args;

/*
 * Causal softmax attention.  Query i stands at position p = i + Tk - Tq (the
 * queries are the last Tq of Tk tokens) and sees the keys j with
 *
 *   max(first[b, i], p - window + 1, 0) <= j <= p
 *
 *   o_i = sum_j P_ij v_j,   P_ij = exp(scale <q_i, k_j> - lse_i)
 *
 * A query that sees no key (or none whose score is above -inf) gives o = 0 and
 * lse = -inf.  What a query does not see has no part in its output, infinities and
 * NaN included.  Of what it does see, a number of v that is not finite makes its
 * output non-finite, in that channel at least and whatever its probability; a score
 * of +inf or NaN makes all of it NaN; a score of -inf is a probability of 0 (an
 * infinite number of bf16 may give one, one of fp32 gives NaN).
 *
 *   B, H, Hk, Tq, Tk  sizes; B, H, Hk >= 1; Hk divides H (head h reads key head
 *                     h / (H / Hk)); Tq, Tk >= 0, Tq > Tk included (queries
 *                     before the first key see nothing).
 *   d                 channels of a head, of v too: 64 or 128.
 *   dtype             PDN_F32 or PDN_BF16: q, k, v.  Scores, their sums and the
 *                     outputs' sums are fp32; with bf16 the probabilities are
 *                     rounded to bf16 for their product with v.  A product of two
 *                     fp32 numbers is within 2^-24 of its own (factors below 2^-110
 *                     count to 2^-133); those from 3.396e38 on count as infinite.
 *                     The outputs' sums run over exponentials of up to 2^8.5 (2^40 in
 *                     rows whose largest score passes 2^23) and are divided at the end:
 *                     they stay finite where |v| Tk is below 2^119 (2^87); beyond, a
 *                     finite o may come out infinite or NaN.
 *   o_dtype           PDN_F32, or PDN_BF16 where dtype is: o.
 *   window            keys that a query sees at most; 0 = all.
 *   scale             finite, > 0, and so times log2(e).  A row's probabilities come from its
 *                     scores' differences, whatever their size; lse is +-inf where it
 *                     passes fp32.
 *   first             [B,Tq] int32 (device): the first key that each query may
 *                     see; NULL = 0.  So a row holds packed sequences (first = the
 *                     start of the query's own, counted in keys), padding before
 *                     them, or queries that see nothing (first >= Tk).
 *   q, o              strided [B,H,Tq,d] (strides sb, sh, st).
 *   k, v              strided [B,Hk,Tk,d].
 *   lse               [B,H,Tq] fp32; NULL = not written.
 *   workspace, workspace_bytes   at least pdn_attn_fwd_workspace_size() bytes.
 * PDN_EUNSUPPORTED where B * H passes 2^24, H / Hk 2^10, Tq H / Hk or Tk 2^30, the
 * step from token to token of k or v (in the backward of q or dO too) 2^28
 * elements, or the call's tiles (of 32 rows at least) a launch's 2^32 threads.
 */
typedef struct pdn_attn_args {
    int32_t B, H, Hk, Tq, Tk, d;
    int32_t dtype, o_dtype;
    int32_t window;
    float scale;
    const int32_t *first;
    const void *q;
    int64_t q_sb, q_sh, q_st;
    const void *k;
    int64_t k_sb, k_sh, k_st;
    const void *v;
    int64_t v_sb, v_sh, v_st;
    void *o;
    int64_t o_sb, o_sh, o_st;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
} pdn_attn_args;

/*
 * Its backward, which forms the probabilities again from q, k and lse:
 *
 *   D_i = <dO_i, o_i> = sum_j P_ij <dO_i, v_j>,  dS_ij = scale P_ij (<dO_i, v_j> - D_i)
 *   dq_i = sum_j dS_ij k_j,  dk_j = sum_i dS_ij q_i,  dv_j = sum_i P_ij dO_i
 *
 * over the heads that share a key head; sums in fp32 in a fixed order (with bf16
 * P and dS are rounded to bf16 for their products, and an fp32 dO for its own).  D is
 * taken from o as it is kept (in bf16 off by its rounding; an fp32 o avoids that), or
 * from P where a row's keys lie together.
 *
 *   fwd               the forward's arguments, o and lse as it wrote them;
 *                     workspace and workspace_bytes are not read.
 *   d_o               strided [B,H,Tq,d] in o_dtype.
 *   g_dtype           PDN_F32, or PDN_BF16 where dtype is: dq, dk, dv.
 *   dq, dk, dv        strided as q, k, v; every element is written.
 * A key or value that is not finite makes dq of all queries that see it non-finite, a
 * query or its dO dk and dv of all keys that it sees, in its own channel at least.
 * Queries that see nothing pass nothing on, whatever their q and dO hold; nor do those
 * that see no score above -inf, where these are finite.  P is formed from lse as it is
 * held, and so off by 2^-21 |lse| of itself at the most (of scores of 2^21 and more the
 * gradients mean nothing).
 */
typedef struct pdn_attn_bwd_args {
    pdn_attn_args fwd;
    int32_t g_dtype;
    const void *d_o;
    int64_t do_sb, do_sh, do_st;
    void *dq;
    int64_t dq_sb, dq_sh, dq_st;
    void *dk;
    int64_t dk_sb, dk_sh, dk_st;
    void *dv;
    int64_t dv_sb, dv_sh, dv_st;
    void *workspace;
    size_t workspace_bytes;
} pdn_attn_bwd_args;

/*
 * A cache of keys and values in pages, and the new tokens that a call brings.
 *
 *   k_pages, v_pages  [pages, page_size, Hk, d], strided (strides sp, st, sh), in
 *                     `dtype`.  page_size: a power of two, 16 to 1024.
 *   table             [B, table_width] int32 (device, contiguous): the pages of
 *                     each sequence in order.  Entries that lie behind a sequence's
 *                     last page are not read.
 *   lens              [B] int32 (device): tokens of each sequence in the cache, the
 *                     new ones included.
 *   starts            [B + 1] int32 (device): sequence b's new tokens are the rows
 *                     starts[b] .. starts[b + 1] - 1 of N, its last ones (starts
 *                     ascends, from row to row); NULL: each sequence has N / B of
 *                     them (B divides N then).
 *   max_new           at least the most new tokens of any sequence (it sizes the
 *                     launch; a sequence's rows past it are left out).
 * None of these device numbers can lead outside the arrays: table entries are
 * held to the pages there are and lens to the table's width, and a sequence whose
 * starts do not ascend within N has no new tokens.  Where they had to be held, the
 * sequence's results mean nothing (an append leaves such tokens out).  Rows that
 * belong to no sequence are left as they were.
 * PDN_EUNSUPPORTED where B passes 2^20, or table_width * page_size 2^30.
 */
typedef struct pdn_cache {
    int32_t B, N, max_new;
    int32_t Hk, d;
    int32_t dtype;
    int32_t pages, page_size, table_width;
    void *k_pages;
    int64_t k_sp, k_st, k_sh;
    void *v_pages;
    int64_t v_sp, v_st, v_sh;
    const int32_t *table;
    const int32_t *lens;
    const int32_t *starts;
} pdn_cache;

/*
 * Writes the new tokens' keys and values to their places: row starts[b] + i to
 * token lens[b] - n_b + i of sequence b, for its n_b new tokens.
 *
 *   k, v              strided [N,Hk,d] (strides sn, sh) in cache.dtype.
 *   d                 any multiple of 8, <= 1024.
 * Two sequences must not write to one page's same token.
 */
typedef struct pdn_cache_append_args {
    pdn_cache cache;
    const void *k;
    int64_t k_sn, k_sh;
    const void *v;
    int64_t v_sn, v_sh;
} pdn_cache_append_args;

/*
 * Attention of the new tokens over their sequences' caches (their own keys and
 * values included, which are there already): the token i of n_b stands at position
 * p = lens[b] - n_b + i and sees max(0, p - window + 1) <= j <= p, as pdn_attn_fwd.
 *
 *   H                 query heads; Hk divides it.       d: 64 or 128.
 *   o_dtype           PDN_F32, or PDN_BF16 where cache.dtype is: o.
 *   window, scale     as pdn_attn_fwd's.
 *   q, o              strided [N,H,d] (strides sn, sh).
 *   lse               [N,H] fp32; NULL = not written.
 *   workspace, workspace_bytes   at least pdn_attn_paged_workspace_size() bytes.
 * PDN_EUNSUPPORTED as pdn_attn_fwd's, max_new for Tq and a page's step from token to
 * token for k's.
 */
typedef struct pdn_attn_paged_args {
    pdn_cache cache;
    int32_t H, o_dtype;
    int32_t window;
    float scale;
    const void *q;
    int64_t q_sn, q_sh;
    void *o;
    int64_t o_sn, o_sh;
    float *lse;
    void *workspace;
    size_t workspace_bytes;
} pdn_attn_paged_args;

/* Validate only (no HIP call, no launch), as pdn_chunk_fwd_check. */
int pdn_add_norm_check(const pdn_add_norm_args *args);
int pdn_add_norm_bwd_check(const pdn_add_norm_bwd_args *args);
int pdn_attn_check(const pdn_attn_args *args);
int pdn_attn_bwd_check(const pdn_attn_bwd_args *args);
int pdn_cache_append_check(const pdn_cache_append_args *args);
int pdn_attn_paged_check(const pdn_attn_paged_args *args);

/* Device scratch bytes of the calls that take some (0 is valid). */
int pdn_add_norm_bwd_workspace_size(const pdn_add_norm_bwd_args *args, size_t *bytes);
int pdn_attn_fwd_workspace_size(const pdn_attn_args *args, size_t *bytes);
int pdn_attn_bwd_workspace_size(const pdn_attn_bwd_args *args, size_t *bytes);
int pdn_attn_paged_workspace_size(const pdn_attn_paged_args *args, size_t *bytes);

/* The calls themselves, on `stream`: PDN_OK, or a PDN_E* code before any
 * launch; PDN_EHIP if a launch fails. */
int pdn_add_norm_fwd(const pdn_add_norm_args *args, void *stream);
int pdn_add_norm_bwd(const pdn_add_norm_bwd_args *args, void *stream);
int pdn_attn_fwd(const pdn_attn_args *args, void *stream);
int pdn_attn_bwd(const pdn_attn_bwd_args *args, void *stream);
int pdn_cache_append(const pdn_cache_append_args *args, void *stream);
int pdn_attn_paged(const pdn_attn_paged_args *args, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PDN_BLOCK_H */
