/*
 * pdr_blocks.h -- C ABI of the operators that make a transformer block of the
 * dense ones (pdr_dense.h), on MI355X (gfx950).
 *
 *   attention   softmax(scale q k^T) v over whole, packed or cached sequences
 *   layer norm  (x - mean) / sqrt(var + eps) * weight + bias
 *   dropout     kept values / (1 - p) + residual, the choice from a counter
 *
 * Conventions are those of pdr_splat.h and pdr_dense.h (device pointers owned
 * by the caller, no allocation, asynchronous on `stream`, arguments checked
 * before anything is enqueued, workspaces 256-byte aligned).  Tensors are
 * PDR_FMT_F32, PDR_FMT_F16 or PDR_FMT_BF16, all of one format; sums, softmax
 * statistics, means and variances are held in fp32.  Results do not depend on
 * the run: no atomics, one fixed order of sums for given sizes and alignments.
 */
#ifndef PDR_BLOCKS_H
#define PDR_BLOCKS_H

#include <stddef.h>

#include "pdr_splat.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------ */
/* Attention.  Query head h reads key head h / (heads / kv_heads):
 *   s_ij = scale q_i . k_j,  L_i = log sum_j exp(s_ij),  p_ij = exp(s_ij - L_i)
 *   o_i = sum_j p_ij v_j
 * over the keys j that query i sees: all of its sequence's, or if `causal` is
 * not 0 those with j <= i + (keys - queries), so that the last query sees every
 * key.  A query that sees no key (or only keys whose score is -infinity) gets
 * zeros and has no gradient.  What a query does not see does not reach its
 * result, whatever it holds.  Nor does it reach gradients across sequences, or
 * from behind a length; but within a causal sequence an infinity or NaN may make
 * gradients not finite that it is masked from, of up to 190 tokens beside it (the
 * rows of a workgroup, 128, and of a tile, 64, without themselves).
 *
 * Sequences.  Without offsets there are `batch` of them, each of q_rows
 * queries and k_rows keys, *_batch elements apart; key_lengths, if not NULL,
 * says how many of its keys each sequence has (int32 [batch]; taken into
 * [0, k_rows]).  With offsets they lie one after another in q_rows and k_rows
 * tokens altogether: sequence b has queries [q_offsets[b], q_offsets[b + 1])
 * and keys [k_offsets[b], k_offsets[b + 1]) (int32 [batch + 1], not descending).
 * Tokens outside of all sequences get zeros.  Offsets and lengths are device
 * memory and not looked at by the host.  Those that leave the tokens are taken
 * to their ends; where they descend results are undefined, but no access leaves
 * the tensors.
 *
 * Layout.  A tensor's element (sequence b, token i, head h, d) is at
 * b batch + i row + h head + d: strides in elements, not negative, all of them
 * multiples of 16 bytes like the pointers and dim; rows at most 2^22 elements
 * apart, heads at most 2^24 and all heads of a tensor at most 2^28.  dim <= 128.
 * Tensors that are written (o, dq, dk, dv) have no two elements at one place.
 *
 * Lengths may be 0.  Queries (of all sequences) times heads stay below 2^29, in
 * the backward also keys times kv_heads, and sequences times kv_heads below 2^23. */
typedef struct {
    int fmt, causal;
    long long batch, heads, kv_heads, dim;
    long long q_rows, k_rows;
    const int *q_offsets, *k_offsets;  /* both or none */
    const int *key_lengths;            /* only without offsets */
    float scale;                       /* in [2^-64, 2^64] */
    const void *q; long long q_row, q_head, q_batch;
    const void *k; long long k_row, k_head, k_batch;
    const void *v; long long v_row, v_head, v_batch;
    void *o; long long o_row, o_head, o_batch;       /* read by the backward */
    float *lse;   /* L / log(2), or +infinity where there is no key; [kv_heads][queries]
                     [heads / kv_heads], queries of all sequences.  May be NULL in the forward */
    /* backward only; a gradient that is NULL is not computed */
    const void *dy; long long dy_row, dy_head, dy_batch;
    void *dq; long long dq_row, dq_head, dq_batch;
    void *dk; long long dk_row, dk_head, dk_batch;   /* dk and dv: both or none */
    void *dv; long long dv_row, dv_head, dv_batch;
} pdr_attention;

long long pdr_attention_forward_workspace_bytes(const pdr_attention *p);
int pdr_attention_forward(const pdr_attention *p, void *workspace, size_t workspace_bytes,
                          void *stream);
/* delta_i = dy_i . o_i, ds_ij = p_ij (dy_i . v_j - delta_i), dq_i = scale sum_j ds_ij k_j,
 * dk_j = scale sum_i ds_ij q_i, dv_j = sum_i p_ij dy_i; sums over i are over
 * all heads that read the key's.  p and ds are rounded to fmt where they enter
 * the products, as p is in the forward (in fp16 under powers of two that keep them
 * in its range: p to 2^-37 of a row's largest in the forward, to 2^-40 here). */
long long pdr_attention_backward_workspace_bytes(const pdr_attention *p);
int pdr_attention_backward(const pdr_attention *p, void *workspace, size_t workspace_bytes,
                           void *stream);

/* ------------------------------------------------------------------------ */
/* Layer norm of each row of x [rows][cols]:
 *   y = (x - mean) rstd weight + bias,  rstd = 1 / sqrt(var + eps)
 * with the variance over cols.  weight and bias [cols] or NULL (one and zero).
 * stats, if not NULL, receives (mean, rstd) of each row for the backward, fp32
 * [rows][2].  Rows are ld* elements apart; any alignment.  There are fewer than
 * 2^31 - 256 rows, of at most 2^30 values. */
typedef struct {
    int fmt;
    long long rows, cols;
    float eps;
    const void *x; long long ldx;
    const void *weight, *bias;
    void *y; long long ldy;
    float *stats;
    /* backward only; a gradient that is NULL is not computed */
    const void *dy; long long lddy;
    void *dx; long long lddx;
    void *dweight, *dbias;
} pdr_layer_norm;

long long pdr_layer_norm_forward_workspace_bytes(const pdr_layer_norm *p);
int pdr_layer_norm_forward(const pdr_layer_norm *p, void *workspace, size_t workspace_bytes,
                           void *stream);
/* xh = (x - mean) rstd, g = dy weight, dx = rstd (g - mean(g) - xh mean(g xh)),
 * dweight = sum of dy xh and dbias = sum of dy over rows. */
long long pdr_layer_norm_backward_workspace_bytes(const pdr_layer_norm *p);
int pdr_layer_norm_backward(const pdr_layer_norm *p, void *workspace, size_t workspace_bytes,
                            void *stream);

/* ------------------------------------------------------------------------ */
/* Dropout: y = (element i is kept ? x / (1 - t / 65536) : 0) + residual, with
 * t = p 65536 rounded to a whole number.  Element i, counted along the rows of
 * [rows][cols], is kept if its 16 bits are not below t: half i % 2 (low first)
 * of word i / 2 % 4 of Philox 4x32 with 10 rounds (Salmon, Moraes, Dror, Shaw
 * 2011) under the key `seed` at the counter (i / 8, offset), low words first.
 * Nothing is stored for the backward, which is the same call on dy without a
 * residual.  rows times cols is below 2^40. */
typedef struct {
    int fmt;
    long long rows, cols;
    double p;                             /* in [0, 1] */
    unsigned long long seed, offset;
    const unsigned long long *seed_at;    /* device memory, or NULL: the seed, instead of `seed` */
    const void *x; long long ldx;
    const void *res; long long ldr;       /* or NULL */
    void *y; long long ldy;
} pdr_dropout_args;

long long pdr_dropout_workspace_bytes(const pdr_dropout_args *p);
int pdr_dropout(const pdr_dropout_args *p, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PDR_BLOCKS_H */
