/*
 * pdr_dense.h -- C ABI of the dense operators beside the splatting layer: the
 * network that predicts the Gaussians' raw values, and the heavy part of the
 * optimiser that trains it, on MI355X (gfx950).
 *
 *   linear         z = x w^T + bias,  y = act(z) + res
 *   gated block    [g | u] = x w_in^T,  h = act(g) * u,  y = h w_out^T + res
 *   orthogonalize  the Newton-Schulz products of the Muon optimiser
 *
 * Conventions, in addition to pdr_splat.h's (device pointers owned by the
 * caller, no allocation, asynchronous on `stream`, arguments checked before
 * anything is enqueued, workspaces 256-byte aligned):
 *
 *  - Operands are PDR_FMT_F32, PDR_FMT_F16 or PDR_FMT_BF16, all of one format
 *    unless said otherwise.  Sums are held in fp32 and rounded once.  fp32
 *    operands are split into three bf16 values each, 24 bits over fp32's own
 *    range (of values below 2^-110, the bits above 2^-133), and multiplied as
 *    the six products of those parts that matter: what is left out of a term
 *    is at most 2^-22 of it, whatever the other terms are.  An infinity in an
 *    operand that is split makes the results it reaches not finite, as NaN or
 *    as an infinity.  (Forward products of at most 64 rows use the fp32 matrix
 *    instruction instead.)
 *  - Matrices are row-major; ld* is the distance between rows in elements
 *    (>= the row's length, <= 2^22).  Rows that begin on 16 bytes (and, where
 *    a row is summed along, hold a multiple of 8 values) are read in place;
 *    others are copied into the workspace first.
 *  - A length may be 0: sums over nothing are 0, and matrices without
 *    elements may be NULL.  Every length is below 2^31 - 256, and a matrix has
 *    fewer than 2^34 - 2^11 values (rows counted in whole 8s); so do an fp32
 *    gated block's h and, in its backward, [dg | du].
 *  - Results do not depend on the run: no atomics, one fixed order of sums
 *    for given sizes and alignments.
 *  - The *_workspace_bytes functions read the same struct as the call (sizes,
 *    strides and the pointers' alignment) and return bytes or a negative
 *    pdr_status.
 */
#ifndef PDR_DENSE_H
#define PDR_DENSE_H

#include <stddef.h>

#include "pdr_splat.h"

#ifdef __cplusplus
extern "C" {
#endif

/* silu z sigmoid(z); gelu z Phi(z) with the error function. */
typedef enum {
    PDR_ACT_NONE = 0, PDR_ACT_RELU = 1, PDR_ACT_SILU = 2, PDR_ACT_GELU = 3
} pdr_activation;

/* Rows of the tensors a forward keeps for its gradient (slope, h, gu) are
 * this many elements apart for a length of n. */
long long pdr_dense_kept_ld(long long n);

/* ------------------------------------------------------------------------ */
/* Linear: x [M][K], w [N][K], bias [N] or NULL (format fmt); res [M][N] or
 * NULL, y [M][N] (format out_fmt: fmt or PDR_FMT_F32).  slope, if not NULL,
 * receives act'(z) for the backward: [M][kept_ld(N)], 2^15 act'(z) in fp16
 * where fmt is bf16 (11 bits of a slope down to 2^-29: below bf16's own
 * rounding), else fp32.  Not used without an activation. */
typedef struct {
    int fmt, out_fmt, activation;
    long long M, N, K;
    const void *x; long long ldx;
    const void *w; long long ldw;
    const void *bias;
    const void *res; long long ldr;
    void *y; long long ldy;
    void *slope;
    /* backward only; a gradient that is NULL is not computed */
    const void *dy; long long lddy;   /* format out_fmt */
    void *dx; long long lddx;         /* [M][K], format fmt */
    void *dw; long long lddw;         /* [N][K], format fmt */
    void *dbias;                      /* [N], format fmt */
} pdr_linear;

long long pdr_linear_forward_workspace_bytes(const pdr_linear *p);
int pdr_linear_forward(const pdr_linear *p, void *workspace, size_t workspace_bytes, void *stream);

/* dz = dy act'(z), dx = dz w, dw = dz^T x, dbias = sum of dz over rows.  The
 * residual's gradient is dy.  Where dz enters the products it is rounded to
 * fmt, like dy itself, which has that format; with 16-bit operands and an fp32
 * dy, to bf16 for bf16, and for fp16 to 16 bits over fp32's range. */
long long pdr_linear_backward_workspace_bytes(const pdr_linear *p);
int pdr_linear_backward(const pdr_linear *p, void *workspace, size_t workspace_bytes,
                        void *stream);

/* ------------------------------------------------------------------------ */
/* Gated feed-forward block: x [M][D], w_in [2F][D] (gate rows, then up rows),
 * w_out [O][F], res and y [M][O].  h [M][kept_ld(F)] (format fmt) receives the
 * gated product; gu, if not NULL, the gate and up sums for the backward, fp32
 * [M][2][kept_ld(F)]. */
typedef struct {
    int fmt, activation;
    long long M, D, F, O;
    const void *x; long long ldx;
    const void *w_in; long long ld_in;
    const void *w_out; long long ld_out;
    const void *res; long long ldr;
    void *y; long long ldy;
    void *h;
    void *gu;
    /* backward only; h and gu as the forward left them; a gradient that is
     * NULL is not computed */
    const void *dy; long long lddy;
    void *dx; long long lddx;         /* [M][D] */
    void *dw_in; long long ldd_in;    /* [2F][D] */
    void *dw_out; long long ldd_out;  /* [O][F] */
} pdr_gated_mlp;

long long pdr_gated_mlp_forward_workspace_bytes(const pdr_gated_mlp *p);
int pdr_gated_mlp_forward(const pdr_gated_mlp *p, void *workspace, size_t workspace_bytes,
                          void *stream);
/* dh = dy w_out, dg = dh u act'(g), du = dh act(g), dx = [dg | du] w_in,
 * dw_in = [dg | du]^T x, dw_out = dy^T h.  dg and du are rounded to fmt, and
 * so is h: in fp16 a product of gate and up values beyond 65504 is an infinity,
 * and gradients are as coarse as fp16's step of 2^-24, as dy's are. */
long long pdr_gated_mlp_backward_workspace_bytes(const pdr_gated_mlp *p);
int pdr_gated_mlp_backward(const pdr_gated_mlp *p, void *workspace, size_t workspace_bytes,
                           void *stream);

/* ------------------------------------------------------------------------ */
/* Newton-Schulz orthogonalisation of each [m][n] matrix of a batch:
 *   X = G / (|G|_F + eps);  `steps` times: A = X X^T (X^T X where m > n),
 *   X <- a X + (b A + c A^2) X
 * For fp16 and fp32 results the iterates are held in two fp16 planes (22 bits)
 * under a power-of-two scale.  For bf16 results they have one (11 bits: every
 * step's rounding of X, A and B is carried on, so that a result is 2.0e-3 to
 * 2.5e-3 off after five steps and 2.3e-3 to 3.0e-3 after six, the more the
 * longer its rows, where rounding it once to bf16 costs 1.7e-3); a caller who
 * wants the 22 bits asks for an fp16 or fp32 result.  Coefficients that take
 * singular values s from [0, 1] on to s > 7.7, or to |b s^2 + c s^4| > 60, in
 * what a step starts from are refused: the planes would not hold them (Muon's
 * (3.4445, -4.775, 2.0315) reach 1.21 and 2.81).  steps >= 0; with 0 the result
 * is G / (|G|_F + eps). */
typedef struct {
    int fmt;                          /* of g and x */
    long long batch, m, n;
    const void *g; long long ldg, batch_g;
    void *x; long long ldx, batch_x;  /* may not alias g */
    int steps;
    float a, b, c, eps;
    int g_f32;                        /* not 0: g is PDR_FMT_F32, only x has format fmt: values that
                                         fmt's range does not hold before they are normalised */
} pdr_orthogonalize_args;

long long pdr_orthogonalize_workspace_bytes(const pdr_orthogonalize_args *p);
int pdr_orthogonalize(const pdr_orthogonalize_args *p, void *workspace, size_t workspace_bytes,
                      void *stream);

/* ------------------------------------------------------------------------ */
/* The products that a call makes, in order, and the kernels that they run in:
 * for tests and tuning.  Returns their number (the first `most` are written to
 * `out`) or a negative pdr_status.  Nothing is enqueued. */
typedef struct {
    long long M, N, K;   /* results, and what one of them sums over (in all segments) */
    int fmt;             /* of the operands' planes */
    int a_mc, b_mc;      /* operands read transposed */
    int epilogue;        /* 0 linear, 1 gated, 2 its gradient, 3 a step's polynomial */
    int batch;
    int tile;            /* rows and columns of a workgroup's tile; 0: the kernel for few rows */
    int groups;          /* of waves that share a tile's sums */
    int parts;           /* that the sums are cut into, joined by a second kernel */
    int lower;           /* only a symmetric result's lower tiles are computed */
} pdr_dense_product;

int pdr_linear_products(const pdr_linear *p, int backward, pdr_dense_product *out, int most);
int pdr_gated_mlp_products(const pdr_gated_mlp *p, int backward, pdr_dense_product *out, int most);
int pdr_orthogonalize_products(const pdr_orthogonalize_args *p, pdr_dense_product *out, int most);

#ifdef __cplusplus
}
#endif

#endif /* PDR_DENSE_H */
