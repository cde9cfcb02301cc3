/*
 * libsgemm: what a model's layer needs next to the products and the operators
 * of sgemm_ops.h, for AMD Instinct MI355X (gfx950).
 *
 *   - the gated feed-forward block, both projections, the activation and the
 *     product in one call, in float32 and for 8-bit operands, and the
 *     parts of its gradient (sgemm_f32_gated, sgemm_e4m3_gated,
 *     sgemm_f32_gated_grad, sgemm_f32_pair);
 *   - the layer norm with the residual's addition, its output in float32 or in
 *     8 bits with one scale a row, and its gradient (sgemm_layernorm_f32,
 *     sgemm_layernorm_e4m3, sgemm_layernorm_f32_grad);
 *   - the norm of all elements of many tensors, and their scaling down to a
 *     largest norm (sgemm_norm_f32, sgemm_clip_f32).
 *
 * Conventions are those of sgemm_ops.h: row-major device memory owned by the
 * caller, asynchronous work on `stream` (a stream of the current device), no
 * device allocation, no synchronisation, re-entrant; every entry point returns
 * a hipError_t as int, and argument errors come back before anything is
 * launched.  Float pointers and workspaces need 4- and 16-byte alignment.
 * Results are reproducible bit for bit for the same arguments on the same
 * device: nothing is added atomically.
 *
 * Overlap: an output must not overlap any other output, an input or the
 * workspace, but for the exceptions each call names, where the two must be the
 * same memory with the same row stride.  Tensors of one row stride that are
 * different columns of one matrix (the halves of a tensor that holds a gated
 * layer's two weights side by side) do not overlap.
 */
#ifndef SGEMM_LAYERS_H
#define SGEMM_LAYERS_H

#include "sgemm_ops.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * What a gated block does to its two sums, g of the gate's product and u of
 * the other one:
 *
 *   g = g + bias_gate[n],  u = u + bias_up[n]
 *   C = act(g) * u, with g and u stored to pre_gate[m][n] and pre_up[m][n]
 *       where those are given (the gradient needs both).
 *
 * activation is one of SGEMM_ACT_*; a null pointer leaves its part out.
 */
typedef struct sgemm_gate {
    int activation;
    const float *bias_gate, *bias_up; /* N values each */
    float *pre_gate;
    int ld_pre_gate;
    float *pre_up;
    int ld_pre_up;
} sgemm_gate;

/* Forms of sgemm_f32_gated: the library's choice, one of the fused tiles
 * (0 .. SGEMM_GATED_TILES - 1), the form that streams the weights for a few rows, and two
 * plain products into the workspace. */
#define SGEMM_GATED_AUTO (-1)
#define SGEMM_GATED_TILES 6
#define SGEMM_GATED_ROWS 6
#define SGEMM_GATED_PRODUCTS 7

/*
 * sgemm_f32_gated: C = act(A x op(B_gate) + bias_gate) * (A x op(B_up) +
 * bias_up) in float32.
 *
 *   A, lda   M x K, lda >= max(1, K).
 *   B_gate, B_up  K x N (transb 0, row strides >= max(1, N)) or N x K (transb
 *            1, >= max(1, K)) each; the halves of one tensor or two tensors.
 *   C, ldc   M x N, ldc >= max(1, N).
 *   workspace  optional (16-byte aligned; NULL with 0 bytes for none): lets the
 *            two products run with K split over workgroups where the output
 *            has few tiles.  The library's wish for these very operands (its
 *            choice depends on their alignment; they are not read) is
 *            sgemm_f32_gated_workspace's.
 *   form     SGEMM_GATED_AUTO, or a form to force; one that does not serve the
 *            call is refused with hipErrorInvalidValue.
 * M, N, K and every ld are at most INT_MAX - 1024.  M == 0 or N == 0 does
 * nothing; K == 0 gives the block of two sums of nothing, without reading A or
 * the weights.
 */
int sgemm_f32_gated(int transb, int M, int N, int K, const float *A, int lda,
                    const float *B_gate, int ldb_gate, const float *B_up, int ldb_up,
                    float *C, int ldc, const sgemm_gate *gate,
                    void *workspace, size_t workspace_bytes, int form, hipStream_t stream);
int sgemm_f32_gated_workspace(int transb, int M, int N, int K, const float *A, int lda,
                              const float *B_gate, int ldb_gate, const float *B_up, int ldb_up,
                              size_t *bytes);

/*
 * sgemm_e4m3_gated: the gated block of 8-bit (e4m3) operands, float32 sums
 * and results: A is M x K codes, B_gate and B_up N x K codes each, with
 * scale_a (M), scale_gate and scale_up (N factors, NULL for ones) as in
 * sgemm_e4m3, whose other conventions hold.
 */
int sgemm_e4m3_gated(int M, int N, int K, const void *A, int lda, const float *scale_a,
                     const void *B_gate, int ldb_gate, const float *scale_gate,
                     const void *B_up, int ldb_up, const float *scale_up,
                     float *C, int ldc, const sgemm_gate *gate,
                     void *workspace, size_t workspace_bytes, hipStream_t stream);
int sgemm_e4m3_gated_workspace(int M, int N, int K, size_t *bytes);

/*
 * sgemm_f32_gated_grad: the elementwise part of a gated block's gradient in
 * one pass, from its output's gradient and the stored g and u,
 *
 *   dG = dY * U * act'(G),   dU = dY * act(G),
 *   dbias_gate, dbias_up = the column sums of dG and of dU.
 *
 *   dG, dU   M x N each, or NULL; each may be the memory of one of the inputs
 *            (same pointer and ld).
 *   dbias_gate, dbias_up   N values each, or NULL.  M == 0 gives zeros.
 *   workspace  16-byte aligned, at least sgemm_f32_gated_grad_workspace's
 *            bytes; NULL with 0 bytes where both sums are NULL.  Too little is
 *            refused.
 * M, N <= INT_MAX - 1024, ld >= max(1, N).  N == 0 does nothing.
 */
int sgemm_f32_gated_grad(int M, int N, int activation, const float *dY, int ldy,
                         const float *G, int ldg, const float *U, int ldu,
                         float *dG, int lddg, float *dU, int lddu, float *dbias_gate, float *dbias_up,
                         void *workspace, size_t workspace_bytes, hipStream_t stream);
int sgemm_f32_gated_grad_workspace(int M, int N, size_t *bytes);

/*
 * sgemm_f32_pair: C = A1 x op(B1) + A2 x op(B2) in float32, such as the
 * gradient that goes on from a gated block, dA = dG x op(B_gate)^T + dU x
 * op(B_up)^T.  A1 and A2 are M x K with one row stride; B1 and B2 are K x N, or
 * N x K with transb.
 *
 *   workspace  optional (16-byte aligned; NULL with 0 bytes for none): lets the
 *            two run together, and with K split over workgroups.  The
 *            library's wish for these very operands (they are not read) is
 *            sgemm_f32_pair_workspace's.
 * Limits, errors and edge cases as sgemm_f32_ex (sgemm.h).
 */
int sgemm_f32_pair(int transb, int M, int N, int K,
                   const float *A1, const float *A2, int lda,
                   const float *B1, int ldb1, const float *B2, int ldb2, float *C, int ldc,
                   void *workspace, size_t workspace_bytes, hipStream_t stream);
int sgemm_f32_pair_workspace(int transb, int M, int N, int K,
                             const float *A1, const float *A2, int lda,
                             const float *B1, int ldb1, const float *B2, int ldb2, size_t *bytes);

/*
 * sgemm_layernorm_f32: per row of D values,
 *
 *   S = X + R,   Y = (S - mean(S)) / sqrt(var(S) + eps) * w + b,
 *
 * var the mean of the squared differences from the mean.
 *
 *   R       the residual, or NULL (S = X).
 *   w, b    D values each, or NULL (ones, zeros).
 *   S       rows x D, or NULL when the sum is not wanted; it may be X's or
 *           R's memory (same pointer and ld).
 *   Y       rows x D; it may be X's, R's memory when S is not.
 *   eps     >= 0, finite.  A constant row with eps == 0 gives NaN (0 / 0).
 * D >= 1, rows >= 0, both <= INT_MAX - 1024; every ld >= D.  The mean and the
 * squares are summed in float64, so no square overflows.  S - mean(S) and the
 * inverse root are float32: a value further from the mean than float32 reaches
 * (3.4e38, with values of both signs near it) is infinite here, and rows whose
 * root passes 2^126 lose bits of the inverse.  A row that holds an infinity or
 * NaN is NaN throughout.
 */
int sgemm_layernorm_f32(int rows, int D, const float *X, int ldx, const float *R, int ldr,
                        const float *w, const float *b, float eps, float *S, int lds, float *Y, int ldy,
                        hipStream_t stream);

/* sgemm_layernorm_e4m3: the same with the output in 8 bits and one float32
 * scale a row, as sgemm_rmsnorm_e4m3 (Y / scale is float64 from S up to
 * the rounding to a code). */
int sgemm_layernorm_e4m3(int rows, int D, const float *X, int ldx, const float *R, int ldr,
                         const float *w, const float *b, float eps, float *S, int lds,
                         void *Q, int ldq, float *scale, hipStream_t stream);

/*
 * sgemm_layernorm_f32_grad: the gradient of Y = h * w + b, h = d * r, d = S -
 * mean(S), r = 1 / sqrt(var(S) + eps), from dY.  With g = dY * w, per row
 *
 *   dX = r * (g - mean(g) - h * mean(g * h)) + dS,
 *   dw = sum over rows of dY * h,   db = sum over rows of dY.
 *
 *   S       the norm's input sum (X + R); dX is the gradient of X and of R.
 *   w       D values, or NULL (ones).
 *   dS      the gradient that reaches S past the norm (the residual stream's),
 *           or NULL; dX may be dS's memory (same pointer and ld).
 *   dX      rows x D.
 *   dw, db  D values each, or NULL.  rows == 0 gives zeros.
 *   workspace  16-byte aligned, at least what
 *           sgemm_layernorm_f32_grad_workspace gives; NULL with 0 bytes where
 *           dw and db are NULL.  Too little is refused.
 * A row's sums are float64, the sums over rows float32; mean(g) and mean(g * h)
 * are rounded to float32, which holds them for rows of any size.
 * Other arguments as sgemm_layernorm_f32.
 */
int sgemm_layernorm_f32_grad(int rows, int D, const float *dY, int ldy, const float *S, int lds,
                             const float *w, float eps, const float *dS, int ldds,
                             float *dX, int lddx, float *dw, float *db,
                             void *workspace, size_t workspace_bytes, hipStream_t stream);
int sgemm_layernorm_f32_grad_workspace(int rows, int D, size_t *bytes);

/* One of many tensors: rows x cols elements, rows ldx (of x) and ldy (of y)
 * elements apart; the strides matter when rows > 1. */
typedef struct sgemm_tensor {
    const float *x;
    float *y;
    long long rows, cols;
    long long ldx, ldy;
} sgemm_tensor;

/*
 * sgemm_clip_f32: over all elements of `count` tensors,
 *
 *   n = sqrt(sum x^2),   y = x * min(1, max_norm / (n + eps)).
 *
 *   tensors  a host array, read before the call returns.  rows and cols >= 0
 *            (an empty tensor is left out, whatever its pointers); rows <=
 *            INT_MAX - 1024, cols too where rows > 1, else <= 2^40; strides >=
 *            cols.  y may be x's memory (same stride).  No two tensors may
 *            share memory that one of them writes; the halves of one matrix
 *            do not.
 *   max_norm, eps   >= 0, finite.
 *   norm     n, one float, or NULL.
 *   workspace  16-byte aligned, at least sgemm_clip_f32_workspace's bytes.
 * Squares and sums are float64, and the factor is taken from the unrounded n
 * and rounded once, to float32's precision wherever it lies (what is stored of n
 * is infinite past float32's range, the factor is not 0 then).  A NaN, or an
 * infinity, anywhere makes n so: the factor is then NaN, or 0.  Where every y is its x and the factor is 1 nothing is
 * written.  Up to 96 tensors take two launches, or one if they are small; more take
 * one for every 96 besides.
 */
int sgemm_clip_f32(int count, const sgemm_tensor *tensors, float max_norm, float eps, float *norm,
                   void *workspace, size_t workspace_bytes, hipStream_t stream);
int sgemm_clip_f32_workspace(int count, size_t *bytes);

/* sgemm_norm_f32: n alone; y and ldy are not read, and the same memory may be
 * named twice (and counts twice).  Workspace as sgemm_clip_f32. */
int sgemm_norm_f32(int count, const sgemm_tensor *tensors, float *norm,
                   void *workspace, size_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_LAYERS_H */
