/*
 * libsgemm: the operators that stand around a matrix product in a model's
 * layers, for AMD Instinct MI355X (gfx950).
 *
 *   - the float32 product with bias, activation and residual in its epilogue,
 *     and the parts of its gradient (sgemm_f32_epilogue,
 *     sgemm_f32_activation_grad);
 *   - the root-mean-square norm with the residual's addition, its output in
 *     float32 or in 8 bits with one scale a row, and its gradient
 *     (sgemm_rmsnorm_f32, sgemm_rmsnorm_e4m3, sgemm_rmsnorm_f32_grad);
 *   - rows of float32 to 8 bits with one scale a row (sgemm_quantize_e4m3);
 *   - the product of two such 8-bit matrices with the same epilogue
 *     (sgemm_e4m3).
 *
 * Conventions are those of sgemm.h: row-major device memory owned by the
 * caller, asynchronous work on `stream` (a stream of the current device), no
 * allocation, no synchronisation, re-entrant; every entry point returns a
 * hipError_t as int, and argument errors come back before anything is
 * launched.  Float pointers and workspaces need 4- and 16-byte alignment.
 * Results are reproducible bit for bit for the same arguments on the same
 * device: nothing is added atomically.
 *
 * Overlap: an output must not overlap any other output, an input or the
 * workspace (the spans from the first to the last element are compared), but
 * for the exceptions each call names, where the two must be the same memory
 * with the same row stride.
 */
#ifndef SGEMM_OPS_H
#define SGEMM_OPS_H

#include "sgemm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Activations, act(z):
 *   RELU       max(z, 0)
 *   GELU       z Phi(z), Phi the normal distribution function
 *   GELU_TANH  z (1 + tanh(sqrt(2/pi) (z + 0.044715 z^3))) / 2
 *   SILU       z / (1 + exp(-z))
 * Each is the formula in float32: NaN gives NaN (and the last three of minus
 * infinity too, as 0 times infinity). */
#define SGEMM_ACT_NONE 0
#define SGEMM_ACT_RELU 1
#define SGEMM_ACT_GELU 2
#define SGEMM_ACT_GELU_TANH 3
#define SGEMM_ACT_SILU 4

/*
 * What a product does to its sum s = sum_k op(A) op(B) before it is written:
 *
 *   z = alpha * s + bias[n]
 *   y = act(z), with z stored to pre[m][n] when pre is given; or
 *   y = z * act'(grad_pre[m][n]) when grad_pre is given
 *   C = y + residual[m][n]
 *
 * A null pointer leaves its part out.  pre and grad_pre exclude each other.
 * act' of RELU is 1 where its argument is above 0 and else 0.  Every ld is at
 * least max(1, N).  Strides (elements between batch entries, >= 0; 0 reuses
 * one bias, grad_pre or residual for every entry) matter when batch > 1; pre's
 * must keep its entries apart as C's do.  C may be the residual's memory (same
 * pointer, ld and stride): the product is then added to it.
 */
typedef struct sgemm_epilogue {
    int activation;
    const float *bias; /* N values */
    long long stride_bias;
    float *pre;
    int ld_pre;
    long long stride_pre;
    const float *grad_pre;
    int ld_grad_pre;
    long long stride_grad_pre;
    const float *residual;
    int ld_residual;
    long long stride_residual;
} sgemm_epilogue;

/*
 * sgemm_f32_epilogue: `batch` products C_z = epilogue(alpha * op(A_z) x
 * op(B_z)).  Arguments, limits, workspace and errors are those of
 * sgemm_f32_ex (sgemm.h), without beta.  The workspace that the selector would
 * like is sgemm_f32_workspace_size's; with a K split the epilogue is applied
 * once, to the sum of the partial products.  K == 0 or alpha == 0 gives s = 0:
 * the epilogue of zero, without reading A or B.
 *
 *   epi   NULL for none (a plain product).
 *   cfg   NULL, or a forced configuration (as sgemm_f32_ex): the direct-load
 *         tiles and the tiles that split K inside the workgroup serve
 *         epilogues, the other variants are refused with
 *         hipErrorInvalidValue.
 */
int sgemm_f32_epilogue(int transa, int transb, int M, int N, int K,
                       float alpha,
                       const float *A, int lda, long long stride_a,
                       const float *B, int ldb, long long stride_b,
                       float *C, int ldc, long long stride_c,
                       int batch, const sgemm_epilogue *epi,
                       void *workspace, size_t workspace_bytes,
                       hipStream_t stream, const sgemm_cfg *cfg);

/*
 * sgemm_f32_activation_grad: the elementwise part of a layer's gradient in
 * one pass over its output's gradient,
 *
 *   dZ[m][n] = dY[m][n] * act'(Z[m][n]),   dbias[n] = sum_m dZ[m][n].
 *
 *   Z       the pre-activations (read only when activation is not NONE, and
 *           then required).
 *   dZ      M x N, or NULL when only dbias is wanted; it may be dY's memory
 *           (same pointer and ld).
 *   dbias   N values, or NULL.  M == 0 gives zeros.
 *   workspace  16-byte aligned, at least the bytes that
 *           sgemm_f32_activation_grad_workspace gives (rows are summed in
 *           chunks, and the chunks' sums in a fixed order); NULL with 0 bytes
 *           where that is 0 or dbias is NULL.  Too little is refused.
 * M, N <= INT_MAX - 1024, ld >= max(1, N).  N == 0 does nothing.
 */
int sgemm_f32_activation_grad(int M, int N, int activation,
                              const float *dY, int ldy, const float *Z, int ldz,
                              float *dZ, int lddz, float *dbias,
                              void *workspace, size_t workspace_bytes, hipStream_t stream);
int sgemm_f32_activation_grad_workspace(int M, int N, size_t *bytes);

/*
 * sgemm_rmsnorm_f32: per row of D values,
 *
 *   S = X + R,   Y = S / sqrt(mean(S^2) + eps) * w.
 *
 *   R       the residual, or NULL (S = X).
 *   w       D values, or NULL (ones).
 *   S       rows x D, or NULL when the sum is not wanted; it may be X's or
 *           R's memory (same pointer and ld).
 *   Y       rows x D; it may be X's, R's memory when S is not.
 *   eps     >= 0, finite.  A row of zeros with eps == 0 gives NaN (0 / 0).
 * D >= 1, rows >= 0, both <= INT_MAX - 1024; every ld >= D.  Squares are
 * float32, their sum across threads float64; S * w is formed in float32.  So
 * |S| above 1.8e19 overflows (Y is 0), and where eps is 0 a row of values below
 * 1e-19 loses its squares' bits, one below 2e-23 all of them (Y is infinite).
 */
int sgemm_rmsnorm_f32(int rows, int D, const float *X, int ldx, const float *R, int ldr,
                      const float *w, float eps, float *S, int lds, float *Y, int ldy,
                      hipStream_t stream);

/*
 * sgemm_rmsnorm_e4m3: the same with the output in 8 bits (OCP e4m3: 4
 * exponent and 3 mantissa bits, largest value 448, one NaN and no infinity)
 * and one float32 scale a row:
 *
 *   scale = max(max_d |Y_d| / 448, 2^-126),   Q_d = e4m3(Y_d / scale),
 *
 * rounded to nearest, ties to even, so that Q_d * scale stands for Y_d (codes
 * are those of the unrounded scale, what is stored is rounded; the row's
 * largest S * w is taken in float32).  NaN
 * values of Y become the NaN code and are left out of the row's maximum; a row
 * that holds an infinity has an infinite scale.  Q is rows x D bytes with row
 * stride ldq >= D.  Rows that start 16-byte aligned (ldq a multiple of 16) are
 * what sgemm_e4m3 reads fastest; the bytes between D and ldq are left as they
 * are.  Other arguments as sgemm_rmsnorm_f32.
 */
int sgemm_rmsnorm_e4m3(int rows, int D, const float *X, int ldx, const float *R, int ldr,
                       const float *w, float eps, float *S, int lds, void *Q, int ldq, float *scale,
                       hipStream_t stream);

/* sgemm_quantize_e4m3: the rows of X themselves to 8 bits (Y = X above). */
int sgemm_quantize_e4m3(int rows, int D, const float *X, int ldx, void *Q, int ldq, float *scale,
                        hipStream_t stream);

/*
 * sgemm_rmsnorm_f32_grad: the gradient of Y = S / sqrt(mean(S^2) + eps) * w
 * from dY.  With r = 1 / sqrt(mean(S^2) + eps) and g = dY * w, per row
 *
 *   dX = r * g - S * r^3 * mean(g * S) + dS,   dw = sum over rows of dY * S * r.
 *
 *   S       the norm's input sum (X + R); dX is the gradient of X and of R.
 *   w       D values, or NULL (ones).
 *   dS      the gradient that reaches S past the norm (the residual stream's),
 *           or NULL; dX may be dS's memory (same pointer and ld).
 *   dX      rows x D.
 *   dw      D values, or NULL.  rows == 0 gives zeros.
 *   workspace  16-byte aligned, at least what sgemm_rmsnorm_f32_grad_workspace
 *           gives on the current device; NULL with 0 bytes where that is 0 or
 *           dw is NULL.  Too little is refused.
 * Other arguments as sgemm_rmsnorm_f32.
 */
int sgemm_rmsnorm_f32_grad(int rows, int D, const float *dY, int ldy, const float *S, int lds,
                           const float *w, float eps, const float *dS, int ldds,
                           float *dX, int lddx, float *dw,
                           void *workspace, size_t workspace_bytes, hipStream_t stream);
int sgemm_rmsnorm_f32_grad_workspace(int rows, int D, size_t *bytes);

/*
 * sgemm_e4m3: the product of two 8-bit (e4m3) matrices, float32 sums,
 *
 *   C = epilogue(scale_a[m] * scale_b[n] * sum_k A[m][k] B[n][k]).
 *
 *   A, lda  M x K bytes, row stride lda >= max(1, K): activations.
 *   B, ldb  N x K bytes, row stride ldb >= max(1, K): weights stored with one
 *           row per output.
 *   scale_a, scale_b   M and N float32 factors, or NULL (ones).
 *   C, ldc  M x N float32.
 *   epi     as sgemm_f32_epilogue (alpha 1; strides are not used), or NULL.
 *   workspace  optional (16-byte aligned; NULL with 0 bytes for none): lets K
 *           be split across workgroups when the output has few tiles.  The
 *           selector's wish is sgemm_e4m3_workspace_size's.
 * Pointers of A and B and lda, ldb may be any (rows that start 16-byte aligned
 * run fastest).  M, N, K and every ld <= INT_MAX - 1024.  M == 0 or N == 0 does
 * nothing; K == 0 gives the epilogue of zero.  Products of codes are exact and
 * summed in float32 by the matrix cores; a NaN code gives NaN.
 */
int sgemm_e4m3(int M, int N, int K, const void *A, int lda, const float *scale_a,
               const void *B, int ldb, const float *scale_b, float *C, int ldc,
               const sgemm_epilogue *epi, void *workspace, size_t workspace_bytes,
               hipStream_t stream);
int sgemm_e4m3_workspace_size(int M, int N, int K, size_t *bytes);

#ifdef __cplusplus
}
#endif

#endif /* SGEMM_OPS_H */
