/*
 * dense_ops.h - C ABI of the dense operators that stand between a table's
 * looked-up rows and the loss: layer norm (forward and backward), the
 * Newton-Schulz orthogonalisation of a matrix, and the Muon step that applies
 * it to a weight.
 *
 * The conventions are those of sparse_opt.h: device pointers owned by the
 * caller, `stream` a hipStream_t as void*, SPOPT_OK or a negative spopt_status,
 * the message in sparse_opt_last_error().  No call here allocates; trusted
 * calls never synchronise and hold nothing that changes from step to step, so
 * they can be captured into a HIP graph.  With SPOPT_VALIDATE a call first
 * reads x (and dy), or the gradient, on the device (one synchronisation) and
 * returns SPOPT_ENONFINITE, having written nothing, where it holds a NaN or an
 * infinity.  Results are the same bit for bit from run to run.
 */
#ifndef DENSE_OPS_H
#define DENSE_OPS_H

#include "sparse_opt.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- element types ------------------------------------------------------ */
#define SPOPT_DTYPE_F32 0
#define SPOPT_DTYPE_BF16 1
#define SPOPT_DTYPE_F16 2

/* ---- layer norm --------------------------------------------------------- */

/* Layer norm over the last axis, for rows x cols values with row k at
 * x + k * x_stride (strides in elements, columns adjacent):
 *   mean = sum(x) / cols, var = sum((x - mean)^2) / cols,
 *   rstd = 1 / sqrt(var + eps), y = (x - mean) * rstd * weight + bias.
 *   x, y      rows x cols of `dtype`; y may be x (then y_stride == x_stride).
 *   weight, bias  [cols] of `wdtype` (that of x, or SPOPT_DTYPE_F32), either may
 *             be NULL: 1 and 0.
 *   mean, rstd    float [rows], what the backward pass takes; either may be NULL.
 * All sums are held in 32 bits; y is rounded once.  A row that holds a NaN or
 * an infinity gives NaN in that row alone; so may one whose centred squares
 * sum to more than float32 holds (values of about 1e18 and more).
 * Errors: SPOPT_EINVAL (NULL x or y with rows > 0, rows < 0, cols < 1, a stride
 * below cols, unknown or mismatched types, eps not finite and > 0 as a float). */
SPOPT_API int layer_norm_forward(const void* x, int64_t x_stride, int64_t rows, int64_t cols,
                                 int32_t dtype, const void* weight, const void* bias,
                                 int32_t wdtype, double eps, void* y, int64_t y_stride,
                                 float* mean, float* rstd, void* stream, uint32_t flags);

/* Bytes of device workspace layer_norm_backward needs. */
SPOPT_API int layer_norm_backward_workspace_size(int64_t rows, int64_t cols, size_t* bytes);

/* The gradients of layer_norm_forward, with xhat = (x - mean) * rstd and
 * z = dy * weight:
 *   dx = rstd * (z - sum(z) / cols - xhat * sum(z * xhat) / cols),
 *   dweight = sum over rows of dy * xhat, dbias = sum over rows of dy.
 *   dy, x, dx   rows x cols of `dtype`, each with its row stride; dx may be dy
 *               or x (then with the same stride), or NULL.
 *   mean, rstd  float [rows], as the forward pass wrote them.
 *   weight      [cols] of `wdtype` or NULL.
 *   dweight, dbias  [cols] of `wdtype`, either may be NULL.  Written, not added
 *               to; all zero for rows == 0.
 * The sums over rows are formed in 32 bits in a fixed order, over slices of the
 * rows where they are many, which are joined in 64.
 * Workspace: device, 16-byte aligned, layer_norm_backward_workspace_size bytes.
 * Errors: as layer_norm_forward, and SPOPT_EWORKSPACE. */
SPOPT_API int layer_norm_backward(const void* dy, int64_t dy_stride, const void* x,
                                  int64_t x_stride, int64_t rows, int64_t cols, int32_t dtype,
                                  const float* mean, const float* rstd, const void* weight,
                                  int32_t wdtype, void* dx, int64_t dx_stride, void* dweight,
                                  void* dbias, void* workspace, size_t workspace_bytes,
                                  void* stream, uint32_t flags);

/* ---- orthogonalised updates ---------------------------------------------- */

/* The Newton-Schulz iteration on a matrix U (m x n, r = min(m, n)):
 *   X0 = U / (|U| + eps), |U| its Frobenius norm;
 *   `steps` times: X <- coef[0] X + (coef[1] A + coef[2] A A) X, A = X X^T
 * (X transposed where m > n, so that A is r x r).  Each step takes every
 * singular value s of X to coef[0] s + coef[1] s^3 + coef[2] s^5 and leaves
 * the singular vectors, so the result is near the orthogonal factor of U.
 * The products are taken in float16 with float32 sums, on matrix cores, for
 * float32 gradients too: X with 2^6 and A with 2^12 in front, which keeps them
 * inside float16's range.  X itself is carried from step to step in float32, as
 * is the diagonal of coef[1] A + coef[2] A A.
 * Accuracy, as the norm of the difference from the iteration in 64 bits over
 * the result's norm, before the rounding to bfloat16, for 5 steps of 3.4445,
 * -4.7750, 2.0315: below 4e-3 where U's shorter side is 8 or more and its
 * values are unlike (Gaussian, of low rank, with few rows that are not zero:
 * 3e-4 to 2.5e-3), below 1e-2 for any U (the largest: 2 or 3 rows, constant
 * matrices).  Directions that U lacks hold what rounding puts there, times
 * coef[0] for each later step: for U of low rank the result is within 5e-3 by 8
 * steps, off by up to 2e-2 by 10, and by as much as its own norm from 14 on; of
 * full rank by up to 2e-2 by 16 and 4e-2 by 64.  Coefficients that converge
 * (coef[0] of 2 and less) leave it within 3e-3 of any of these by 16 steps.
 * The scaling holds for singular values up to 2 and |coef[1] s^2 + coef[2] s^4|
 * up to 8; coefficients that leave these bounds in any of the steps are refused
 * (on the host, from the largest value that [0, 1] reaches).
 *   steps in [1, 64], coef finite, eps finite and > 0. */
typedef struct spopt_ns_config {
    double coef[3];
    double eps;
    int32_t steps;
} spopt_ns_config;

/* Bytes of device workspace newton_schulz and muon_step need for `batch`
 * matrices of m x n.  SPOPT_EINVAL for batch < 0, m or n < 1, m or n > 2^20 or
 * sizes beyond 2^40 values. */
SPOPT_API int newton_schulz_workspace_size(int64_t batch, int64_t m, int64_t n, size_t* bytes);

/* out = the iteration's result for each of `batch` matrices.
 *   g     batch x m x n of `dtype` (SPOPT_DTYPE_F32 or SPOPT_DTYPE_BF16),
 *         contiguous; read only.
 *   out   batch x m x n, bfloat16; must not overlap g or the workspace.
 * A zero matrix gives zeros.  Norms are summed in 64 bits.  A matrix that
 * holds a NaN or an infinity has an unspecified result; the others of the
 * batch are not affected.
 * Workspace: device, 16-byte aligned, newton_schulz_workspace_size bytes.
 * Errors: SPOPT_EINVAL (NULL, sizes, types, configuration), SPOPT_EWORKSPACE. */
SPOPT_API int newton_schulz(const void* g, int32_t dtype, int64_t batch, int64_t m, int64_t n,
                            const spopt_ns_config* config, void* out, void* workspace,
                            size_t workspace_bytes, void* stream, uint32_t flags);

/* Muon: momentum, orthogonalisation and the update of a weight matrix.
 *   buf <- momentum * buf + g
 *   u    = g + momentum * buf (nesterov), or buf
 *   p   <- (1 - lr * weight_decay) * p - lr * scale * newton_schulz(u)
 * lr >= 0, momentum in [0, 1), weight_decay >= 0, scale finite.  momentum == 0
 * takes u = g and no buf. */
typedef struct spopt_muon_config {
    double lr, momentum, weight_decay, scale;
    int32_t nesterov;
    spopt_ns_config ns;
} spopt_muon_config;

/* One Muon step of `batch` matrices of m x n, contiguous.
 *   params  of `pdtype` (SPOPT_DTYPE_F32 or SPOPT_DTYPE_BF16), updated in
 *           place; the update is formed in 32 bits and rounded once.
 *   buf     float, updated in place; NULL only for momentum == 0 (then unread).
 *   g       of `gdtype` (SPOPT_DTYPE_F32 or SPOPT_DTYPE_BF16), read only.
 * None of them may overlap another or the workspace.  The configuration is
 * read at the call: a captured call replays the values it was captured with.
 * Errors: as newton_schulz. */
SPOPT_API int muon_step(void* params, int32_t pdtype, float* buf, const void* g, int32_t gdtype,
                        int64_t batch, int64_t m, int64_t n, const spopt_muon_config* config,
                        void* workspace, size_t workspace_bytes, void* stream, uint32_t flags);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_OPS_H */
