/*
 * dense_ops.h - C ABI of the dense operators that stand between a table's
 * looked-up rows and the loss, and of the loss: layer norm and dropout (forward
 * and backward), the Newton-Schulz orthogonalisation of a matrix, the Muon step
 * that applies it to a weight, and the softmax cross entropy over a table of
 * classes (forward and backward).
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

/* ---- the loss over a table of classes ------------------------------------ */

#define SPOPT_REDUCE_NONE 0
#define SPOPT_REDUCE_SUM 1
#define SPOPT_REDUCE_MEAN 2

/* Softmax cross entropy of rows x cols hidden states against a table of
 * classes x cols, with z = x weight^T, e = label_smoothing and t = targets[i]:
 *   lse_i  = log(sum over j of exp(z_ij)),
 *   loss_i = lse_i - (1 - e) z_it - (e / classes) sum over j of z_ij.
 * The rows x classes logits are never stored.  Rows whose target is
 * ignore_index do not count: their loss and lse are 0, and what x holds there
 * reaches nothing.
 *   x         rows x cols of `dtype`, row k at x + k * x_stride.
 *   weight    classes x cols of `dtype`, with its row stride.
 *   targets   int64 [rows]; one that is neither a class nor ignore_index gives
 *             NaN for its loss (SPOPT_ERANGE under SPOPT_VALIDATE).
 *   loss      float: [rows] for SPOPT_REDUCE_NONE; one value, the sum over the
 *             rows that count or their mean, for SPOPT_REDUCE_SUM and _MEAN (0
 *             where no row counts).
 *   lse       float [rows], what the backward pass takes.
 * Types: 16-bit operands are multiplied as they are, with float32 sums, and so
 * are float32 ones in small calls.  In others (which is which goes by the sizes
 * alone) each value of a float32 operand is taken as two float16 after a power of
 * two that brings the operand's largest finite value (of x: in rows that count) to
 * 2^14: 22 bits, for values below 2^-18 of the largest an absolute 2^-39 of it.
 * The products of the two low parts are left out, sums are float32.  A NaN in x
 * makes its row NaN, in weight every row; an infinity does so too, or leaves an
 * infinite or a finite value where the formula does.
 * Workspace: device, 16-byte aligned, linear_cross_entropy_workspace_size bytes
 * for the pass (backward 0 or 1).  Small calls read their inputs in place.  In
 * others those with cols a multiple of 64, strides multiples of 8 and 16-byte
 * aligned bases are read in place where they are of 16 bits, and the rest (x
 * always in the backward pass, float16 and float32 with room for a second copy) are
 * copied into the workspace, the weight up to 256 MiB (or 2048 rows) at a time.
 * Errors: SPOPT_EINVAL (NULL, sizes, a stride below cols, types, reduction,
 * label_smoothing outside [0, 1]), SPOPT_EWORKSPACE; rows up to 2^27, cols to
 * 2^20, classes to 2^30, either matrix to 2^36 values.  SPOPT_VALIDATE reads
 * the targets, the rows of x that count, and weight. */
SPOPT_API int linear_cross_entropy_workspace_size(int64_t rows, int64_t cols, int64_t classes,
                                                  int32_t dtype, int32_t backward, size_t* bytes);

/* Which kernels a pass takes, which goes by its sizes and type alone: for tests of each
 * and for measurements of the rule. */
typedef struct spopt_ce_plan {
    int32_t direct;       /* 1: operands read in place by kernels for small calls; tiles below 16 or 64 */
    int32_t tile_logits;  /* rows of a tile of the logits, */
    int32_t tile_dx;      /* and (backward; else 0) of the two products: 64, 128 or 256 */
    int32_t tile_dw;
    int32_t splits_dx;    /* parts that their inner axes are cut into */
    int32_t splits_dw;
    int64_t piece;        /* classes at a time */
} spopt_ce_plan;

/* Errors: SPOPT_EINVAL (rows < 1, and as linear_cross_entropy_workspace_size). */
SPOPT_API int linear_cross_entropy_plan(int64_t rows, int64_t cols, int64_t classes, int32_t dtype,
                                        int32_t backward, spopt_ce_plan* plan);

SPOPT_API int linear_cross_entropy_forward(const void* x, int64_t x_stride, const void* weight,
                                           int64_t weight_stride, int64_t rows, int64_t cols,
                                           int64_t classes, int32_t dtype, const int64_t* targets,
                                           int64_t ignore_index, double label_smoothing,
                                           int32_t reduction, float* loss, float* lse,
                                           void* workspace, size_t workspace_bytes, void* stream,
                                           uint32_t flags);

/* The gradients of linear_cross_entropy_forward, with c_i = dloss[i], dloss[0]
 * or dloss[0] / (rows that count) by the reduction, 0 for rows that do not:
 *   g_ij = c_i (exp(z_ij - lse_i) - (1 - e) [j == t] - e / classes),
 *   dx = g weight, dweight = g^T x.
 *   dloss     float: [rows] for SPOPT_REDUCE_NONE, else one value.
 *   lse       float [rows], as the forward pass wrote it.
 *   dx        rows x cols of `dtype`, with its row stride, or NULL.  Rows that do
 *             not count get zeros.
 *   dweight   classes x cols of `dtype`, with its row stride, or NULL.  Written,
 *             not added to; all zero for rows == 0.
 * None of the outputs may overlap another, an input or the workspace.
 * In small calls g is float32, which the products of 16-bit types take as two values
 * of the type; in others it is rounded to the operands' type (float32: taken as two
 * float16, like the operands).  It has a factor in front that brings max |c_i| (1 - e)
 * to 2^13; under SPOPT_REDUCE_NONE each row in float16 or two has a power of two more,
 * to the same binade.  So g_ij is off by half a step of its type (two float16: 2^-22
 * of it, two bfloat16: 2^-16), and in float16 or two by 2^-38 |c_i| at least: a row
 * gives nothing to classes of less probability than that.  For dweight the powers are
 * taken back from x's rows, c_i x_i then being off by 2^-37 of the largest (small calls
 * have none there: g is off by 2^-38 of max |c_i| in two float16).  Sums are
 * float32, rounded once.  g exists for one piece of the classes at a time, of up
 * to 512 MiB (or 2048 classes).  A row whose target is
 * neither a class nor ignore_index makes its row of dx and all of dweight NaN.
 * Workspace, errors and validation as above. */
SPOPT_API int linear_cross_entropy_backward(
    const float* dloss, const void* x, int64_t x_stride, const void* weight, int64_t weight_stride,
    int64_t rows, int64_t cols, int64_t classes, int32_t dtype, const int64_t* targets,
    int64_t ignore_index, double label_smoothing, int32_t reduction, const float* lse, void* dx,
    int64_t dx_stride, void* dweight, int64_t dweight_stride, void* workspace,
    size_t workspace_bytes, void* stream, uint32_t flags);

/* ---- dropout ------------------------------------------------------------- */

/* Dropout whose mask is a function of (seed, offset, index) and is never
 * stored: with q = round(p * 2^16) and value i = row * cols + col,
 *   y_i = (bits_i >= q ? x_i * 2^16 / (2^16 - q) : 0) + residual_i,
 * bits_i the (i % 8)th 16 bits, from the lowest of the first word on, of
 * Philox4x32-10 (Salmon et al., "Parallel random numbers: as easy as 1, 2, 3",
 * 2011) at counter words (i / 8 low, i / 8 high, offset low, offset high) under
 * the key words (seed low, seed high).  So p counts in steps of 2^-16, and the
 * factor is that of the p taken: the mean of y is x.  Offsets give independent
 * masks under one seed (one for each layer and step).
 *   x, y      rows x cols of `dtype`, each with its row stride; y may be x or
 *             residual (then with the same stride).
 *   residual  rows x cols of `dtype` with its row stride, or NULL: 0.
 *   p         in [0, 1]; q == 2^16 drops every value.
 *   d_seed    device int64[1] or NULL.  Where given, the seed is read from it when
 *             the call's kernel runs, so that a captured call can be replayed
 *             with other masks; `seed` is not used.
 * Values that are dropped are not looked at: a NaN or an infinity there leaves
 * nothing.  y is formed in float32 and rounded once.  Rows and strides only
 * change where values lie, not which are dropped.
 * Errors: SPOPT_EINVAL (NULL x or y with rows > 0, rows < 0, cols < 1, a stride
 * below cols, unknown type, p outside [0, 1]). */
SPOPT_API int dropout_forward(const void* x, int64_t x_stride, const void* residual,
                              int64_t residual_stride, int64_t rows, int64_t cols, int32_t dtype,
                              double p, uint64_t seed, const int64_t* d_seed, uint64_t offset,
                              void* y, int64_t y_stride, void* stream, uint32_t flags);

/* The gradient: dx_i = bits_i >= q ? dy_i * 2^16 / (2^16 - q) : 0 (the residual's
 * is dy).  dx may be dy.  Otherwise as dropout_forward. */
SPOPT_API int dropout_backward(const void* dy, int64_t dy_stride, int64_t rows, int64_t cols,
                               int32_t dtype, double p, uint64_t seed, const int64_t* d_seed,
                               uint64_t offset, void* dx, int64_t dx_stride, void* stream,
                               uint32_t flags);

#ifdef __cplusplus
}
#endif

#endif /* DENSE_OPS_H */
