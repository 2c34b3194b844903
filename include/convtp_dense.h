/*
 * convtp_dense.h - C ABI of the dense operators around the convolution
 *                  (MI355X / gfx950), in the same library as convtp.h:
 *                  linear layers with bias, activation and residual, the
 *                  gated feed-forward form, their first and second gradients,
 *                  and the orthogonalisation of an optimiser's updates.
 *
 * Conventions are convtp_train.h's: device pointers unless marked host, the
 * caller owns every buffer, outputs are overwritten, every call enqueues its
 * kernels on `stream` and returns, arguments are checked on the host before
 * any HIP call, nothing is allocated, copied or set by the runtime, so the
 * calls can be captured in a graph (a workspace belongs to one call at a time:
 * graphs that may run at once need one each).  Rows may begin at any address
 * that suits their elements.  Results are bitwise reproducible.
 *
 * Products are summed in fp32.  Operands of 16 bits enter the matrix cores as
 * they are; floats enter as three bfloat16 parts, which gives a float product's
 * accuracy; results that come out not finite are formed once more of the floats
 * themselves, so infinities, NaN and what passes float's range are a float
 * product's.
 *
 * What a gradient multiplies - grad act'(z), and the second pass's factors - is
 * rounded to the features' type first, as a stored z is.  In float16 that has
 * float16's range: grad act'(z), in the gated form grad z[1] act'(z[0]) and
 * grad act(z[0]), beyond 65504 is an infinity although the gradient itself may
 * be finite, and below 2^-24 it is zero.  Scale the loss to suit.  The biases'
 * gradients sum these values in fp32 before that rounding.
 */
#ifndef CONVTP_DENSE_H
#define CONVTP_DENSE_H

#include <stdint.h>

#include "convtp_train.h"

#ifdef __cplusplus
extern "C" {
#endif

/* gelu is z Phi(z) with the normal distribution Phi; silu is z sigmoid(z). */
enum conv_tp_act { CTP_ACT_NONE = 0, CTP_ACT_RELU = 1, CTP_ACT_SILU = 2, CTP_ACT_GELU = 3, CTP_ACT_SIGMOID = 4, CTP_ACT_TANH = 5 };

/* ---------------------------------------------------------------------------
 * Linear layers.  A row of x is [D][inner], of y [D][outer], D = (lmax + 1)^2
 * components of the degrees 0..lmax (lmax = 0: plain rows); w is
 * [lmax + 1][outer][inner], one matrix a degree, so the layer commutes with
 * rotations; bias [outer] is added to component 0.
 *
 *   gated = 0:  z = x w^T + bias,  y = act(z) + residual      (lmax > 0: no act)
 *   gated = 1:  z[h] = x w[h]^T + bias[h], h = 0, 1,  y = act(z[0]) z[1]
 *               (lmax = 0; w [2][outer][inner], bias [2][outer], z [rows][2][outer], no residual)
 *
 * bias, residual: NULL for none.  z: written for a backward pass, NULL if not
 * wanted; y is formed from z before its rounding. */
typedef struct conv_tp_linear_problem {
    int64_t n_rows;           /* 0 .. 2^31 - 1 */
    int64_t x_stride;         /* elements from row to row of each input, >= its row; outputs and z are dense */
    int64_t residual_stride;
    int64_t grad_stride;
    int32_t lmax;             /* 0 .. 3 */
    int32_t inner, outer;     /* 1 .. 2^20, D times either at most 2^20 */
    int32_t dtype;            /* conv_tp_dtype of every array */
    int32_t act;              /* conv_tp_act */
    int32_t gated;            /* 0 or 1 */
} conv_tp_linear_problem;

/* workspace here and below: 16-byte aligned, at least the bytes that the call of the same name with _workspace gives
 * for the same problem, its strides included (0: may be NULL); contents undefined afterwards. */
int32_t conv_tp_linear_fwd(const conv_tp_linear_problem *prob, const void *x, const void *w, const void *bias,
                           const void *residual, void *y, void *z, void *workspace, int64_t workspace_bytes,
                           void *stream);
int32_t conv_tp_linear_fwd_workspace(const conv_tp_linear_problem *prob, int64_t *bytes);

/* Gradients for grad = dL/dy (the residual's is grad itself), each NULL if not
 * wanted: d_x, d_w, d_bias.  z: the forward's, not read (may be NULL) with
 * CTP_ACT_NONE and gated = 0. */
int32_t conv_tp_linear_bwd(const conv_tp_linear_problem *prob, const void *grad, const void *x, const void *w,
                           const void *z, void *d_x, void *d_w, void *d_bias, void *workspace,
                           int64_t workspace_bytes, void *stream);
int32_t conv_tp_linear_bwd_workspace(const conv_tp_linear_problem *prob, int64_t *bytes);

/* The second backward pass, for losses on first gradients (training on
 * forces): with a cotangent a_d_x of conv_tp_linear_bwd's d_x (dense), the
 * gradients of <a_d_x, d_x> in grad, x, w and bias, each NULL if not wanted;
 * z counts as the function of x, w and bias that it is.  With CTP_ACT_NONE and
 * gated = 0 those in x and bias are zero: g_x and g_bias have to be NULL. */
int32_t conv_tp_linear_bwd_bwd(const conv_tp_linear_problem *prob, const void *a_d_x, const void *grad, const void *x,
                               const void *w, const void *z, void *g_grad, void *g_x, void *g_w, void *g_bias,
                               void *workspace, int64_t workspace_bytes, void *stream);
int32_t conv_tp_linear_bwd_bwd_workspace(const conv_tp_linear_problem *prob, int64_t *bytes);

/* ---------------------------------------------------------------------------
 * Orthogonalising matrices: X = M / (|M| + eps) with the root of the sum of
 * squares, then `steps` times X <- a X + (b A + c A A) X, A = X X^T, with
 * a, b, c = 3.4445, -4.7750, 2.0315 (for tall matrices the same of M^T), and
 * out = scale X: singular values between some 0.003 and 1 of |M| come out
 * between 0.7 and 1.2 times scale, the singular vectors stay.  (The
 * coefficients are the ones published with the Muon optimiser, K. Jordan 2024.)
 *
 * Tensor k holds batch[k] dense matrices [rows[k]][cols[k]], one after the
 * other, each orthogonalised by itself.  in, out (host arrays of device
 * pointers), batch, rows, cols, dtype: host arrays of n_tensors entries, read
 * before the call returns.  out[k] has in[k]'s type and may be in[k]; other
 * overlaps are not allowed.  X, A and b A + c A A are held in 32 bits whatever
 * the type (two float16, 22 significant bits), their products summed in fp32.  A
 * matrix of zeros gives zeros (eps > 0), one with a value that is not finite
 * gives NaN.  A matrix's result does not depend on the matrices beside it, to
 * the last bit. */
int32_t conv_tp_orthogonalise(int32_t n_tensors, const void *const *in, void *const *out, const int64_t *batch,
                              const int32_t *rows, const int32_t *cols, const int32_t *dtype, int32_t steps, float eps,
                              float scale, void *workspace, int64_t workspace_bytes, void *stream);
int32_t conv_tp_orthogonalise_workspace(int32_t n_tensors, const int64_t *batch, const int32_t *rows,
                                        const int32_t *cols, int64_t *bytes);

/* Message of the last non-zero status of a call of this header on this thread ("" if none). */
const char *conv_tp_dense_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* CONVTP_DENSE_H */
