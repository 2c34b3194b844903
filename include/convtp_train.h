/*
 * convtp_train.h - C ABI of the operators of a training step around the
 *                  convolution (MI355X / gfx950), in the same library as
 *                  convtp.h: embedding lookup and its gradient, norms fused
 *                  with a block's gate and residual and their gradient, and
 *                  the clipping of gradients by their global norm.
 *
 * Conventions are convtp.h's where nothing else is said: array pointers are
 * DEVICE pointers unless marked host, the caller owns every buffer, outputs
 * are overwritten, `stream` is a hipStream_t, every call enqueues its kernels
 * and returns without synchronising, arguments are checked on the host before
 * any HIP call, statuses are convtp.h's CTP_* codes.  The calls allocate
 * nothing and record no copies or memsets: they can be captured in a graph
 * (the addresses that a capture saw are replayed).  They are launched on the
 * device that is current, which must be the stream's.
 *
 * Element types are conv_tp_dtype values.  Sums, statistics and products are
 * formed in 32 bits or more whatever the type, and every output value is
 * rounded once.  Rows may begin at any address that suits their elements
 * (CTP_EALIGN otherwise) and lie any stride apart that the arguments allow.
 * Results are bitwise reproducible: nothing is added with atomics.
 */
#ifndef CONVTP_TRAIN_H
#define CONVTP_TRAIN_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum conv_tp_dtype { CTP_F32 = 0, CTP_BF16 = 1, CTP_F16 = 2 };

/* ---------------------------------------------------------------------------
 * Embedding:  out[t, c] = scale * table[token[t], c]
 *
 * A token outside [0, n_rows) is padding: its row of out is zero, and it has
 * no share of the gradient.  (Tokens are checked on the device, so any content
 * is safe.) */
typedef struct conv_tp_embed_problem {
    int64_t n_tokens;     /* 0 .. 2^31 - 1 */
    int64_t n_rows;       /* rows of the table, 0 .. 2^31 - 2 */
    int64_t src_stride;   /* elements from row to row of table (forward) or grad_out (backward), >= channels */
    int64_t dst_stride;   /* of out (forward) or d_table (backward), >= channels */
    int32_t channels;     /* 1 .. 2^20 */
    int32_t dtype;        /* of table and out; of grad_out */
    int32_t out_dtype;    /* backward: of d_table, dtype or CTP_F32; forward: dtype */
    int32_t index_bits;   /* tokens are int32 (32) or int64 (64) */
    float scale;
} conv_tp_embed_problem;

int32_t conv_tp_embed_fwd(const conv_tp_embed_problem *prob, const void *table, const void *tokens, void *out,
                          void *stream);

/* d_table[v, c] = scale * sum over the t with token[t] = v of grad_out[t, c],
 * every row written (zeros where no token is).  Tokens are sorted and each
 * row's sum is formed in their order.  workspace: 16-byte aligned, at least
 * conv_tp_embed_bwd_workspace bytes, contents undefined afterwards. */
int32_t conv_tp_embed_bwd(const conv_tp_embed_problem *prob, const void *grad_out, const void *tokens, void *d_table,
                          void *workspace, int64_t workspace_bytes, void *stream);
int32_t conv_tp_embed_bwd_workspace(const conv_tp_embed_problem *prob, int64_t *bytes);

/* ---------------------------------------------------------------------------
 * Norms after and before a block, with the block's gate and the scaled
 * residual.  A row is [D][C], D = (lmax + 1)^2 components of the degrees
 * 0..lmax as in convtp.h (lmax = 0: a plain row of C values), and
 *
 *   N(x; w)[l m, c] = w[l, c] x[l m, c] s(x)
 *   s(x) = (eps + 1/((lmax+1) C) sum_{l,c} 1/(2l+1) sum_m x[l m, c]^2)^(-1/2)
 *
 * one s a row: it commutes with rotations, and for lmax = 0 it is the
 * root-mean-square norm.  Forward, for the block's output h and the residual r:
 *
 *   r' = r + alpha * gate * N(h; w_post)        u = N(r'; w_pre)
 *
 * u, the next block's input, is formed from r' before its rounding.
 *   h      NULL: there is no block (the first norm): r' is r, which is not written.
 *   w_post NULL: the block's output is not normalised (N(h) is h).
 *   w_pre  NULL: no u (after the last block).  h and w_pre are not both NULL.
 *   gate   0: none; 1: gate[l, c]; 2: gate[row, l, c] (in `dtype`). */
typedef struct conv_tp_norm_problem {
    int64_t n_rows;       /* 0 .. 2^31 - 1 */
    int64_t h_stride;     /* elements from row to row of each input, >= its row; outputs are dense */
    int64_t r_stride;
    int64_t gate_stride;
    int64_t grad_r_stride;
    int64_t grad_u_stride;
    int32_t lmax;         /* 0 .. 3 */
    int32_t channels;     /* >= 1, D * channels <= 16384 */
    int32_t dtype;        /* of h, r, r', u, their gradients and a gate of every row */
    int32_t param_dtype;  /* of w_post, w_pre, gate[l, c] and their gradients: dtype or CTP_F32 */
    int32_t gate;
    float alpha, eps;     /* eps >= 0 */
} conv_tp_norm_problem;

int32_t conv_tp_norm_fwd(const conv_tp_norm_problem *prob, const void *h, const void *r, const void *w_post,
                         const void *w_pre, const void *gate, void *r_out, void *u, void *stream);

/* Gradients for grad_r = dL/dr' and grad_u = dL/du; either may be NULL: zero.
 * r_out is the forward's r' (r itself where h is NULL); not read, and may be
 * NULL, without w_pre.  Written: d_r always, d_h with h, d_w_post, d_w_pre and
 * d_gate with their parameters; pointers of what is absent are ignored.
 * workspace: 16-byte aligned, at least conv_tp_norm_bwd_workspace bytes. */
int32_t conv_tp_norm_bwd(const conv_tp_norm_problem *prob, const void *grad_r, const void *grad_u, const void *h,
                         const void *r_out, const void *w_post, const void *w_pre, const void *gate, void *d_h,
                         void *d_r, void *d_w_post, void *d_w_pre, void *d_gate, void *workspace,
                         int64_t workspace_bytes, void *stream);
int32_t conv_tp_norm_bwd_workspace(const conv_tp_norm_problem *prob, int64_t *bytes);

/* The second backward pass, for losses on first gradients (training on
 * forces): with cotangents a_d_h and a_d_r of conv_tp_norm_bwd's d_h and d_r
 * (dense; one may be NULL: zero), the gradients of <a_d_h, d_h> + <a_d_r, d_r>
 * in that call's inputs: g_grad_r, g_grad_u (NULL: not wanted), g_h (with h),
 * g_r (in r_out, with w_pre) and g_w_post, g_w_pre, g_gate with their
 * parameters.  All outputs are dense.  The parameters' first gradients have
 * no cotangents here.  workspace as for conv_tp_norm_bwd. */
int32_t conv_tp_norm_bwd_bwd(const conv_tp_norm_problem *prob, const void *a_d_h, const void *a_d_r, const void *grad_r,
                             const void *grad_u, const void *h, const void *r_out, const void *w_post,
                             const void *w_pre, const void *gate, void *g_grad_r, void *g_grad_u, void *g_h, void *g_r,
                             void *g_w_post, void *g_w_pre, void *g_gate, void *workspace, int64_t workspace_bytes,
                             void *stream);

/* ---------------------------------------------------------------------------
 * Clipping by the global norm of n_tensors dense tensors:
 *
 *   norm = sqrt(sum over all elements of g^2),  out = g * min(1, max_norm / (norm + eps))
 *
 * in, out (host arrays of device pointers), numel, dtype: host arrays of
 * n_tensors entries, read before the call returns.  out NULL: the norm alone.
 * out[k] may be in[k] (in place; where nothing is clipped it is not rewritten)
 * and has in[k]'s type; other overlaps are not allowed.  norm: device, one
 * float.  Squares are summed in 64 bits, and out is the formula's also where the
 * norm leaves a float's range (it is then reported as infinity) or the factor
 * does.  A norm that is not finite gives what the formula gives.  workspace:
 * 16-byte aligned, at least conv_tp_clip_workspace(n_tensors) bytes. */
int32_t conv_tp_clip(int32_t n_tensors, const void *const *in, void *const *out, const int64_t *numel,
                     const int32_t *dtype, float max_norm, float eps, float *norm, void *workspace,
                     int64_t workspace_bytes, void *stream);
int64_t conv_tp_clip_workspace(int32_t n_tensors);

/* Message of the last non-zero status of a call of this header on this thread ("" if none). */
const char *conv_tp_train_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* CONVTP_TRAIN_H */
