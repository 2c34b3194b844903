"""Torch-facing binding of the training-step operators (include/convtp_train.h):
embedding lookup and gradient, norms fused with a block's gate and residual,
gradient clipping by the global norm.  The functions here name the arguments
and wrap autograd; csrc/train_binding.cpp checks tensors' metadata, takes
outputs and workspaces from torch's allocator and calls the library on the
current HIP stream.

Types: float32, bfloat16, float16; every sum is formed in 32 bits or more and
every output rounded once.  A tensor's rows may lie any stride apart (a slice
of a wider tensor), but within a row values are contiguous.  Wrong metadata
raises TypeError or ValueError, what the library refuses ConvTPError.  A
tensor given to write into counts as modified in place: a backward pass that
saved it raises.

Shapes (lmax = 0: plain rows; else D = (lmax + 1)^2 components a row):
    h, r, grad_r, grad_u, d_h, d_r  : [..., C], or [..., D, C]
    w_post, w_pre, gate of channels : [C], or [lmax + 1, C]
    gate of rows                    : [..., C], or [..., lmax + 1, C]; in the features' type
"""
from __future__ import annotations

import torch

from ._capi import native

# ---------------------------------------------------------------- embedding


def embed_fwd(table, tokens, scale: float = 1.0, out=None):
    """out[..., C] = scale * table[tokens]; a token outside the table is padding and gives a zero row."""
    return native().embed_fwd(table, tokens, scale, out)


def embed_bwd(grad_out, tokens, n_rows: int, scale: float = 1.0, out=None, dtype=None, workspace=None):
    """d_table[n_rows, C]: row v is scale times the sum of grad_out's rows whose token is v, zeros where there is
    none.  dtype: grad_out's, or float32.  workspace: any device tensor of enough bytes, allocated here if None."""
    return native().embed_bwd(grad_out, tokens, n_rows, scale, out, dtype, workspace)


class EmbedFunction(torch.autograd.Function):
    """Autograd of embed_fwd; linear in the table, so its gradient's own gradient is a lookup again."""

    @staticmethod
    def forward(ctx, table, tokens, scale):
        ctx.save_for_backward(tokens)
        ctx.n_rows, ctx.scale = table.shape[0], scale
        return embed_fwd(table, tokens, scale)

    @staticmethod
    def backward(ctx, grad_out):
        tokens, = ctx.saved_tensors
        return EmbedBackward.apply(grad_out.contiguous(), tokens, ctx.n_rows, ctx.scale), None, None


class EmbedBackward(torch.autograd.Function):
    @staticmethod
    def forward(ctx, grad_out, tokens, n_rows, scale):
        ctx.save_for_backward(tokens)
        ctx.scale = scale
        return embed_bwd(grad_out, tokens, n_rows, scale)

    @staticmethod
    def backward(ctx, a_table):
        tokens, = ctx.saved_tensors
        return EmbedFunction.apply(a_table.contiguous(), tokens, ctx.scale), None, None, None


def embed(table, tokens, scale: float = 1.0):
    """Differentiable embed_fwd (any number of times, in the table)."""
    return EmbedFunction.apply(table, tokens.contiguous(), float(scale))


# ---------------------------------------------------------------- norms


def norm_residual_fwd(h, r, w_post, w_pre, gate=None, alpha: float = 1.0, eps: float = 1e-6, lmax: int = 0, out=None):
    """(r', u) with r' = r + alpha * gate * N(h; w_post) and u = N(r'; w_pre), N the root-mean-square norm over a
    row (balanced over the degrees for lmax > 0; see include/convtp_train.h).  h None: u = N(r; w_pre) alone, r'
    is r itself.  w_post None: h is added without a norm.  w_pre None: u is None.  gate: one row, or one for every
    row.  out: (r', u) to write into, None for a new one; r' may be r.  What is not computed is not written: r'
    without h, u without w_pre."""
    r_out, u = (None, None) if out is None else out
    return native().norm_fwd(h, r, w_post, w_pre, gate, alpha, eps, lmax, r_out, u)


def norm_residual_bwd(grad_r, grad_u, h, r_out, w_post, w_pre, gate=None, alpha: float = 1.0, eps: float = 1e-6,
                      lmax: int = 0, workspace=None):
    """Gradients (d_h, d_r, d_w_post, d_w_pre, d_gate) of norm_residual_fwd for grad_r (of r') and grad_u (of u),
    either of which may be None (zero); r_out is the forward's r'.  None in the place of what is absent."""
    return native().norm_bwd(grad_r, grad_u, h, r_out, w_post, w_pre, gate, alpha, eps, lmax, workspace)


def norm_residual_bwd_bwd(a_d_h, a_d_r, grad_r, grad_u, h, r_out, w_post, w_pre, gate=None, alpha: float = 1.0,
                          eps: float = 1e-6, lmax: int = 0, workspace=None):
    """Gradients (g_grad_r, g_grad_u, g_h, g_r_out, g_w_post, g_w_pre, g_gate) of <a_d_h, d_h> + <a_d_r, d_r> with
    norm_residual_bwd's d_h and d_r, in its inputs; a_d_h or a_d_r may be None (zero).  None in the place of what
    is absent."""
    return native().norm_bwd_bwd(a_d_h, a_d_r, grad_r, grad_u, h, r_out, w_post, w_pre, gate, alpha, eps, lmax,
                                 workspace)


class NormResidualFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, r, w_post, w_pre, gate, alpha, eps, lmax):
        r_out, u = norm_residual_fwd(h, r, w_post, w_pre, gate, alpha, eps, lmax)
        ctx.save_for_backward(h, r_out if w_pre is not None else None, w_post, w_pre, gate)
        ctx.alpha, ctx.eps, ctx.lmax = alpha, eps, lmax
        ctx.set_materialize_grads(False)
        return (r_out.view_as(r_out) if h is None else r_out), u

    @staticmethod
    def backward(ctx, grad_r, grad_u):
        h, r_out, w_post, w_pre, gate = ctx.saved_tensors
        if grad_r is None and grad_u is None:
            return (None,) * 8
        grad_r, grad_u = (None if g is None else g.contiguous() for g in (grad_r, grad_u))
        return (*NormResidualBackward.apply(grad_r, grad_u, h, r_out, w_post, w_pre, gate, ctx.alpha, ctx.eps,
                                            ctx.lmax), None, None, None)


class NormResidualBackward(torch.autograd.Function):
    """The VJP of norm_residual as a function of its own inputs, differentiable once more in the features' gradients
    (a loss on forces); the parameters' gradients are not differentiated."""

    @staticmethod
    def forward(ctx, grad_r, grad_u, h, r_out, w_post, w_pre, gate, alpha, eps, lmax):
        ctx.save_for_backward(grad_r, grad_u, h, r_out, w_post, w_pre, gate)
        ctx.alpha, ctx.eps, ctx.lmax = alpha, eps, lmax
        ctx.set_materialize_grads(False)
        return norm_residual_bwd(grad_r, grad_u, h, r_out, w_post, w_pre, gate, alpha, eps, lmax)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, a_d_h, a_d_r, *a_params):
        if any(a is not None for a in a_params):
            raise NotImplementedError("norm_residual: the gradients of its parameters cannot be differentiated again")
        if a_d_h is None and a_d_r is None:
            return (None,) * 10
        a_d_h, a_d_r = (None if a is None else a.contiguous() for a in (a_d_h, a_d_r))
        return (*norm_residual_bwd_bwd(a_d_h, a_d_r, *ctx.saved_tensors, ctx.alpha, ctx.eps, ctx.lmax), None, None,
                None)


def norm_residual(h, r, w_post, w_pre, gate=None, alpha: float = 1.0, eps: float = 1e-6, lmax: int = 0):
    """Differentiable norm_residual_fwd (twice in the features, as a loss on forces needs it)."""
    return NormResidualFunction.apply(h, r, w_post, w_pre, gate, float(alpha), float(eps), int(lmax))


# ---------------------------------------------------------------- clipping


def grad_norm(tensors, out=None):
    """The 2-norm of all elements of `tensors` together, a float32 value on their device."""
    return native().clip(list(tensors), None, 0.0, 0.0, out)


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6, out=None):
    """(out, norm): every tensor times min(1, max_norm / (norm + eps)) with the global norm of all of them.
    out: the tensors to write, sizes and types like `tensors`; `tensors` itself clips in place; new ones if None.
    Nothing waits for the GPU."""
    tensors = list(tensors)
    out = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in tensors] if out is None else list(out)
    return out, native().clip(tensors, out, max_norm, eps, None)
