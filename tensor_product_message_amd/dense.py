"""Torch-facing binding of the dense operators (include/convtp_dense.h): linear
layers with bias, activation and residual, the gated feed-forward form, and
the orthogonalisation of an optimiser's updates.  As in train.py the functions
here name the arguments and wrap autograd; csrc/dense_binding.cpp checks
metadata, takes outputs and workspaces from torch's allocator and calls the
library on the current HIP stream.

Types: float32, bfloat16, float16, the same for all tensors of a call; products
are summed in 32 bits and every output rounded once.  What a backward pass
multiplies, grad act'(z), is rounded to that type first (in float16 it has
float16's range: beyond 65504 an infinity); the biases' gradients sum it before
that.  Rows of x, residual and grad may lie any stride apart; w, bias and z are
contiguous.

Activations: "none", "relu", "silu", "gelu" (z Phi(z)), "sigmoid", "tanh".

Shapes (lmax > 0: D = (lmax + 1)^2 components a row, one matrix a degree, no activation):
    x, d_x                  : [..., inner], or [..., D, inner]
    y, z, residual, grad    : [..., outer], or [..., D, outer]
    w                       : [outer, inner], or [lmax + 1, outer, inner]
    bias                    : [outer], for lmax > 0 of component 0
Gated: w [2, outer, inner], bias [2, outer], z [..., 2, outer].
"""
from __future__ import annotations

import torch
from torch.autograd import forward_ad

from ._capi import dense_native

ACTIVATIONS = {"none": 0, "relu": 1, "silu": 2, "gelu": 3, "sigmoid": 4, "tanh": 5}


def _code(act: str) -> int:
    code = ACTIVATIONS.get(act)
    if code is None:
        raise ValueError(f"act must be one of {', '.join(ACTIVATIONS)}, got {act!r}")
    return code


# ---------------------------------------------------------------- linear layers


def linear_fwd(x, w, bias=None, residual=None, act: str = "none", lmax: int = 0, keep_z: bool = False, out=None):
    """(y, z) with z = x w^T + bias and y = act(z) + residual; z is None unless keep_z (a backward pass through an
    activation takes it).  out: y to write into, which may be residual, but must not overlap x or w."""
    return dense_native().linear_fwd(x, w, bias, residual, _code(act), lmax, False, keep_z, out)


def linear_bwd(grad, x, w, z=None, act: str = "none", lmax: int = 0, needs=(True, True, True), workspace=None):
    """Gradients (d_x, d_w, d_bias) of linear_fwd for grad (of y; it is the residual's too), None where `needs` has a
    false value.  z: the forward's, where there is an activation.  workspace: any device tensor of enough bytes,
    allocated here if None."""
    need_x, need_w, need_bias = needs
    return dense_native().linear_bwd(grad, x, w, z, _code(act), lmax, False, need_x, need_w, need_bias, workspace)


def linear_bwd_bwd(a_d_x, grad, x, w, z=None, act: str = "none", lmax: int = 0, needs=(True, True, True, True),
                   workspace=None):
    """Gradients (g_grad, g_x, g_w, g_bias) of <a_d_x, d_x> with linear_bwd's d_x, in grad, x, w and bias, z counting as
    the function of them that it is.  None where `needs` has a false value, and for g_x and g_bias without an
    activation (zero)."""
    return _second(a_d_x, grad, x, w, z, act, lmax, False, needs, workspace)


def _second(a_d_x, grad, x, w, z, act, lmax, gated, needs, workspace):
    need_grad, need_x, need_w, need_bias = needs
    code = _code(act)
    curved = gated or code != 0
    return dense_native().linear_bwd_bwd(a_d_x, grad, x, w, z, code, lmax, gated, need_grad, need_x and curved, need_w,
                                         need_bias and curved, workspace)


# ---------------------------------------------------------------- gated feed-forward


def gated_linear_fwd(x, w, bias=None, act: str = "silu", keep_z: bool = False, out=None):
    """(h, z) with z[h] = x w[h]^T + bias[h], h = 0, 1, and h = act(z[0]) z[1]; z is None unless keep_z."""
    return dense_native().linear_fwd(x, w, bias, None, _code(act), 0, True, keep_z, out)


def gated_linear_bwd(grad, x, w, z, act: str = "silu", needs=(True, True, True), workspace=None):
    """Gradients (d_x, d_w, d_bias) of gated_linear_fwd for grad (of h) and its z, as linear_bwd."""
    need_x, need_w, need_bias = needs
    return dense_native().linear_bwd(grad, x, w, z, _code(act), 0, True, need_x, need_w, need_bias, workspace)


def gated_linear_bwd_bwd(a_d_x, grad, x, w, z, act: str = "silu", needs=(True, True, True, True), workspace=None):
    """Gradients (g_grad, g_x, g_w, g_bias) of <a_d_x, d_x> with gated_linear_bwd's d_x, as linear_bwd_bwd."""
    return _second(a_d_x, grad, x, w, z, act, 0, True, needs, workspace)


# ---------------------------------------------------------------- autograd


class LinearFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, bias, residual, act, lmax, gated):
        curved = gated or act != "none"
        keep_z = curved and any(ctx.needs_input_grad[:3])
        y, z = dense_native().linear_fwd(x, w, bias, residual, _code(act), lmax, gated, keep_z, None)
        ctx.save_for_backward(x, w, bias, z)
        ctx.act, ctx.lmax, ctx.gated = act, lmax, gated
        ctx.set_materialize_grads(False)
        return y

    @staticmethod
    def backward(ctx, grad):
        if grad is None:
            return (None,) * 7
        x, w, bias, z = ctx.saved_tensors
        need_x, need_w, need_bias, need_residual = ctx.needs_input_grad[:4]
        d_x = d_w = d_bias = None
        if need_x or need_w or need_bias:
            d_x, d_w, d_bias = LinearBackward.apply(grad.contiguous(), x, w, bias, z, ctx.act, ctx.lmax, ctx.gated,
                                                    (need_x, need_w, need_bias))
        return d_x, d_w, d_bias, grad if need_residual else None, None, None, None


class LinearBackward(torch.autograd.Function):
    """The VJP of a linear layer as a function of its own inputs, differentiable once more in d_x (a loss on forces);
    the parameters' gradients are not differentiated."""

    @staticmethod
    def forward(ctx, grad, x, w, bias, z, act, lmax, gated, needs):
        ctx.save_for_backward(grad, x, w, z)
        ctx.act, ctx.lmax, ctx.gated = act, lmax, gated
        ctx.set_materialize_grads(False)
        return dense_native().linear_bwd(grad, x, w, z, _code(act), lmax, gated, *needs, None)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, a_d_x, *a_params):
        if any(a is not None for a in a_params):
            raise NotImplementedError("linear: the gradients of its parameters cannot be differentiated again")
        if a_d_x is None:
            return (None,) * 9
        grad, x, w, z = ctx.saved_tensors
        return (*_second(a_d_x.contiguous(), grad, x, w, z, ctx.act, ctx.lmax, ctx.gated, ctx.needs_input_grad[:4], None),
                None, None, None, None, None)


def _no_derivatives() -> bool:
    """Whether no derivative can be asked of a call, so that it may go past autograd: a level of forward mode works
    without grad mode too (autograd refuses it: there is no forward-mode formula)."""
    return not torch.is_grad_enabled() and getattr(forward_ad, "_current_level", 0) < 0


def linear(x, w, bias=None, residual=None, act: str = "none", lmax: int = 0):
    """Differentiable linear_fwd: act(x w^T + bias) + residual (twice in x, as a loss on forces needs it; not in
    forward mode)."""
    if _no_derivatives():
        return linear_fwd(x, w, bias, residual, act, int(lmax))[0]
    return LinearFunction.apply(x, w, bias, residual, act, int(lmax), False)


def gated_linear(x, w, bias=None, act: str = "silu"):
    """Differentiable gated_linear_fwd: act(x w[0]^T + bias[0]) (x w[1]^T + bias[1]) (twice in x;
    not in forward mode)."""
    if _no_derivatives():
        return gated_linear_fwd(x, w, bias, act)[0]
    return LinearFunction.apply(x, w, bias, None, act, 0, True)


# ---------------------------------------------------------------- orthogonalising


def orthogonalise(tensors, steps: int = 5, eps: float = 1e-7, scale: float = 1.0, out=None, workspace=None):
    """Every matrix [..., rows, cols] of `tensors` with its singular values brought near 1 (0.7 .. 1.2) by `steps`
    Newton-Schulz steps, times scale: X = M / (|M| + eps), X <- a X + (b A + c A A) X with A = X X^T.  out: the tensors
    to write, shapes and types like `tensors`; `tensors` itself works in place; new ones if None.  Returns out.  Not
    differentiable.  A matrix's result does not depend on the others of the list, to the last bit."""
    tensors = list(tensors)
    out = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in tensors] if out is None else list(out)
    dense_native().orthogonalise(tensors, out, steps, eps, scale, workspace)
    return out
