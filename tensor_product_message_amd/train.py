"""Torch-facing binding of the training-step operators (include/convtp_train.h):
embedding lookup and gradient, norms fused with a block's gate and residual,
gradient clipping by the global norm.  As in `ops`, only argument marshalling:
metadata checks, raw pointers, the current HIP stream, workspaces from torch's
allocator.

Types: float32, bfloat16, float16; every sum is formed in 32 bits or more and
every output rounded once.  A tensor's rows may lie any stride apart (a slice
of a wider tensor), but within a row values are contiguous.

Shapes (lmax = 0: plain rows; else D = (lmax + 1)^2 components a row):
    h, r, grad_r, grad_u, d_h, d_r  : [..., C], or [..., D, C]
    w_post, w_pre, gate of channels : [C], or [lmax + 1, C]
    gate of rows                    : [..., C], or [..., lmax + 1, C]
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from ._capi import EmbedProblem, NormProblem, train_check, train_lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_INDEX_BITS = {torch.int32: 32, torch.int64: 64}


def _float_code(t, name):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    code = _DTYPES.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    return code


def _on(t, name, device):
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _hip_device(t, name):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    return t.device


def _rows(t, name, tail, dtype, device, rows=None):
    """(rows, stride) of a tensor [..., *tail] as rows of dense tails."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    _on(t, name, device)
    k = t.dim() - len(tail)
    if k < 0 or tuple(t.shape[k:]) != tail:
        raise ValueError(f"{name} must have shape [..., {', '.join(map(str, tail))}], got {tuple(t.shape)}")
    width = 1
    for v in tail:
        width *= v
    n = t.numel() // width if width else 0
    if rows is not None and n != rows:
        raise ValueError(f"{name} has {n} rows, expected {rows}")
    if t.is_contiguous():
        return n, width
    if k == 1 and n <= 1 or k == 0:
        inner, stride = t, width
    elif k == 1 and t.stride(0) >= width:
        inner, stride = t[0], t.stride(0)
    else:
        raise ValueError(f"{name}: its rows must lie one stride apart (strides {t.stride()})")
    if not inner.is_contiguous() and n > 0:
        raise ValueError(f"{name}: a row must be contiguous (strides {t.stride()})")
    return n, stride


class _OnDevice:
    """Makes a tensor's device current around a launch where it is not."""
    __slots__ = ("index", "before")

    def __init__(self, device):
        self.index = device.index

    def __enter__(self):
        self.before = torch.cuda.current_device()
        if self.before != self.index:
            torch.cuda.set_device(self.index)
        return torch.cuda.current_stream().cuda_stream

    def __exit__(self, *exc):
        if self.before != self.index:
            torch.cuda.set_device(self.before)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(nbytes, device, given):
    if given is None:
        return torch.empty(max(16, nbytes), dtype=torch.uint8, device=device)
    if given.device != device or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return given


def _nbytes(t):
    return t.numel() * t.element_size()


def _tokens(tokens, device):
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a tensor")
    bits = _INDEX_BITS.get(tokens.dtype)
    if bits is None:
        raise ValueError(f"tokens must be int32 or int64, got {tokens.dtype}")
    _on(tokens, "tokens", device)
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return bits


# ---------------------------------------------------------------- embedding


def embed_fwd(table, tokens, scale: float = 1.0, out=None):
    """out[..., C] = scale * table[tokens]; a token outside the table is padding and gives a zero row."""
    code = _float_code(table, "table")
    if table.dim() != 2 or table.shape[1] < 1:
        raise ValueError(f"table must be [rows, C], got {tuple(table.shape)}")
    device = _hip_device(table, "table")
    bits = _tokens(tokens, device)
    v, c = table.shape
    _, src = _rows(table, "table", (c,), table.dtype, device)
    n = tokens.numel()
    if out is None:
        out = torch.empty((*tokens.shape, c), dtype=table.dtype, device=device)
        dst = c
    else:
        if tuple(out.shape) != (*tokens.shape, c):
            raise ValueError(f"out must have shape {(*tokens.shape, c)}, got {tuple(out.shape)}")
        _, dst = _rows(out, "out", (c,), table.dtype, device)
    prob = EmbedProblem(n, v, src, dst, c, code, code, bits, scale)
    with _OnDevice(device) as st:
        train_check(train_lib().conv_tp_embed_fwd(ctypes.byref(prob), table.data_ptr(), tokens.data_ptr(),
                                                  out.data_ptr(), st))
    return out


def embed_bwd(grad_out, tokens, n_rows: int, scale: float = 1.0, out=None, dtype=None, workspace=None):
    """d_table[n_rows, C]: row v is scale times the sum of grad_out's rows whose token is v, zeros where there is
    none.  dtype: grad_out's, or float32.  workspace: any device tensor of enough bytes, allocated here if None."""
    code = _float_code(grad_out, "grad_out")
    device = _hip_device(grad_out, "grad_out")
    bits = _tokens(tokens, device)
    c = grad_out.shape[-1] if grad_out.dim() else 0
    if c < 1 or tuple(grad_out.shape[:-1]) != tuple(tokens.shape):
        raise ValueError(f"grad_out must have shape {(*tokens.shape, 'C')}, got {tuple(grad_out.shape)}")
    n, src = _rows(grad_out, "grad_out", (c,), grad_out.dtype, device, tokens.numel())
    n_rows = int(n_rows)
    if out is None:
        out = torch.empty((n_rows, c), dtype=dtype or grad_out.dtype, device=device)
    elif tuple(out.shape) != (n_rows, c) or dtype not in (None, out.dtype):
        raise ValueError(f"out must be [{n_rows}, {c}] {dtype or ''}, got {tuple(out.shape)} {out.dtype}")
    _, dst = _rows(out, "out", (c,), out.dtype, device)
    prob = EmbedProblem(n, n_rows, src, dst, c, code, _float_code(out, "out"), bits, scale)
    L = train_lib()
    nbytes = ctypes.c_int64()
    train_check(L.conv_tp_embed_bwd_workspace(ctypes.byref(prob), ctypes.byref(nbytes)))
    workspace = _workspace(nbytes.value, device, workspace)
    with _OnDevice(device) as st:
        train_check(L.conv_tp_embed_bwd(ctypes.byref(prob), grad_out.data_ptr(), tokens.data_ptr(), out.data_ptr(),
                                        workspace.data_ptr(), _nbytes(workspace), st))
    return out


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

_GATE_NONE, _GATE_CHANNEL, _GATE_ROW = 0, 1, 2


def _norm_problem(h, r, w_post, w_pre, gate, alpha, eps, lmax, grad_r=None, grad_u=None):
    """Checks a norm's arguments; (problem, device, row shape, parameter shape)."""
    lmax = int(lmax)
    if not 0 <= lmax <= 3:
        raise ValueError(f"lmax must be 0..3, got {lmax}")
    first = next((t for t in (h, r, grad_r) if t is not None), None)
    code = _float_code(first, "h" if h is not None else "r")
    device = _hip_device(first, "h" if h is not None else "r")
    dt = first.dtype
    if first.dim() < (1 if lmax == 0 else 2):
        raise ValueError(f"features must be [..., C] or [..., D, C], got {tuple(first.shape)}")
    c = first.shape[-1]
    tail = (c,) if lmax == 0 else ((lmax + 1) ** 2, c)
    per = (c,) if lmax == 0 else (lmax + 1, c)
    n, hs = _rows(first, "h" if h is not None else "r", tail, dt, device)
    strides = []
    for t, name in ((r, "r"), (grad_r, "grad_r"), (grad_u, "grad_u")):
        if t is None:
            strides.append(0)
            continue
        if t.shape != first.shape:
            raise ValueError(f"{name} must have shape {tuple(first.shape)}, got {tuple(t.shape)}")
        strides.append(_rows(t, name, tail, dt, device, n)[1])
    kind, gs = _GATE_NONE, 0
    params = [(t, name) for t, name in ((w_post, "w_post"), (w_pre, "w_pre")) if t is not None]
    if gate is not None:
        if not isinstance(gate, torch.Tensor):
            raise TypeError("gate must be a tensor")
        if tuple(gate.shape) == per and tuple(first.shape) != per:
            kind = _GATE_CHANNEL
            params.append((gate, "gate"))
        else:
            kind = _GATE_ROW
            if tuple(gate.shape) != (*first.shape[:first.dim() - len(tail)], *per):
                raise ValueError(f"gate must have shape {per} or one such for every row, got {tuple(gate.shape)}")
            gs = _rows(gate, "gate", per, dt, device, n)[1]
    pdt = params[0][0].dtype if params else dt
    if pdt != dt and pdt != torch.float32:
        raise ValueError(f"parameters must be {dt} or float32, got {pdt}")
    for t, name in params:
        if t.dtype != pdt:
            raise ValueError(f"{name} must be {pdt} like the other parameters, got {t.dtype}")
        if tuple(t.shape) != per:
            raise ValueError(f"{name} must have shape {per}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        _on(t, name, device)
    prob = NormProblem(n, hs, strides[0], gs, strides[1], strides[2], lmax, c, code, _DTYPES[pdt], kind, alpha, eps)
    return prob, device, first


def norm_residual_fwd(h, r, w_post, w_pre, gate=None, alpha: float = 1.0, eps: float = 1e-6, lmax: int = 0, out=None):
    """(r', u) with r' = r + alpha * gate * N(h; w_post) and u = N(r'; w_pre), N the root-mean-square norm over a
    row (balanced over the degrees for lmax > 0; see include/convtp_train.h).  h None: u = N(r; w_pre) alone, r'
    is r itself.  w_post None: h is added without a norm.  w_pre None: u is None.  gate: one row, or one for every
    row.  out: (r', u) to write into; r' may be r."""
    if r is None:
        raise TypeError("r must be a tensor")
    prob, device, first = _norm_problem(h, r, w_post, w_pre, gate, alpha, eps, lmax)
    r_out, u = out if out is not None else (None, None)
    if h is None:
        r_out = r
    elif r_out is None:
        r_out = torch.empty(first.shape, dtype=first.dtype, device=device)
    if w_pre is None:
        u = None
    elif u is None:
        u = torch.empty(first.shape, dtype=first.dtype, device=device)
    if out is not None:
        for t, name in ((r_out if h is not None else None, "r'"), (u, "u")):
            if t is not None and (t.shape != first.shape or t.dtype != first.dtype or t.device != device
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be a contiguous {first.dtype} tensor of shape {tuple(first.shape)}")
    with _OnDevice(device) as st:
        train_check(train_lib().conv_tp_norm_fwd(ctypes.byref(prob), _ptr(h), r.data_ptr(), _ptr(w_post), _ptr(w_pre),
                                                 _ptr(gate), _ptr(r_out if h is not None else None), _ptr(u), st))
    return r_out, u


def norm_residual_bwd(grad_r, grad_u, h, r_out, w_post, w_pre, gate=None, alpha: float = 1.0, eps: float = 1e-6,
                      lmax: int = 0, workspace=None):
    """Gradients (d_h, d_r, d_w_post, d_w_pre, d_gate) of norm_residual_fwd for grad_r (of r') and grad_u (of u),
    either of which may be None (zero); r_out is the forward's r'.  None in the place of what is absent."""
    if grad_r is None and grad_u is None:
        raise TypeError("grad_r and grad_u are both None")
    if grad_u is not None and w_pre is None:
        raise ValueError("grad_u without w_pre")
    if w_pre is not None and r_out is None:
        raise TypeError("r_out must be a tensor where there is w_pre")
    prob, device, first = _norm_problem(h, r_out, w_post, w_pre, gate, alpha, eps, lmax, grad_r, grad_u)
    new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=device)  # noqa: E731
    d_h, d_w_post, d_w_pre, d_gate = new(h), new(w_post), new(w_pre), new(gate)
    d_r = torch.empty(first.shape, dtype=first.dtype, device=device)
    L = train_lib()
    nbytes = ctypes.c_int64()
    train_check(L.conv_tp_norm_bwd_workspace(ctypes.byref(prob), ctypes.byref(nbytes)))
    workspace = _workspace(nbytes.value, device, workspace)
    with _OnDevice(device) as st:
        train_check(L.conv_tp_norm_bwd(ctypes.byref(prob), _ptr(grad_r), _ptr(grad_u), _ptr(h), _ptr(r_out),
                                       _ptr(w_post), _ptr(w_pre), _ptr(gate), _ptr(d_h), d_r.data_ptr(),
                                       _ptr(d_w_post), _ptr(d_w_pre), _ptr(d_gate), workspace.data_ptr(),
                                       _nbytes(workspace), st))
    return d_h, d_r, d_w_post, d_w_pre, d_gate


class NormResidualFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, h, r, w_post, w_pre, gate, alpha, eps, lmax):
        r_out, u = norm_residual_fwd(h, r, w_post, w_pre, gate, alpha, eps, lmax)
        ctx.save_for_backward(h, r_out if w_pre is not None else None, w_post, w_pre, gate)
        ctx.alpha, ctx.eps, ctx.lmax = alpha, eps, lmax
        ctx.set_materialize_grads(False)
        return (r_out.view_as(r_out) if h is None else r_out), u

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_r, grad_u):
        h, r_out, w_post, w_pre, gate = ctx.saved_tensors
        if grad_r is None and grad_u is None:
            return (None,) * 8
        grad_r, grad_u = (None if g is None else g.contiguous() for g in (grad_r, grad_u))
        d_h, d_r, d_w_post, d_w_pre, d_gate = norm_residual_bwd(grad_r, grad_u, h, r_out, w_post, w_pre, gate,
                                                                ctx.alpha, ctx.eps, ctx.lmax)
        return d_h, d_r, d_w_post, d_w_pre, d_gate, None, None, None


def norm_residual(h, r, w_post, w_pre, gate=None, alpha: float = 1.0, eps: float = 1e-6, lmax: int = 0):
    """Differentiable norm_residual_fwd (once)."""
    return NormResidualFunction.apply(h, r, w_post, w_pre, gate, float(alpha), float(eps), int(lmax))


# ---------------------------------------------------------------- clipping


def _address_list(tensors, name, device):
    """(addresses, elements, dtype codes) of dense tensors as arrays."""
    codes = [_DTYPES.get(t.dtype, -1) for t in tensors]
    if -1 in codes:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {tensors[codes.index(-1)].dtype}")
    for t in tensors:
        if t.device != device:
            raise ValueError(f"{name} must be on one device: {t.device} and {device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous (strides {t.stride()})")
    return (np.array([t.data_ptr() for t in tensors], dtype=np.int64),
            np.array([t.numel() for t in tensors], dtype=np.int64), np.array(codes, dtype=np.int32))


def _clip(tensors, out, max_norm, eps, norm):
    device = _hip_device(tensors[0], "tensors")
    at, numel, codes = _address_list(tensors, "tensors", device)
    to = None
    if out is not None:
        if out is tensors:
            to = at
        else:
            to, out_numel, out_codes = _address_list(out, "out", device)
            if not (np.array_equal(numel, out_numel) and np.array_equal(codes, out_codes)):
                raise ValueError("out must have the tensors' sizes and types")
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=device)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.device != device:
        raise ValueError("norm must be one float32 value on the tensors' device")
    L = train_lib()
    nbytes = L.conv_tp_clip_workspace(len(tensors))
    workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)
    with _OnDevice(device) as st:
        train_check(L.conv_tp_clip(len(tensors), at.ctypes.data, None if to is None else to.ctypes.data,
                                   numel.ctypes.data, codes.ctypes.data, max_norm, eps, norm.data_ptr(),
                                   workspace.data_ptr(), nbytes, st))
    return norm


def grad_norm(tensors, out=None):
    """The 2-norm of all elements of `tensors` together, a float32 value on their device."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no tensors")
    return _clip(tensors, None, 0.0, 0.0, out)


def clip_grad_norm(tensors, max_norm: float, eps: float = 1e-6, out=None):
    """(out, norm): every tensor times min(1, max_norm / (norm + eps)) with the global norm of all of them.
    out: the tensors to write, sizes and types like `tensors`; `tensors` itself clips in place; new ones if None.
    Nothing waits for the GPU."""
    tensors = list(tensors)
    if not tensors:
        raise ValueError("no tensors")
    out = [torch.empty_like(t, memory_format=torch.contiguous_format) for t in tensors] if out is None else list(out)
    if len(out) != len(tensors):
        raise ValueError(f"{len(out)} outputs for {len(tensors)} tensors")
    norm = _clip(tensors, out, float(max_norm), float(eps), None)
    return out, norm
