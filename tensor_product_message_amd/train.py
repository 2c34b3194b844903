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

import array
import ctypes
import functools
import struct

import torch

from ._capi import EmbedProblem, NormProblem, train_check, train_lib

_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
_INDEX_BITS = {torch.int32: 32, torch.int64: 64}

# The problem structs as packed bytes: a tenth of the time of filling a ctypes.Structure.
_EMBED = struct.Struct("@qqqqiiiif4x")
_NORM = struct.Struct("@qqqqqqiiiiiff4x")
assert _EMBED.size == ctypes.sizeof(EmbedProblem) and _NORM.size == ctypes.sizeof(NormProblem)


def _tensor(t, name):
    """The device index of a float tensor on a HIP device."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {t.dtype}")
    index = t.get_device()
    if index < 0:
        raise ValueError(f"{name} must be on a HIP device, got {t.device}")
    return index


def _row_stride(t, name, shape, tail, width, dtype, index):
    """Elements from row to row of a tensor [..., *tail] of rows of `width` dense values."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected device {index}")
    if t.is_contiguous():
        return width
    strides = t.stride()
    inner, dense = strides[t.dim() - tail:], 1
    for size, stride in zip(reversed(shape[t.dim() - tail:]), reversed(inner)):
        if size > 1 and stride != dense:
            raise ValueError(f"{name}: a row must be contiguous (strides {strides})")
        dense *= size
    rows = [(n, s) for n, s in zip(shape[:t.dim() - tail], strides) if n > 1]
    if not rows:
        return width
    if len(rows) > 1 and any(a != n * b for (_, a), (n, b) in zip(rows, rows[1:])) or rows[-1][1] < width:
        raise ValueError(f"{name}: its rows must lie one stride apart and not overlap (strides {strides})")
    return rows[-1][1]


def _run(index, call, *args):
    """A library call on a device's current stream, with the device current."""
    before = torch.cuda.current_device()
    if before == index:
        train_check(call(*args, torch._C._cuda_getCurrentRawStream(index)))
        return
    torch.cuda.set_device(index)
    try:
        train_check(call(*args, torch._C._cuda_getCurrentRawStream(index)))
    finally:
        torch.cuda.set_device(before)


def _ptr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _workspace_bytes(kind, problem):
    """Bytes of workspace of a problem (sizes alone, so the answer never changes)."""
    out = ctypes.c_int64()
    train_check(getattr(train_lib(), f"conv_tp_{kind}_bwd_workspace")(problem, ctypes.byref(out)))
    return out.value


def _workspace(kind, problem, like, given):
    """(tensor, bytes): the caller's workspace, or one from torch's allocator."""
    if given is None:
        nbytes = max(16, _workspace_bytes(kind, problem))
        return torch.empty(nbytes, dtype=torch.uint8, device=like.device), nbytes
    if given.get_device() != like.get_device() or not given.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    return given, given.numel() * given.element_size()


def _tokens(tokens, index):
    if not isinstance(tokens, torch.Tensor):
        raise TypeError("tokens must be a tensor")
    bits = _INDEX_BITS.get(tokens.dtype)
    if bits is None:
        raise ValueError(f"tokens must be int32 or int64, got {tokens.dtype}")
    if tokens.get_device() != index:
        raise ValueError(f"tokens is on {tokens.device}, expected device {index}")
    if not tokens.is_contiguous():
        raise ValueError("tokens must be contiguous")
    return bits


# ---------------------------------------------------------------- embedding


def embed_fwd(table, tokens, scale: float = 1.0, out=None):
    """out[..., C] = scale * table[tokens]; a token outside the table is padding and gives a zero row."""
    index = _tensor(table, "table")
    if table.dim() != 2 or table.shape[1] < 1:
        raise ValueError(f"table must be [rows, C], got {tuple(table.shape)}")
    bits = _tokens(tokens, index)
    v, c = table.shape
    dt = table.dtype
    src = _row_stride(table, "table", table.shape, 1, c, dt, index)
    if out is None:
        out = torch.empty((*tokens.shape, c), dtype=dt, device=table.device)
        dst = c
    else:
        dst = _row_stride(out, "out", torch.Size((*tokens.shape, c)), 1, c, dt, index)
    code = _DTYPES[dt]
    prob = _EMBED.pack(tokens.numel(), v, src, dst, c, code, code, bits, scale)
    _run(index, train_lib().conv_tp_embed_fwd, prob, table.data_ptr(), tokens.data_ptr(), out.data_ptr())
    return out


def embed_bwd(grad_out, tokens, n_rows: int, scale: float = 1.0, out=None, dtype=None, workspace=None):
    """d_table[n_rows, C]: row v is scale times the sum of grad_out's rows whose token is v, zeros where there is
    none.  dtype: grad_out's, or float32.  workspace: any device tensor of enough bytes, allocated here if None."""
    index = _tensor(grad_out, "grad_out")
    bits = _tokens(tokens, index)
    shape, dt = grad_out.shape, grad_out.dtype
    c = shape[-1] if len(shape) else 0
    if c < 1 or shape[:-1] != tokens.shape:
        raise ValueError(f"grad_out must have shape {(*tokens.shape, 'C')}, got {tuple(shape)}")
    src = _row_stride(grad_out, "grad_out", shape, 1, c, dt, index)
    n_rows = int(n_rows)
    if out is None:
        out = torch.empty((n_rows, c), dtype=dtype or dt, device=grad_out.device)
        dst = c
    else:
        dst = _row_stride(out, "out", torch.Size((n_rows, c)), 1, c, dtype or out.dtype, index)
    if out.dtype not in _DTYPES:
        raise ValueError(f"out must be {dt} or float32, got {out.dtype}")
    prob = _EMBED.pack(tokens.numel(), n_rows, src, dst, c, _DTYPES[dt], _DTYPES[out.dtype], bits, scale)
    ws, nbytes = _workspace("embed", prob, grad_out, workspace)
    _run(index, train_lib().conv_tp_embed_bwd, prob, grad_out.data_ptr(), tokens.data_ptr(), out.data_ptr(),
         ws.data_ptr(), nbytes)
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
    """Checks a norm's arguments: (packed problem, device index, a tensor of the features' shape)."""
    lmax = int(lmax)
    if not 0 <= lmax <= 3:
        raise ValueError(f"lmax must be 0..3, got {lmax}")
    first, name = (h, "h") if h is not None else (r, "r") if r is not None else (grad_r, "grad_r")
    index = _tensor(first, name)
    dt, shape = first.dtype, first.shape
    tail = 1 if lmax == 0 else 2
    lead = len(shape) - tail
    if lead < 0 or shape[-1] < 1 or (lmax and shape[-2] != (lmax + 1) ** 2):
        raise ValueError(f"features must be [..., C], for lmax = {lmax} > 0 [..., {(lmax + 1) ** 2}, C], "
                         f"got {tuple(shape)}")
    c = shape[-1]
    width, per = (c, shape[lead:]) if lmax == 0 else (c * (lmax + 1) ** 2, torch.Size((lmax + 1, c)))
    stride = lambda t, name: 0 if t is None else _row_stride(t, name, shape, tail, width, dt, index)  # noqa: E731
    hs, rs, grs, gus = stride(h, "h"), stride(r, "r"), stride(grad_r, "grad_r"), stride(grad_u, "grad_u")
    kind, gs, pdt = _GATE_NONE, 0, None
    for t, name in ((w_post, "w_post"), (w_pre, "w_pre"), (gate, "gate")):
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a tensor")
        if name == "gate":
            if t.shape != per or lead == 0:
                kind = _GATE_ROW
                gs = _row_stride(t, "gate", shape[:lead] + per, tail, c * (lmax + 1), dt, index)
                continue
            kind = _GATE_CHANNEL
        if pdt is None:
            pdt = t.dtype
            if pdt != dt and pdt != torch.float32:
                raise ValueError(f"parameters must be {dt} or float32, got {pdt}")
        if t.dtype != pdt:
            raise ValueError(f"{name} must be {pdt} like the other parameters, got {t.dtype}")
        if t.shape != per:
            raise ValueError(f"{name} must have shape {tuple(per)}, got {tuple(t.shape)}")
        if t.get_device() != index:
            raise ValueError(f"{name} is on {t.device}, expected device {index}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    n = 1
    for size in shape[:lead]:
        n *= size
    prob = _NORM.pack(n, hs, rs, gs, grs, gus, lmax, c, _DTYPES[dt], _DTYPES[pdt or dt], kind, alpha, eps)
    return prob, index, first


def _dense(t):
    """A new dense tensor like t."""
    return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)


def norm_residual_fwd(h, r, w_post, w_pre, gate=None, alpha: float = 1.0, eps: float = 1e-6, lmax: int = 0, out=None):
    """(r', u) with r' = r + alpha * gate * N(h; w_post) and u = N(r'; w_pre), N the root-mean-square norm over a
    row (balanced over the degrees for lmax > 0; see include/convtp_train.h).  h None: u = N(r; w_pre) alone, r'
    is r itself.  w_post None: h is added without a norm.  w_pre None: u is None.  gate: one row, or one for every
    row.  out: (r', u) to write into, None for a new one; r' may be r."""
    if r is None:
        raise TypeError("r must be a tensor")
    prob, index, first = _norm_problem(h, r, w_post, w_pre, gate, alpha, eps, lmax)
    r_out, u = out if out is not None else (None, None)
    for t, name in ((r_out, "r'"), (u, "u")):
        if t is not None and (t.shape != first.shape or t.dtype != first.dtype or t.get_device() != index
                              or not t.is_contiguous()):
            raise ValueError(f"{name} must be a contiguous {first.dtype} tensor of shape {tuple(first.shape)}")
    if h is not None and r_out is None:
        r_out = _dense(first)
    if w_pre is None:
        u = None
    elif u is None:
        u = _dense(first)
    _run(index, train_lib().conv_tp_norm_fwd, prob, _ptr(h), r.data_ptr(), _ptr(w_post), _ptr(w_pre), _ptr(gate),
         None if h is None else r_out.data_ptr(), _ptr(u))
    return r if h is None else r_out, u


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
    prob, index, first = _norm_problem(h, r_out, w_post, w_pre, gate, alpha, eps, lmax, grad_r, grad_u)
    d_r, d_h, d_w_post, d_w_pre, d_gate = _dense(first), _dense(h), _dense(w_post), _dense(w_pre), _dense(gate)
    ws, nbytes = _workspace("norm", prob, first, workspace)
    _run(index, train_lib().conv_tp_norm_bwd, prob, _ptr(grad_r), _ptr(grad_u), _ptr(h), _ptr(r_out), _ptr(w_post),
         _ptr(w_pre), _ptr(gate), _ptr(d_h), d_r.data_ptr(), _ptr(d_w_post), _ptr(d_w_pre), _ptr(d_gate),
         ws.data_ptr(), nbytes)
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


def _addresses(tensors, name, index):
    """(addresses, elements, dtype codes) of dense tensors on one device."""
    T = torch.Tensor
    if not all(map(T.is_contiguous, tensors)):
        raise ValueError(f"{name} must be contiguous")
    if set(map(T.get_device, tensors)) != {index}:
        raise ValueError(f"{name} must be on one HIP device, {index}")
    dtypes = [t.dtype for t in tensors]
    kinds = set(dtypes)
    if not kinds <= _DTYPES.keys():
        raise ValueError(f"{name} must be float32, bfloat16 or float16, got {kinds - _DTYPES.keys()}")
    codes = [_DTYPES[dtypes[0]]] * len(dtypes) if len(kinds) == 1 else [_DTYPES[d] for d in dtypes]
    return list(map(T.data_ptr, tensors)), list(map(T.numel, tensors)), codes


def _clip(tensors, out, max_norm, eps, norm):
    index = _tensor(tensors[0], "tensors")
    at, numel, codes = _addresses(tensors, "tensors", index)
    to = 0
    if out is not None:
        to, out_numel, out_codes = _addresses(out, "out", index)
        if out_numel != numel or out_codes != codes:
            raise ValueError("out must have the tensors' sizes and types")
        to = array.array("q", to)
    if norm is None:
        norm = torch.empty((), dtype=torch.float32, device=tensors[0].device)
    elif norm.dtype != torch.float32 or norm.numel() != 1 or norm.get_device() != index:
        raise ValueError("norm must be one float32 value on the tensors' device")
    L = train_lib()
    at, numel, codes = array.array("q", at), array.array("q", numel), array.array("i", codes)
    nbytes = L.conv_tp_clip_workspace(len(tensors))
    ws = torch.empty(nbytes, dtype=torch.uint8, device=norm.device)
    _run(index, L.conv_tp_clip, len(tensors), at.buffer_info()[0], to.buffer_info()[0] if to else None,
         numel.buffer_info()[0], codes.buffer_info()[0], max_norm, eps, norm.data_ptr(), ws.data_ptr(), nbytes)
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
