"""The C ABI of the dense operators without a GPU: every symbol of
include/convtp_dense.h is exported, and every invalid argument is refused on
the host, with its status and a message, before any HIP call."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D = (ctypes.c_void_p(0x10000 * k) for k in (1, 2, 3, 4))   # aligned addresses that nothing may touch
MIS4, MIS16 = ctypes.c_void_p(0x10002), ctypes.c_void_p(0x10008)
BIG = 1 << 50


@pytest.fixture(scope="module")
def capi():
    from tensor_product_message_amd import _capi
    if not os.path.exists(_capi.LIB_PATH):
        from tensor_product_message_amd.build import build
        build(verbose=False)
    return _capi


@pytest.fixture(scope="module")
def L(capi):
    return capi.dense_lib()


def message(L):
    return L.conv_tp_dense_last_error().decode()


def test_exports_every_declared_symbol(capi, L):
    src = open(os.path.join(ROOT, "include", "convtp_dense.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    declared = set(re.findall(r"\b(conv_tp_\w+)\s*\(", src))
    assert declared == set(capi.DENSE_EXPORTS)
    for name in declared:
        assert hasattr(L, name), name


def linear(capi, **kw):
    d = dict(n_rows=4, x_stride=8, residual_stride=6, grad_stride=6, lmax=0, inner=8, outer=6, dtype=0, act=2, gated=0)
    d.update(kw)
    return capi.LinearProblem(**d)


def fwd(L, p, x=A, w=A, bias=B, residual=None, y=C, z=D, ws=D, nbytes=BIG):
    return L.conv_tp_linear_fwd(ctypes.byref(p), x, w, bias, residual, y, z, ws, nbytes, None)


def bwd(L, p, grad=A, x=A, w=A, z=A, d_x=C, d_w=C, d_bias=C, ws=D, nbytes=BIG):
    return L.conv_tp_linear_bwd(ctypes.byref(p), grad, x, w, z, d_x, d_w, d_bias, ws, nbytes, None)


def second(L, p, a_d_x=A, grad=A, x=A, w=A, z=A, g_grad=C, g_x=C, g_w=C, g_bias=C, ws=D, nbytes=BIG):
    return L.conv_tp_linear_bwd_bwd(ctypes.byref(p), a_d_x, grad, x, w, z, g_grad, g_x, g_w, g_bias, ws, nbytes, None)


BAD = [
    (dict(n_rows=-1), "CTP_EINVAL"), (dict(n_rows=2 ** 31), "CTP_EUNSUPPORTED"), (dict(lmax=-1), "CTP_EUNSUPPORTED"),
    (dict(lmax=4), "CTP_EUNSUPPORTED"), (dict(inner=0), "CTP_EINVAL"), (dict(outer=0), "CTP_EINVAL"),
    (dict(inner=2 ** 20 + 1), "CTP_EUNSUPPORTED"), (dict(outer=2 ** 20 + 1), "CTP_EUNSUPPORTED"),
    (dict(act=0, lmax=3, inner=2 ** 16 + 1), "CTP_EUNSUPPORTED"), (dict(dtype=3), "CTP_EINVAL"), (dict(dtype=-1), "CTP_EINVAL"),
    (dict(act=6), "CTP_EINVAL"), (dict(act=-1), "CTP_EINVAL"), (dict(gated=2), "CTP_EINVAL"), (dict(lmax=1), "CTP_EINVAL"),
    (dict(lmax=1, act=0, gated=1), "CTP_EINVAL"), (dict(x_stride=7), "CTP_EINVAL"), (dict(x_stride=2 ** 41), "CTP_EINVAL"),
    (dict(x_stride=-8), "CTP_EINVAL"),
]


@pytest.mark.parametrize("bad,status", BAD)
def test_linear_rejects_problems(capi, L, bad, status):
    want = getattr(capi, status)
    p = linear(capi, **bad)
    n = ctypes.c_int64()
    assert [fwd(L, p), bwd(L, p), second(L, p)] == [want] * 3 and message(L)
    if "x_stride" not in bad:       # strides are not what a workspace depends on
        for size in (L.conv_tp_linear_fwd_workspace, L.conv_tp_linear_bwd_workspace, L.conv_tp_linear_bwd_bwd_workspace):
            assert size(ctypes.byref(p), ctypes.byref(n)) == want


def test_linear_rejects_arrays(capi, L):
    E, AL = capi.CTP_EINVAL, capi.CTP_EALIGN
    p = linear(capi)
    assert L.conv_tp_linear_fwd(None, A, A, B, None, C, D, D, BIG, None) == E
    assert [fwd(L, p, x=None), fwd(L, p, w=None), fwd(L, p, y=None), fwd(L, linear(capi, gated=1), residual=A),
            fwd(L, linear(capi, residual_stride=5), residual=A), fwd(L, p, nbytes=-1)] == [E] * 6
    for name in ("x", "w", "bias", "residual", "y", "z"):
        assert fwd(L, p, **{name: MIS4}) == AL, name
    for name in ("grad", "x", "w", "z", "ws"):
        assert bwd(L, p, **{name: None}) == E, name
    for name in ("grad", "x", "w", "z", "d_x", "d_w", "d_bias"):
        assert bwd(L, p, **{name: MIS4}) == AL, name
    for name in ("a_d_x", "grad", "x", "w", "z", "ws"):
        assert second(L, p, **{name: None}) == E, name
    for name in ("a_d_x", "grad", "x", "w", "z", "g_grad", "g_x", "g_w", "g_bias"):
        assert second(L, p, **{name: MIS4}) == AL, name
    assert [bwd(L, linear(capi, grad_stride=5)), second(L, linear(capi, grad_stride=5))] == [E] * 2
    assert [second(L, linear(capi, act=0)), second(L, linear(capi, act=0), g_x=None)] == [E] * 2
    n = ctypes.c_int64()
    for call, size in ((bwd, L.conv_tp_linear_bwd_workspace), (second, L.conv_tp_linear_bwd_bwd_workspace)):
        assert size(ctypes.byref(p), None) == E
        assert size(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK and n.value > 0 and message(L) == ""
        assert call(L, p, nbytes=n.value - 1) == E and "workspace" in message(L)
        assert call(L, p, ws=MIS16, nbytes=n.value) == AL


def test_workspaces_at_the_limits_are_counted_in_64_bits(capi, L):
    n = ctypes.c_int64()
    for gated in (0, 1):
        p = linear(capi, n_rows=2 ** 31 - 1, inner=2 ** 20, outer=2 ** 20, x_stride=2 ** 20, grad_stride=2 ** 20, gated=gated)
        for size in (L.conv_tp_linear_bwd_workspace, L.conv_tp_linear_bwd_bwd_workspace):
            assert size(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK
            assert n.value >= (2 ** 31 - 1) * 2 ** 20 * 4 * (1 + gated)


def test_workspaces_without_rows(capi, L):
    n = ctypes.c_int64()
    for kw in (dict(), dict(gated=1), dict(act=0), dict(act=0, lmax=2)):
        for dtype in (0, 1, 2):
            p = linear(capi, n_rows=0, inner=2049, outer=4096, x_stride=2 ** 16, grad_stride=2 ** 16, dtype=dtype, **kw)
            for size in (L.conv_tp_linear_fwd_workspace, L.conv_tp_linear_bwd_workspace, L.conv_tp_linear_bwd_bwd_workspace):
                assert size(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK and n.value >= 0


def ortho(L, ins=(A, B), outs=(C, D), batch=(1, 2), rows=(4, 5), cols=(6, 7), dtype=(0, 1), steps=5, eps=1e-7, scale=1.0,
          ws=B, nbytes=BIG, n=None):
    k = len(batch) if batch else 2
    arr = lambda t, v: None if v is None else (t * max(1, len(v)))(*v)  # noqa: E731
    val = lambda ps: None if ps is None else [p.value if p else None for p in ps]  # noqa: E731
    i32, i64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p
    return L.conv_tp_orthogonalise(k if n is None else n, arr(vp, val(ins)), arr(vp, val(outs)), arr(i64, batch), arr(i32, rows),
                                   arr(i32, cols), arr(i32, dtype), steps, eps, scale, ws, nbytes, None)


def test_orthogonalise_rejects(capi, L):
    E, AL, UN = capi.CTP_EINVAL, capi.CTP_EALIGN, capi.CTP_EUNSUPPORTED
    inf, nan = float("inf"), float("nan")
    assert [ortho(L, n=-1), ortho(L, ins=None), ortho(L, outs=None), ortho(L, batch=None), ortho(L, rows=None), ortho(L, cols=None),
            ortho(L, dtype=None), ortho(L, ins=(A, None)), ortho(L, outs=(None, D)), ortho(L, batch=(1, -1)),
            ortho(L, rows=(-1, 5)), ortho(L, cols=(6, -7)), ortho(L, dtype=(0, 3)), ortho(L, steps=0), ortho(L, steps=65),
            ortho(L, eps=-1.0), ortho(L, eps=nan), ortho(L, eps=inf), ortho(L, scale=nan), ortho(L, scale=inf),
            ortho(L, ws=None), ortho(L, nbytes=8)] == [E] * 22
    assert "workspace" in message(L)
    assert [ortho(L, rows=(2 ** 17 + 1, 5)), ortho(L, cols=(6, 2 ** 17 + 1)), ortho(L, batch=(2 ** 16 + 1, 2)),
            ortho(L, batch=(1, 2 ** 16), rows=(4, 2 ** 12), cols=(6, 2 ** 11))] == [UN] * 4
    assert [ortho(L, ins=(MIS4, B)), ortho(L, outs=(C, ctypes.c_void_p(0x40001))), ortho(L, ws=MIS16)] == [AL] * 3
    n = ctypes.c_int64()
    args = ((ctypes.c_int64 * 2)(1, 2), (ctypes.c_int32 * 2)(4, 5), (ctypes.c_int32 * 2)(6, 7))
    assert L.conv_tp_orthogonalise_workspace(2, *args, None) == E
    assert L.conv_tp_orthogonalise_workspace(2, *args, ctypes.byref(n)) == capi.CTP_OK and n.value > 0
    assert ortho(L, nbytes=n.value - 1) == E


def test_accepted_empty_calls_launch_nothing(capi, L):
    assert fwd(L, linear(capi, n_rows=0), x=None, w=None, y=None, z=None) == capi.CTP_OK
    assert bwd(L, linear(capi, n_rows=0), grad=None, x=None, w=None, z=None, d_w=None, d_bias=None) == capi.CTP_OK
    assert ortho(L, ins=(), outs=(), batch=(), rows=(), cols=(), dtype=(), n=0, ws=None, nbytes=0) == capi.CTP_OK
    assert ortho(L, batch=(0, 0)) == capi.CTP_OK and ortho(L, rows=(0, 0)) == capi.CTP_OK
    assert message(L) == ""


def test_binding_refuses_cpu_tensors():
    import torch

    import tensor_product_message_amd as ctp
    x, w, w2 = torch.zeros(4, 8), torch.zeros(6, 8), torch.zeros(2, 3, 8)
    g, g2 = torch.zeros(4, 6), torch.zeros(4, 3)
    for call in (lambda: ctp.linear_fwd(x, w), lambda: ctp.linear_bwd(g, x, w), lambda: ctp.linear_bwd_bwd(x, g, x, w),
                 lambda: ctp.gated_linear_fwd(x, w2), lambda: ctp.gated_linear_bwd(g2, x, w2, torch.zeros(4, 2, 3)),
                 lambda: ctp.linear(x, w), lambda: ctp.gated_linear(x, w2), lambda: ctp.orthogonalise([w])):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    with pytest.raises(TypeError):
        ctp.linear_fwd(None, w)
    with pytest.raises(ValueError, match="act must be"):
        ctp.linear_fwd(x, w, act="softmax")
