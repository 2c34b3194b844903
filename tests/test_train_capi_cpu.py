"""The C ABI of the training-step operators without a GPU: every symbol of
include/convtp_train.h is exported, and every invalid argument is refused on
the host, with its status and a message, before any HIP call."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A, B, C, D = (ctypes.c_void_p(0x10000 * k) for k in (1, 2, 3, 4))   # aligned addresses that nothing may touch
ODD, MIS4 = ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10002)


@pytest.fixture(scope="module")
def capi():
    from tensor_product_message_amd import _capi
    if not os.path.exists(_capi.LIB_PATH):
        from tensor_product_message_amd.build import build
        build(verbose=False)
    return _capi


@pytest.fixture(scope="module")
def L(capi):
    return capi.train_lib()


def message(L):
    return L.conv_tp_train_last_error().decode()


def test_exports_every_declared_symbol(capi, L):
    src = open(os.path.join(ROOT, "include", "convtp_train.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    declared = set(re.findall(r"\b(conv_tp_\w+)\s*\(", src))
    assert declared == set(capi.TRAIN_EXPORTS)
    for name in declared:
        assert hasattr(L, name), name


def embed(capi, **kw):
    d = dict(n_tokens=4, n_rows=3, src_stride=8, dst_stride=8, channels=8, dtype=0, out_dtype=0, index_bits=32, scale=1.0)
    d.update(kw)
    return capi.EmbedProblem(**d)


EMBED_BAD = [  # field, value, status where both directions refuse it
    (dict(n_tokens=-1), "CTP_EINVAL"), (dict(n_rows=-1), "CTP_EINVAL"), (dict(channels=0), "CTP_EINVAL"),
    (dict(n_tokens=2 ** 31), "CTP_EUNSUPPORTED"), (dict(n_rows=2 ** 31 - 1), "CTP_EUNSUPPORTED"),
    (dict(channels=2 ** 20 + 1, src_stride=2 ** 21, dst_stride=2 ** 21), "CTP_EUNSUPPORTED"),
    (dict(dtype=3, out_dtype=3), "CTP_EINVAL"), (dict(dtype=-1, out_dtype=-1), "CTP_EINVAL"),
    (dict(out_dtype=1), "CTP_EINVAL"), (dict(out_dtype=7), "CTP_EINVAL"), (dict(index_bits=16), "CTP_EINVAL"),
    (dict(src_stride=7), "CTP_EINVAL"), (dict(dst_stride=7), "CTP_EINVAL"), (dict(src_stride=-8), "CTP_EINVAL"),
    (dict(src_stride=2 ** 41), "CTP_EINVAL"),
]


@pytest.mark.parametrize("bad,status", EMBED_BAD)
def test_embed_rejects_problems(capi, L, bad, status):
    want = getattr(capi, status)
    p = embed(capi, **bad)
    assert L.conv_tp_embed_fwd(ctypes.byref(p), A, B, C, None) == want and message(L)
    assert L.conv_tp_embed_bwd(ctypes.byref(p), A, B, C, D, 1 << 40, None) == want
    n = ctypes.c_int64()
    assert L.conv_tp_embed_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == want


def test_embed_rejects_arrays(capi, L):
    p = embed(capi)
    fwd = lambda p, *a: L.conv_tp_embed_fwd(ctypes.byref(p), *a, None)  # noqa: E731
    bwd = lambda p, *a: L.conv_tp_embed_bwd(ctypes.byref(p), *a, None)  # noqa: E731
    E, AL = capi.CTP_EINVAL, capi.CTP_EALIGN
    assert L.conv_tp_embed_fwd(None, A, B, C, None) == E
    assert [fwd(p, None, B, C), fwd(p, A, None, C), fwd(p, A, B, None)] == [E] * 3
    assert [fwd(p, MIS4, B, C), fwd(p, A, MIS4, C), fwd(p, A, B, MIS4)] == [AL] * 3
    assert fwd(embed(capi, dtype=1, out_dtype=1), ODD, B, C) == AL
    assert fwd(embed(capi, index_bits=64), A, ctypes.c_void_p(0x10004), C) == AL
    assert fwd(embed(capi, dtype=1, out_dtype=0), A, B, C) == E        # another type is for gradients alone
    n = ctypes.c_int64()
    assert L.conv_tp_embed_bwd_workspace(ctypes.byref(p), None) == E
    assert L.conv_tp_embed_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK and n.value > 0
    assert message(L) == ""
    big = n.value
    assert [bwd(p, None, B, C, D, big), bwd(p, A, None, C, D, big), bwd(p, A, B, None, D, big),
            bwd(p, A, B, C, None, big), bwd(p, A, B, C, D, big - 1), bwd(p, A, B, C, D, -1)] == [E] * 6
    assert bwd(p, A, B, C, ctypes.c_void_p(0x10008), big) == AL
    assert "workspace" in message(L)


def norm(capi, **kw):
    d = dict(n_rows=4, h_stride=32, r_stride=32, gate_stride=16, grad_r_stride=32, grad_u_stride=32, lmax=1, channels=8,
             dtype=0, param_dtype=0, gate=0, alpha=1.0, eps=1e-6)
    d.update(kw)
    return capi.NormProblem(**d)


def fwd(L, p, h=A, r=A, w_post=B, w_pre=B, gate=None, r_out=C, u=D):
    return L.conv_tp_norm_fwd(ctypes.byref(p), h, r, w_post, w_pre, gate, r_out, u, None)


def bwd(L, p, grad_r=A, grad_u=A, h=A, r_out=A, w_post=B, w_pre=B, gate=None, d_h=C, d_r=C, d_w_post=D, d_w_pre=D,
        d_gate=None, ws=D, nbytes=1 << 40):
    return L.conv_tp_norm_bwd(ctypes.byref(p), grad_r, grad_u, h, r_out, w_post, w_pre, gate, d_h, d_r, d_w_post,
                              d_w_pre, d_gate, ws, nbytes, None)


NORM_BAD = [
    (dict(n_rows=-1), "CTP_EINVAL"), (dict(n_rows=2 ** 31), "CTP_EUNSUPPORTED"), (dict(lmax=-1), "CTP_EUNSUPPORTED"),
    (dict(lmax=4), "CTP_EUNSUPPORTED"), (dict(channels=0), "CTP_EINVAL"), (dict(channels=4097), "CTP_EUNSUPPORTED"),
    (dict(dtype=5, param_dtype=5), "CTP_EINVAL"), (dict(param_dtype=1), "CTP_EINVAL"), (dict(gate=3), "CTP_EINVAL"),
    (dict(gate=-1), "CTP_EINVAL"), (dict(eps=-1e-6), "CTP_EINVAL"), (dict(eps=float("nan")), "CTP_EINVAL"),
]


@pytest.mark.parametrize("bad,status", NORM_BAD)
def test_norm_rejects_problems(capi, L, bad, status):
    want = getattr(capi, status)
    p = norm(capi, **bad)
    n = ctypes.c_int64()
    assert fwd(L, p) == want and message(L)
    assert bwd(L, p) == want
    assert L.conv_tp_norm_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == want


def test_norm_rejects_arrays(capi, L):
    E, AL = capi.CTP_EINVAL, capi.CTP_EALIGN
    p = norm(capi)
    assert L.conv_tp_norm_fwd(None, A, A, B, B, None, C, D, None) == E
    assert [fwd(L, p, r=None), fwd(L, p, r_out=None), fwd(L, p, u=None), fwd(L, p, h=None, w_pre=None),
            fwd(L, p, h=None), fwd(L, norm(capi, gate=1)), fwd(L, norm(capi, gate=2)),
            fwd(L, norm(capi, gate=1), h=None, w_post=None, gate=B)] == [E] * 8
    for name in ("h", "r", "w_post", "w_pre", "r_out", "u"):
        assert fwd(L, p, **{name: MIS4}) == AL, name
    assert [fwd(L, norm(capi, gate=1), gate=MIS4), fwd(L, norm(capi, gate=2), gate=MIS4)] == [AL] * 2
    assert fwd(L, norm(capi, dtype=1, param_dtype=0), w_post=MIS4) == AL     # float32 parameters
    assert [fwd(L, norm(capi, h_stride=31)), fwd(L, norm(capi, r_stride=0)),
            fwd(L, norm(capi, gate=2, gate_stride=15), gate=B)] == [E] * 3
    for name in ("r_out", "d_h", "d_r", "d_w_post", "d_w_pre", "ws"):
        assert bwd(L, p, **{name: None}) == E, name
    assert [bwd(L, p, w_pre=None), bwd(L, norm(capi, gate=1), gate=B), bwd(L, norm(capi, gate=2), gate=B),
            bwd(L, norm(capi, grad_r_stride=31)), bwd(L, norm(capi, grad_u_stride=31))] == [E] * 5
    for name in ("grad_r", "grad_u", "h", "r_out", "d_h", "d_r", "d_w_post", "d_w_pre"):
        assert bwd(L, p, **{name: MIS4}) == AL, name
    n = ctypes.c_int64()
    assert L.conv_tp_norm_bwd_workspace(ctypes.byref(p), None) == E
    assert L.conv_tp_norm_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK and n.value > 0
    assert bwd(L, p, nbytes=n.value - 1) == E
    assert bwd(L, p, ws=ctypes.c_void_p(0x10008), nbytes=n.value) == AL


def clip(L, ins=(A, B), outs=(C, D), numel=(4, 5), dtype=(0, 1), max_norm=1.0, eps=0.0, norm_=A, ws=B, nbytes=None, n=None):
    k = len(numel)
    arr = lambda t, v: (t * max(1, len(v)))(*v) if v is not None else None  # noqa: E731
    val = lambda ps: None if ps is None else [p.value if p else None for p in ps]  # noqa: E731
    i, o = arr(ctypes.c_void_p, val(ins)), arr(ctypes.c_void_p, val(outs))
    m, d = arr(ctypes.c_int64, numel), arr(ctypes.c_int32, dtype)
    need = L.conv_tp_clip_workspace(k)
    return L.conv_tp_clip(k if n is None else n, i, o, m, d, max_norm, eps, norm_, ws, need if nbytes is None else nbytes, None)


def test_clip_rejects(capi, L):
    E, AL = capi.CTP_EINVAL, capi.CTP_EALIGN
    assert [clip(L, n=-1), clip(L, ins=None), clip(L, dtype=(0, 3)), clip(L, numel=(4, -1)), clip(L, numel=(4, 2 ** 41)),
            clip(L, ins=(A, None)), clip(L, outs=(None, D)), clip(L, max_norm=-1.0), clip(L, max_norm=float("nan")),
            clip(L, eps=-1.0), clip(L, eps=float("nan")), clip(L, norm_=None), clip(L, ws=None), clip(L, nbytes=8)] == [E] * 14
    assert "workspace" in message(L)
    assert [clip(L, ins=(MIS4, B)), clip(L, ins=(A, ODD)), clip(L, outs=(MIS4, D)), clip(L, norm_=MIS4),
            clip(L, ws=ctypes.c_void_p(0x10008))] == [AL] * 5
    assert L.conv_tp_clip_workspace(-3) >= 0


def test_accepted_empty_calls_launch_nothing(capi, L):
    assert L.conv_tp_embed_fwd(ctypes.byref(embed(capi, n_tokens=0)), None, None, None, None) == capi.CTP_OK
    assert L.conv_tp_embed_bwd(ctypes.byref(embed(capi, n_rows=0)), A, B, None, D, 1 << 40, None) == capi.CTP_OK
    assert fwd(L, norm(capi, n_rows=0), h=None, r=None, r_out=None, u=None) == capi.CTP_OK
    assert message(L) == ""


def test_binding_refuses_cpu_tensors():
    import torch

    import tensor_product_message_amd as ctp
    x, ids = torch.zeros(4, 8), torch.zeros(4, dtype=torch.int64)
    for call in (lambda: ctp.embed_fwd(x, ids), lambda: ctp.embed_bwd(x, ids, 4),
                 lambda: ctp.norm_residual_fwd(x, x, x[0], x[0]), lambda: ctp.norm_residual_bwd(x, x, x, x, x[0], x[0]),
                 lambda: ctp.grad_norm([x]), lambda: ctp.clip_grad_norm([x], 1.0)):
        with pytest.raises(ValueError, match="HIP device"):
            call()
    for call in (lambda: ctp.embed_fwd(None, ids), lambda: ctp.norm_residual_fwd(x, None, None, None)):
        with pytest.raises(TypeError):
            call()


def second(L, p, a_d_h=A, a_d_r=A, grad_r=A, grad_u=A, h=A, r_out=A, w_post=B, w_pre=B, gate=None, g_grad_r=C, g_grad_u=C,
           g_h=C, g_r=C, g_w_post=D, g_w_pre=D, g_gate=None, ws=D, nbytes=1 << 40):
    return L.conv_tp_norm_bwd_bwd(ctypes.byref(p), a_d_h, a_d_r, grad_r, grad_u, h, r_out, w_post, w_pre, gate,
                                  g_grad_r, g_grad_u, g_h, g_r, g_w_post, g_w_pre, g_gate, ws, nbytes, None)


def test_norm_second_backward_rejects(capi, L):
    E, AL = capi.CTP_EINVAL, capi.CTP_EALIGN
    p = norm(capi)
    for name in ("r_out", "g_h", "g_r", "g_w_post", "g_w_pre", "ws"):
        assert second(L, p, **{name: None}) == E, name
    for name in ("a_d_h", "a_d_r", "grad_r", "grad_u", "h", "r_out", "g_grad_r", "g_grad_u", "g_h", "g_r", "g_w_post", "g_w_pre"):
        assert second(L, p, **{name: MIS4}) == AL, name
    assert [second(L, p, w_pre=None), second(L, p, h=None, w_post=None), second(L, norm(capi, gate=1), gate=B),
            second(L, norm(capi, grad_r_stride=31)), second(L, p, nbytes=0)] == [E] * 5
    for bad, status in NORM_BAD:
        assert second(L, norm(capi, **bad)) == getattr(capi, status), bad
