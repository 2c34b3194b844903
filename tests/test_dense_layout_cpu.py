"""How the dense operators lay out their workspaces, without a GPU: through the C ABI, and on the host under
AddressSanitizer and UndefinedBehaviorSanitizer (tests/sanitize/ortho_layout.hip, dense_access.hip)."""
import ctypes
import os

import pytest

from tests.test_sanitizers_cpu import HIPCC, ROOT, SAN_ENV, _run


@pytest.fixture(scope="module")
def capi():
    from tensor_product_message_amd import _capi
    if not os.path.exists(_capi.LIB_PATH):
        from tensor_product_message_amd.build import build
        build(verbose=False)
    return _capi


def ortho_workspace(capi, shapes):
    n, arr = ctypes.c_int64(-1), lambda t, k: (t * len(shapes))(*(s[k] for s in shapes))  # noqa: E731
    status = capi.dense_lib().conv_tp_orthogonalise_workspace(len(shapes), arr(ctypes.c_int64, 0), arr(ctypes.c_int32, 1),
                                                              arr(ctypes.c_int32, 2), ctypes.byref(n))
    assert status == capi.CTP_OK
    return n.value


@pytest.mark.parametrize("shapes", [[(65536, 3, 2)], [(1024, 1024, 1024)], [(60000, 3, 2)], [(1, 131072, 4096)], [(1, 131072, 131072)],
                                    [(1, 16384, 8192)] * 7, [(4, 2048, 8192)] * 20, [(1, 64, 64)] * 31 + [(200, 1000, 1500)] * 5])
def test_workspace_of_many_matrices_is_counted_in_64_bits(capi, shapes):
    pad = lambda n: (n + 63) // 64 * 64  # noqa: E731
    least = 0
    for first in range(0, len(shapes), 32):     # a launch's tensors
        # X, the next X, A and b A + c A A of every matrix, 32 bits a value
        least = max(least, sum(8 * b * (pad(r) * pad(c) + pad(min(r, c)) ** 2) for b, r, c in shapes[first:first + 32]))
    n = ortho_workspace(capi, shapes)
    assert least <= n <= 40 * least
    assert least > 2 ** 31 or shapes[0] == (1, 131072, 4096)


@pytest.mark.parametrize("rows,lmax,act,inner,outer", [(5, 1, 0, 16384, 16384), (300, 3, 0, 65536, 2048), (64, 1, 0, 131072, 131072),
                                                       (40, 0, 2, 16384, 16384), (7, 0, 1, 2 ** 20, 1024), (65, 0, 4, 65536, 65536)])
@pytest.mark.parametrize("gated", [0, 1])
@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_workspace_of_large_matrices_is_counted_in_64_bits(capi, rows, lmax, act, inner, outer, gated, dtype):
    """The parts of d_w: one a component, of the second pass one of each of its two products, in fp32."""
    if gated and lmax:
        return
    L, n, comps = capi.dense_lib(), ctypes.c_int64(), (lmax + 1) ** 2
    p = capi.LinearProblem(rows, comps * inner, comps * outer, comps * outer, lmax, inner, outer, dtype, act, gated)
    matrix = 4 * inner * outer * (1 + gated)
    assert L.conv_tp_linear_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK
    assert n.value >= (comps * matrix if lmax else 0)
    assert L.conv_tp_linear_bwd_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK
    assert n.value >= (comps if lmax else 2) * matrix >= 2 ** 31


HOST = [HIPCC, "-O2", "-g", "-std=c++20", "--offload-arch=gfx950", "--offload-host-only", "-ffp-contract=off", "-Wno-undefined-inline",
        # no kernel is launched, and none is there
        "-Wl,--unresolved-symbols=ignore-all", "-Xarch_host", "-fsanitize=undefined", "-Xarch_host", "-fno-sanitize-recover=all"]


def run_on_host(tmp_path, source, *flags):
    exe = str(tmp_path / "program")
    _run([*HOST, *flags, os.path.join(ROOT, "tests", "sanitize", source), "-o", exe])
    r = _run([exe], env=dict(os.environ, **SAN_ENV))
    assert r.stdout.startswith("checked ") and "runtime error" not in r.stderr


def test_layout_of_orthogonalised_matrices_under_sanitizers(tmp_path):
    run_on_host(tmp_path, "ortho_layout.hip", "-Xarch_host", "-fsanitize=address")


@pytest.mark.parametrize("dtype", [0, 1, 2])
def test_reads_and_regions_of_linear_layers_under_ubsan(tmp_path, dtype):
    run_on_host(tmp_path, "dense_access.hip", f"-DCTP_DENSE_TYPE={dtype}")


@pytest.mark.parametrize("shape", [(1, 0, 0), (1, 0, 5), (1, 5, 0), (2, 0, 0), (0, 5, 5), (0, 0, 0)])
def test_empty_matrices(capi, shape):
    assert ortho_workspace(capi, [shape]) == 0 and ortho_workspace(capi, [shape, (1, 3, 4), shape]) == ortho_workspace(capi, [(1, 3, 4)])
    one, none = lambda t, x: (t * 1)(x), (ctypes.c_void_p * 1)(None)  # noqa: E731
    sizes = one(ctypes.c_int64, shape[0]), one(ctypes.c_int32, shape[1]), one(ctypes.c_int32, shape[2])
    assert capi.dense_lib().conv_tp_orthogonalise(1, none, none, *sizes, one(ctypes.c_int32, 0), 5, 1e-7, 1.0, None, 0, None) == capi.CTP_OK


def test_workspaces_go_by_the_strides(capi):
    """16-bit rows that do not begin on 16 bytes are laid out anew, which takes room: a query's strides are its call's."""
    L, n = capi.dense_lib(), ctypes.c_int64()
    sizes = {}
    for x_stride in (1000, 1001, 1008):
        for grad_stride in (1000, 1001, 1008):
            p = capi.LinearProblem(5000, x_stride, 1000, grad_stride, 0, 1000, 1000, 1, 0, 0)
            assert L.conv_tp_linear_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK
            sizes[x_stride % 8, grad_stride % 8] = n.value
    rows = 5000 * 1000 * 2
    assert sizes[1, 0] >= sizes[0, 0] + rows and sizes[0, 1] >= sizes[0, 0] + rows and sizes[1, 1] >= sizes[0, 0] + 2 * rows


@pytest.mark.parametrize("lmax,x_stride,grad_stride", [(0, 7, 6), (0, 0, 6), (0, 2 ** 41, 6), (0, -8, 6), (1, 31, 24), (0, 8, 5), (0, 8, 0), (2, 72, 53)])
def test_workspace_queries_refuse_the_strides_that_calls_refuse(capi, lmax, x_stride, grad_stride):
    L, n = capi.dense_lib(), ctypes.c_int64()
    p = capi.LinearProblem(4, x_stride, 0, grad_stride, lmax, 8, 6, 0, 0, 0)
    bad_x = x_stride < 8 * (lmax + 1) ** 2 or x_stride > 2 ** 40
    assert L.conv_tp_linear_fwd_workspace(ctypes.byref(p), ctypes.byref(n)) == (capi.CTP_EINVAL if bad_x else capi.CTP_OK)
    for size in (L.conv_tp_linear_bwd_workspace, L.conv_tp_linear_bwd_bwd_workspace):
        assert size(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_EINVAL
        assert b"stride" in L.conv_tp_dense_last_error()
    for rows in (0, 1):         # strides of no next row
        p.n_rows = rows
        assert L.conv_tp_linear_bwd_workspace(ctypes.byref(p), ctypes.byref(n)) == capi.CTP_OK
