"""The C ABI front of the dense operators (csrc/dense_api.hip) under
AddressSanitizer and UndefinedBehaviorSanitizer, linked against stubs of its
kernels and run under tests/test_dense_capi_cpu.py in a child process, as
tests/test_train_sanitizers_cpu.py does for the training step's."""
import os

import pytest

from tests.test_sanitizers_cpu import CSRC, HIPCC, ROOT, _child_pytest, _clang_asan_runtime, _run


def test_dense_front_under_asan_and_ubsan(tmp_path):
    runtime = _clang_asan_runtime()
    if runtime is None:
        pytest.skip("clang AddressSanitizer runtime not found under /opt/rocm/llvm")
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all", "-Xarch_host", "-fno-omit-frame-pointer"]
    common = ["-O1", "-g", "-std=c++20", "-fPIC", "--offload-arch=gfx950", "-ffp-contract=off"]
    stubs = os.path.join(ROOT, "tests", "sanitize")
    objects = []
    for src, flags in ((os.path.join(CSRC, "dense_api.hip"), san), (os.path.join(CSRC, "convtp_api.hip"), []),
                       (os.path.join(stubs, "dense_stubs.hip"), []), (os.path.join(stubs, "launch_stubs.hip"), [])):
        objects.append(str(tmp_path / (os.path.basename(src) + ".o")))
        _run([HIPCC, *common, *flags, "-c", src, "-o", objects[-1]])
    lib = str(tmp_path / "libconvtp_dense_asan.so")
    _run([HIPCC, "-shared", "-fPIC", "--offload-arch=gfx950", "-o", lib, *objects])
    out = _child_pytest({"CONVTP_LIB": lib}, [runtime], [os.path.join("tests", "test_dense_capi_cpu.py"), "-k", "not binding"])
    assert " passed" in out
