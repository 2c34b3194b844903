"""Where the training-step kernels' lanes read a row's vectors and how far they
shift them, on the host under UndefinedBehaviorSanitizer
(tests/sanitize/row_access.hip)."""
import os

from tests.test_sanitizers_cpu import HIPCC, ROOT, SAN_ENV, _run


def test_vectors_of_a_row_under_ubsan(tmp_path):
    exe = str(tmp_path / "row_access")
    _run([HIPCC, "-O1", "-g", "-std=c++20", "--offload-arch=gfx950", "-ffp-contract=off", "-Xarch_host", "-fsanitize=undefined",
          "-Xarch_host", "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "sanitize", "row_access.hip"), "-o", exe])
    r = _run([exe], env=dict(os.environ, **SAN_ENV))
    assert r.stdout.startswith("checked ") and "runtime error" not in r.stderr
