"""Where tiles of the dense operators' 16-bit operands are read from, on the host
under UndefinedBehaviorSanitizer (tests/sanitize/dense_places.hip)."""
import os

from tests.test_sanitizers_cpu import HIPCC, ROOT, SAN_ENV, _run


def test_places_of_direct_tiles_under_ubsan(tmp_path):
    exe = str(tmp_path / "dense_places")
    _run([HIPCC, "-O1", "-g", "-std=c++20", "--offload-arch=gfx950", "-ffp-contract=off", "-Xarch_host", "-fsanitize=undefined",
          "-Xarch_host", "-fno-sanitize-recover=all", os.path.join(ROOT, "tests", "sanitize", "dense_places.hip"), "-o", exe])
    r = _run([exe], env=dict(os.environ, **SAN_ENV))
    assert r.stdout.startswith("checked ") and "runtime error" not in r.stderr
