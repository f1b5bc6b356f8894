"""Window attention's choice of shapes on the host: tests/sanitize/window_shapes_driver.cpp under the sanitizers (CPU only)."""
import os

import pytest

from tests.test_host_sanitizers import CLANG, HIPCC, ROOT, SAN, SAN_FLAGS, _env, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="hipcc / clang++ not available")
def test_window_shapes_under_asan_ubsan(tmp_path):
    obj, exe = str(tmp_path / "shapes.o"), str(tmp_path / "shapes_driver")
    host_san = [x for f in SAN_FLAGS for x in (["-Xarch_host", f] if f.startswith(("-fsanitize", "-fno-sanitize")) else [f])]
    _run([HIPCC, "-x", "hip", "--cuda-host-only", "-std=c++17", *host_san, "-I", os.path.join(ROOT, "sparse_convolution_amd", "csrc"),
          "-c", os.path.join(SAN, "window_shapes_driver.cpp"), "-o", obj])
    _run([CLANG, *SAN_FLAGS, obj, "-o", exe, "-lpthread"])
    r = _run([exe], env=_env(tmp_path))
    assert "window shapes driver: ok" in r.stdout
