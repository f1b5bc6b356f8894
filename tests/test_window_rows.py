"""The index arithmetic of sliding windows under the host sanitizers: tests/sanitize/window_driver.cpp walks every row, key and
tile of many small problems and compares them with the formula (CPU only)."""
import os

import pytest

from tests.test_host_sanitizers import CLANG, HIPCC, ROOT, SAN, SAN_FLAGS, _env, _run


@pytest.mark.skipif(not (os.path.exists(HIPCC) and os.path.exists(CLANG)), reason="hipcc / clang++ not available")
def test_window_rows_under_asan_ubsan(tmp_path):
    obj, exe = str(tmp_path / "window.o"), str(tmp_path / "window_driver")
    host_san = [x for f in SAN_FLAGS for x in (["-Xarch_host", f] if f.startswith(("-fsanitize", "-fno-sanitize")) else [f])]
    _run([HIPCC, "-x", "hip", "--cuda-host-only", "-std=c++17", *host_san, "-I", os.path.join(ROOT, "sparse_convolution_amd", "csrc"),
          "-c", os.path.join(SAN, "window_driver.cpp"), "-o", obj])
    _run([CLANG, *SAN_FLAGS, obj, "-o", exe, "-lpthread"])
    r = _run([exe], env=_env(tmp_path))
    assert "window driver: ok" in r.stdout
