"""Whether the key axis of single tokens is read whole or in parts, as the forward workspace tells it (no parts: no bytes)."""
import ctypes
import os

import pytest


@pytest.fixture(scope="module")
def lib():
    from sparse_convolution_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libigconv.so is not built; run `python -m sparse_convolution_amd.build`")
    return _lib.load()


def workspace(lib, dtype, dim, batch, group, keys, kv_heads=4):
    from tests.test_block_refusals import _problem
    size = ctypes.c_size_t(0)
    p = _problem(dtype=dtype, batch=batch, heads=group * kv_heads, kv_heads=kv_heads, dim=dim, n_q=batch, n_k=batch * 8000,
                 d_q_offsets=4096, d_kv_offsets=4096)
    # The window, the token itself and no sinks: `keys` in all.
    assert lib.igc_window_attention_workspace(ctypes.byref(p), keys - 1, 0, 0, 0, ctypes.byref(size)) == 0
    return size.value


@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("dtype,dim,step", [(0, 20, 256), (0, 32, 256), (0, 64, 128), (0, 96, 64), (0, 128, 64), (1, 32, 256), (1, 64, 128)])
def test_the_limit_counts_rounds(lib, dtype, dim, step, group):
    # A round takes 1,024 keys over the lanes that hold one (4, 8 or 16).
    limit = (8 + 2 * group) * step
    assert workspace(lib, dtype, dim, 64, group, limit) == 0
    assert workspace(lib, dtype, dim, 64, group, limit + 1) > 0
    # Too few workgroups to fill the GPU: parts at any length that has two.
    assert workspace(lib, dtype, dim, 63, group, 512) > 0
    assert workspace(lib, dtype, dim, 64, group, 511) == 0 and workspace(lib, dtype, dim, 63, group, 511) == 0
