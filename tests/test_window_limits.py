"""Sizes of window attention that do not fit one launch are refused on the host (addresses here are never read: no call gets past its
checks)."""
import ctypes
import os

import pytest

INVALID, RANGE, CAPACITY = 1, 5, 6
P = ctypes.c_void_p(4096)  # stands for a device pointer
Q = ctypes.c_void_p(8192)


@pytest.fixture(scope="module")
def lib():
    from sparse_convolution_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libigconv.so is not built; run `python -m sparse_convolution_amd.build`")
    return _lib.load()


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("sinks,batch", [(2 ** 31 - 1, 1), (1_199_999_000, 1), (11_000_000, 100)])
def test_far_rows_of_sinks_share_the_launch_of_dk_and_dv(lib, sinks, batch, dtype):
    # 1.2e9 keys take 2.4e9 threads, and as many again where all tiles may hold sinks: more than 2^32 together.
    from tests.test_block_refusals import _problem
    n = 1_200_000_000
    p = ctypes.byref(_problem(dtype=dtype, batch=batch, heads=1, kv_heads=1, dim=1, n_q=n, n_k=n, d_q_offsets=4096, d_kv_offsets=4096))

    def backward(sinks, dq=Q, dk=Q, dv=Q):
        return lib.igc_window_attention_backward(p, 9, 0, sinks, P, P, P, P, P, P, dq, dk, dv, Q, 8, None)

    assert backward(sinks) == RANGE, lib.igc_last_error()
    assert b"one launch" in lib.igc_last_error()
    # dq alone, or no sinks: these would run, and want their workspace.
    assert backward(sinks, dk=None, dv=None) == CAPACITY
    assert backward(0) == CAPACITY
