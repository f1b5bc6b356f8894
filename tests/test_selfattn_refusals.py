"""What the operators of self-attention refuse, decided on the host before any launch: status codes and messages of the C
ABI (addresses here are never read), and the binding's own checks."""
import ctypes
import os

import pytest
import torch

INVALID, UNSUPPORTED, RANGE, CAPACITY = 1, 2, 5, 6
P = ctypes.c_void_p(4096)  # stands for a device pointer
Q = ctypes.c_void_p(8192)
R = ctypes.c_void_p(12288)


@pytest.fixture(scope="module")
def lib():
    from sparse_convolution_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libigconv.so is not built; run `python -m sparse_convolution_amd.build`")
    return _lib.load()


def _refused(lib, status, rc, word):
    assert rc == status, (rc, lib.igc_last_error())
    assert word in lib.igc_last_error(), lib.igc_last_error()


def _qk(**kw):
    from sparse_convolution_amd import _lib
    pair = ctypes.c_int64 * 2
    p = dict(dtype=1, heads=4, kv_heads=2, dim=64, axes=3, pairs=10, layout=0, norm=1, eps=1e-6, amplitude=1.0, n=100,
             q_stride=pair(256, 64), k_stride=pair(128, 64), d_positions=4096, d_frequencies=4096)
    p.update(kw)
    return ctypes.byref(_lib.Qk(**p))


@pytest.mark.parametrize("change,status,word", [
    ({"dtype": 2}, INVALID, b"dtype"), ({"n": -1}, INVALID, b"negative"), ({"heads": 0}, INVALID, b"positive"),
    ({"kv_heads": -1}, INVALID, b"kv_heads"), ({"dim": 0}, INVALID, b"positive"), ({"dim": 129}, UNSUPPORTED, b"128"),
    ({"n": 1 << 31}, RANGE, b"2^31"), ({"heads": 65535}, RANGE, b"65535"), ({"axes": 4}, INVALID, b"axes"), ({"axes": -1}, INVALID, b"axes"),
    ({"pairs": 11}, INVALID, b"pairs"), ({"pairs": 0}, INVALID, b"pairs"), ({"pairs": 1 << 30}, INVALID, b"pairs"),
    ({"layout": 2}, INVALID, b"layout"), ({"eps": -1.0}, INVALID, b"eps"), ({"eps": float("nan")}, INVALID, b"eps"),
    ({"eps": float("inf")}, INVALID, b"eps"), ({"amplitude": float("inf")}, INVALID, b"amplitude"),
    ({"amplitude": float("nan")}, INVALID, b"amplitude")])
def test_qk_problems(lib, change, status, word):
    p, size = _qk(**change), ctypes.c_size_t(0)
    _refused(lib, status, lib.igc_qk_norm_rotary_workspace(p, ctypes.byref(size)), word)
    _refused(lib, status, lib.igc_qk_norm_rotary(p, P, P, P, P, 0, Q, R, None), word)
    _refused(lib, status, lib.igc_qk_norm_rotary_backward(p, P, P, P, P, P, P, 0, Q, R, Q, Q, Q, 1 << 30, None), word)


def test_qk_arrays(lib):
    p, fwd, bwd = _qk(), lib.igc_qk_norm_rotary, lib.igc_qk_norm_rotary_backward
    _refused(lib, INVALID, fwd(None, P, P, P, P, 0, Q, R, None), b"problem")
    _refused(lib, INVALID, fwd(p, None, P, P, P, 0, Q, R, None), b"null")
    _refused(lib, INVALID, fwd(p, P, None, P, P, 0, Q, R, None), b"null")
    _refused(lib, INVALID, fwd(p, P, P, P, P, 0, Q, None, None), b"null")
    _refused(lib, INVALID, fwd(p, P, P, P, P, 2, Q, R, None), b"weights")
    _refused(lib, INVALID, fwd(_qk(dtype=0), P, P, P, P, 1, Q, R, None), b"weights")
    _refused(lib, INVALID, fwd(p, P, P, P, P, 0, P, R, None), b"aliases an input")
    _refused(lib, INVALID, fwd(p, P, P, P, P, 0, Q, Q, None), b"alias each other")
    _refused(lib, INVALID, fwd(_qk(d_positions=None), P, P, P, P, 0, Q, R, None), b"d_positions")
    _refused(lib, INVALID, fwd(_qk(d_frequencies=None), P, P, P, P, 0, Q, R, None), b"d_frequencies")
    assert fwd(_qk(n=0), None, None, None, None, 0, None, None, None) == 0
    _refused(lib, INVALID, bwd(p, None, P, P, P, P, P, 0, Q, R, Q, Q, Q, 1 << 30, None), b"d_dyq")
    _refused(lib, INVALID, bwd(p, P, None, P, P, P, P, 0, Q, R, Q, Q, Q, 1 << 30, None), b"d_dyk")
    _refused(lib, INVALID, bwd(p, P, P, None, P, P, P, 0, Q, R, Q, Q, Q, 1 << 30, None), b"null")
    _refused(lib, INVALID, bwd(p, P, P, P, P, P, P, 0, Q, R, Q, None, Q, 1 << 30, None), b"together")
    _refused(lib, INVALID, bwd(p, Q, P, P, P, P, P, 0, Q, R, Q, Q, Q, 1 << 30, None), b"aliases an input")
    _refused(lib, CAPACITY, bwd(p, P, P, P, P, P, P, 0, Q, R, Q, Q, Q, 8, None), b"workspace")
    _refused(lib, CAPACITY, bwd(p, P, P, P, P, P, P, 0, Q, R, Q, Q, None, 0, None), b"workspace")
    _refused(lib, INVALID, bwd(_qk(norm=0), P, P, None, None, None, None, 0, Q, R, Q, Q, Q, 1 << 30, None), b"without the norm")
    assert bwd(_qk(n=0), None, None, None, None, None, None, 0, None, None, None, None, None, 0, None) == 0
    _refused(lib, INVALID, lib.igc_qk_norm_rotary_workspace(p, None), b"bytes")


def test_dropout(lib):
    def drop(x=P, r=None, n=100, dt=0, p=0.1, seed=1, offset=2, d_offset=None, y=Q):
        return lib.igc_dropout(x, r, n, dt, p, seed, offset, d_offset, y, None)

    _refused(lib, INVALID, drop(dt=3), b"dtype")
    _refused(lib, INVALID, drop(n=-1), b"negative")
    for p in (-0.1, 1.1, float("nan"), float("inf")):
        _refused(lib, INVALID, drop(p=p), b"p must be")
    _refused(lib, INVALID, drop(x=None), b"null")
    _refused(lib, INVALID, drop(y=None), b"null")
    assert drop(n=0, x=None, y=None) == 0


def test_binding():
    import sparse_convolution_amd as igc
    x = torch.zeros(4, 2, 8)
    with pytest.raises(TypeError, match="q must be a CUDA"):
        igc.qk_norm_rotary(x, x)
    with pytest.raises(ValueError, match="needs positions"):
        igc.rotary(x, None, None)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        igc.dropout(x, 0.1, 3)
    with pytest.raises(TypeError, match="unsupported dtype"):
        igc.dropout(x.double(), 0.1, 3)
    for bad in (dict(axes=0), dict(axes=4), dict(axes=3, dim=4), dict(base=-1.0), dict(factor=0.0), dict(scaling="other"),
                dict(scaling="parts"), dict(scaling="parts", original=100, low=3.0, high=2.0)):
        with pytest.raises(ValueError):
            igc.rotary_frequencies(**{"dim": 64, **bad})


@pytest.mark.gpu
def test_binding_on_the_device():
    from tests._gpu import require_gpu
    require_gpu()
    import sparse_convolution_amd as igc
    x = torch.zeros(4, 2, 8, device="cuda")
    f, pos = igc.rotary_frequencies(8).cuda(), torch.arange(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="k must have shape"):
        igc.qk_norm_rotary(x, x[:3])
    with pytest.raises(ValueError, match="come together"):
        igc.qk_norm_rotary(x, x, pos)
    with pytest.raises(ValueError, match="layout"):
        igc.qk_norm_rotary(x, x, pos, f, layout="other")
    with pytest.raises(TypeError, match="positions must have dtype"):
        igc.rotary(x, pos.long(), f)
    with pytest.raises(ValueError, match="positions must have shape"):
        igc.rotary(x, pos[:3], f)
    with pytest.raises(ValueError, match="positions must have shape"):
        igc.rotary(x, pos, f.expand(2, -1).contiguous())
    with pytest.raises(igc.IgcError, match="pairs"):
        igc.rotary(x, pos, torch.ones(5, device="cuda"))
    with pytest.raises(ValueError, match="contiguous along"):
        igc.rotary(x.transpose(1, 2), pos, f)
    with pytest.raises(TypeError, match="float32 or"):
        igc.qk_norm_rotary(x, x, q_weight=torch.ones(8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="q_weight must have shape"):
        igc.qk_norm_rotary(x, x, q_weight=torch.ones(7, device="cuda"))
    with pytest.raises(ValueError, match="dq must have shape"):
        igc.qk_norm_rotary_backward(x[:3], x, x, x)
    with pytest.raises(ValueError, match="contiguous"):
        igc.dropout(x.transpose(0, 1), 0.1, 3)
    with pytest.raises(ValueError, match="residual must have shape"):
        igc.dropout(x, 0.1, 3, residual=x[:2])
    with pytest.raises(TypeError, match="offset must have dtype"):
        igc.dropout(x, 0.1, 3, torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="seed and offset"):
        igc.dropout(x, 0.1, -1)
    with pytest.raises(igc.IgcError, match="p must be"):
        igc.dropout(x, 1.5, 3)


@pytest.mark.parametrize("left,right,sinks,word", [(-2, 0, 0, b"left"), (3, -2, 0, b"right"), (3, 0, -1, b"sinks")])
def test_windows(lib, left, right, sinks, word):
    from tests.test_block_refusals import _problem
    p, size = ctypes.byref(_problem()), ctypes.c_size_t(0)
    _refused(lib, INVALID, lib.igc_window_attention_workspace(p, left, right, sinks, 0, ctypes.byref(size)), word)
    _refused(lib, INVALID, lib.igc_window_attention(p, left, right, sinks, None, P, P, P, Q, Q, Q, 1 << 40, None), word)
    _refused(lib, INVALID, lib.igc_window_attention_backward(p, left, right, sinks, P, P, P, P, P, P, Q, Q, Q, Q, 1 << 40, None), word)


def test_window_problems_and_operands(lib):
    from tests.test_block_refusals import _problem
    size = ctypes.c_size_t(0)
    for change, status, word in (({"dtype": 3}, INVALID, b"dtype"), ({"dim": 129}, UNSUPPORTED, b"128"), ({"n_k": 1 << 31}, RANGE, b"2^31"),
                                 ({"batch": 2}, INVALID, b"offsets"), ({"scale": 0.0}, INVALID, b"scale")):
        p = ctypes.byref(_problem(**change))
        _refused(lib, status, lib.igc_window_attention_workspace(p, 9, 0, 2, 1, ctypes.byref(size)), word)
        _refused(lib, status, lib.igc_window_attention(p, 9, 0, 2, None, P, P, P, Q, Q, Q, 1 << 40, None), word)
        assert b"igc_window_attention:" in lib.igc_last_error()
    p, few = ctypes.byref(_problem()), ctypes.byref(_problem(n_q=1, n_k=100000))
    fwd, bwd = lib.igc_window_attention, lib.igc_window_attention_backward
    _refused(lib, INVALID, fwd(None, 9, 0, 2, None, P, P, P, Q, Q, None, 0, None), b"problem")
    _refused(lib, INVALID, fwd(p, 9, 0, 2, None, None, P, P, Q, Q, None, 0, None), b"d_q")
    _refused(lib, INVALID, fwd(p, 9, 0, 2, None, P, P, P, P, Q, None, 0, None), b"aliases")
    _refused(lib, CAPACITY, fwd(few, 9000, 0, 2, None, P, P, P, Q, Q, None, 0, None), b"igc_window_attention_workspace")
    _refused(lib, CAPACITY, bwd(p, 9, 0, 2, P, P, P, P, P, P, Q, Q, Q, Q, 8, None), b"igc_window_attention_workspace")
    _refused(lib, INVALID, bwd(p, 9, 0, 2, P, P, P, P, P, P, Q, Q, Q, ctypes.c_void_p(8196), 1 << 40, None), b"aligned")
    _refused(lib, INVALID, bwd(p, 9, 0, 2, P, P, P, P, P, P, Q, Q, None, Q, 1 << 40, None), b"together")
    _refused(lib, INVALID, lib.igc_window_attention_workspace(p, 9, 0, 2, 0, None), b"bytes")
    _refused(lib, INVALID, fwd(p, -1, -1, 0, P, P, P, P, Q, Q, None, 0, None), b"d_kv_lengths need a limit")
    none = ctypes.byref(_problem(n_q=0, n_k=0))
    assert fwd(none, 9, 0, 2, None, None, None, None, None, None, None, 0, None) == 0
    assert bwd(none, 9, 0, 2, None, None, None, None, None, None, None, None, None, None, 0, None) == 0
    import sparse_convolution_amd as igc
    x = torch.zeros(4, 2, 8)
    with pytest.raises(TypeError, match="q must be a CUDA"):
        igc.window_attention(x, x, x, 3, 0)
    for kw in (dict(left=-1), dict(right=-1), dict(sinks=-1), dict(left=1 << 31), dict(sinks=1 << 31)):
        with pytest.raises(ValueError, match="must be 0 to"):
            igc.window_attention(x, x, x, **kw)
