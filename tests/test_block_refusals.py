"""What the operators between convolutions refuse, decided on the host before any launch: status codes and
messages of the C ABI (addresses here are never read), and the binding's own checks."""
import ctypes
import os

import pytest
import torch

INVALID, UNSUPPORTED, RANGE, CAPACITY = 1, 2, 5, 6
P = ctypes.c_void_p(4096)  # stands for a device pointer
Q = ctypes.c_void_p(8192)


@pytest.fixture(scope="module")
def lib():
    from sparse_convolution_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        pytest.fail("libigconv.so is not built; run `python -m sparse_convolution_amd.build`")
    return _lib.load()


def _refused(lib, status, rc, word):
    assert rc == status, (rc, lib.igc_last_error())
    assert word in lib.igc_last_error(), lib.igc_last_error()


def test_layer_norm(lib):
    def norm(x=P, n=3, c=8, dt=0, w=P, b=P, wd=0, eps=1e-5, y=Q, mean=Q, rstd=Q):
        return lib.igc_layer_norm(x, n, c, dt, w, b, wd, eps, y, mean, rstd, None)

    _refused(lib, INVALID, norm(dt=2), b"igc_layer_norm: bad dtype")
    _refused(lib, INVALID, norm(n=-1), b"n is negative")
    _refused(lib, INVALID, norm(c=0), b"c must be positive")
    _refused(lib, UNSUPPORTED, norm(c=4097), b"4096")
    _refused(lib, RANGE, norm(n=1 << 31), b"2^31")
    _refused(lib, INVALID, norm(wd=1), b"weight")
    _refused(lib, INVALID, norm(eps=-1.0), b"eps")
    _refused(lib, INVALID, norm(eps=float("nan")), b"eps")
    _refused(lib, INVALID, norm(x=None), b"null")
    _refused(lib, INVALID, norm(y=P), b"aliases")
    _refused(lib, INVALID, norm(mean=None), b"d_mean")
    assert norm(n=0, x=None, y=None, mean=None, rstd=None) == 0
    _refused(lib, INVALID, lib.igc_layer_norm_q8(P, 3, 8, 0, P, P, 0, 1e-5, Q, None, Q, Q, None), b"igc_layer_norm_q8")


def test_layer_norm_backward(lib):
    size = ctypes.c_size_t(0)
    assert lib.igc_layer_norm_workspace(1000, 64, ctypes.byref(size)) == 0 and size.value >= 2 * 64 * 4
    _refused(lib, INVALID, lib.igc_layer_norm_workspace(1000, 64, None), b"bytes")
    _refused(lib, UNSUPPORTED, lib.igc_layer_norm_workspace(1000, 5000, ctypes.byref(size)), b"4096")

    def grad(dy=P, x=P, mean=P, rstd=P, n=1000, c=64, dt=1, w=P, wd=0, dx=Q, dw=Q, db=Q, ws=Q, nb=1 << 30):
        return lib.igc_layer_norm_backward(dy, x, mean, rstd, n, c, dt, w, wd, dx, dw, db, ws, nb, None)

    _refused(lib, INVALID, grad(dy=None), b"d_dy")
    _refused(lib, INVALID, grad(x=None), b"d_x")
    _refused(lib, INVALID, grad(db=None), b"together")
    _refused(lib, INVALID, grad(dx=P), b"aliases")
    _refused(lib, INVALID, grad(dt=0, wd=1), b"weight")
    _refused(lib, CAPACITY, grad(nb=100), b"workspace")
    _refused(lib, CAPACITY, grad(ws=None), b"workspace")
    _refused(lib, INVALID, lib.igc_layer_norm_q8_backward(P, None, P, P, 3, 8, 1, P, 0, Q, Q, Q, Q, 1 << 30, None), b"d_codes")


def test_checkpoints(lib):
    _refused(lib, INVALID, lib.igc_checkpoint_pack(None, 3, 8, 0, P, P, None), b"igc_checkpoint_pack")
    _refused(lib, INVALID, lib.igc_checkpoint_pack(P, 3, 8, 7, P, P, None), b"dtype")
    _refused(lib, UNSUPPORTED, lib.igc_checkpoint_pack(P, 3, 9999, 0, P, P, None), b"4096")
    _refused(lib, INVALID, lib.igc_checkpoint_unpack(P, None, 3, 8, 0, P, None), b"igc_checkpoint_unpack")
    _refused(lib, INVALID, lib.igc_sparse_conv_backward_q8(None, P, P, P, 1, 64, P, 64, P, None, P, 0, None),
             b"igc_sparse_conv_backward_q8: grid")


def _problem(**kw):
    from sparse_convolution_amd import _lib
    pair = ctypes.c_int64 * 2
    p = dict(dtype=1, batch=1, heads=4, kv_heads=2, dim=64, scale=0.125, n_q=100, n_k=50, q_stride=pair(256, 64),
             k_stride=pair(128, 64), v_stride=pair(128, 64), d_q_offsets=None, d_kv_offsets=None, d_key_mask=None)
    p.update(kw)
    return _lib.Attention(**p)


@pytest.mark.parametrize("change,status,word", [
    ({"dtype": 3}, INVALID, b"dtype"), ({"n_q": -1}, INVALID, b"negative"), ({"heads": 0}, INVALID, b"positive"),
    ({"batch": 0}, INVALID, b"positive"), ({"heads": 3}, INVALID, b"multiple"), ({"dim": 129}, UNSUPPORTED, b"128"),
    ({"batch": 2}, INVALID, b"offsets"), ({"scale": 0.0}, INVALID, b"scale"), ({"scale": float("nan")}, INVALID, b"scale"),
    ({"scale": -1.0}, INVALID, b"scale"), ({"scale": float("inf")}, INVALID, b"scale"), ({"n_k": 1 << 31}, RANGE, b"2^31"),
    ({"n_q": 1 << 30}, RANGE, b"2^31"), ({"n_q": 1 << 28, "heads": 1024, "kv_heads": 1024}, RANGE, b"launch")])
def test_attention_problems(lib, change, status, word):
    p, size = ctypes.byref(_problem(**change)), ctypes.c_size_t(0)
    _refused(lib, status, lib.igc_cross_attention_workspace(p, 0, ctypes.byref(size)), word)
    _refused(lib, status, lib.igc_cross_attention(p, P, P, P, Q, Q, Q, 1 << 40, None), word)
    _refused(lib, status, lib.igc_cross_attention_backward(p, P, P, P, P, P, P, Q, Q, Q, Q, 1 << 40, None), word)


@pytest.mark.parametrize("change", [{"n_k": (1 << 31) - 1}, {"n_k": (1 << 31) - 129}, {"n_k": (1 << 31) - 1023}, {"n_q": (1 << 31) - 1023},
                                    {"n_q": (1 << 30) - 511, "heads": 2}])
def test_attention_row_counts_within_a_tile_of_2_to_the_31(lib, change):
    # The kernels step up to 256 past a sequence's end in 32 bits. 2^31 - 1024 is the largest count taken.
    problem = dict({"n_q": 3, "n_k": 3, "heads": 1, "kv_heads": 1}, **change)
    p, size = ctypes.byref(_problem(**problem)), ctypes.c_size_t(0)
    _refused(lib, RANGE, lib.igc_cross_attention_workspace(p, 0, ctypes.byref(size)), b"2^31 - 1024")
    _refused(lib, RANGE, lib.igc_cross_attention(p, P, P, P, Q, Q, Q, 1 << 40, None), b"2^31 - 1024")
    _refused(lib, RANGE, lib.igc_cross_attention_backward(p, P, P, P, P, P, P, Q, Q, Q, Q, 1 << 40, None), b"2^31 - 1024")
    largest = _problem(n_q=3, n_k=(1 << 31) - 1024, heads=1, kv_heads=1)
    assert lib.igc_cross_attention_workspace(ctypes.byref(largest), 0, ctypes.byref(size)) == 0, lib.igc_last_error()


def test_attention_scales_that_overflow_in_base_2(lib):
    # Finite, but not times log2(e), which the kernels exponentiate with: every result would be NaN.
    p, size = ctypes.byref(_problem(scale=3e38)), ctypes.c_size_t(0)
    _refused(lib, INVALID, lib.igc_cross_attention_workspace(p, 0, ctypes.byref(size)), b"scale must be positive, and finite times")
    assert lib.igc_cross_attention_workspace(ctypes.byref(_problem(scale=2e38)), 0, ctypes.byref(size)) == 0


def test_attention_workspaces_are_aligned(lib):
    # 1 query, 1 head of 33 channels, 1000 keys in 3 parts: 99 partial results, then 3 pairs of statistics that are read as
    # pairs, from the next multiple of 16 bytes on.
    size = ctypes.c_size_t(0)
    odd = ctypes.byref(_problem(dtype=0, n_q=1, n_k=1000, heads=1, kv_heads=1, dim=33))
    assert lib.igc_cross_attention_workspace(odd, 0, ctypes.byref(size)) == 0
    assert size.value == 4 * (100 + 3 * 2)
    off = ctypes.c_void_p(8192 + 4)
    _refused(lib, INVALID, lib.igc_cross_attention(odd, P, P, P, Q, Q, off, 1 << 30, None), b"d_ws must be aligned to 16 bytes")
    p = ctypes.byref(_problem())
    _refused(lib, INVALID, lib.igc_cross_attention_backward(p, P, P, P, P, P, P, Q, Q, Q, off, 1 << 30, None),
             b"d_ws must be aligned to 16 bytes")


def test_attention_operands(lib):
    p = ctypes.byref(_problem())
    _refused(lib, INVALID, lib.igc_cross_attention(None, P, P, P, Q, Q, None, 0, None), b"problem")
    _refused(lib, INVALID, lib.igc_cross_attention(p, None, P, P, Q, Q, None, 0, None), b"d_q")
    _refused(lib, INVALID, lib.igc_cross_attention(p, P, None, P, Q, Q, None, 0, None), b"d_k")
    _refused(lib, INVALID, lib.igc_cross_attention(p, P, P, P, P, Q, None, 0, None), b"aliases")
    few = ctypes.byref(_problem(n_q=1, n_k=100000))
    _refused(lib, CAPACITY, lib.igc_cross_attention(few, P, P, P, Q, Q, None, 0, None), b"workspace")
    _refused(lib, INVALID, lib.igc_cross_attention_backward(p, P, P, P, P, P, None, Q, Q, Q, Q, 1 << 40, None), b"d_dout")
    _refused(lib, INVALID, lib.igc_cross_attention_backward(p, P, P, P, P, P, P, Q, Q, None, Q, 1 << 40, None), b"together")
    _refused(lib, INVALID, lib.igc_cross_attention_backward(p, P, P, P, P, P, P, P, Q, Q, Q, 1 << 40, None), b"aliases")
    _refused(lib, CAPACITY, lib.igc_cross_attention_backward(p, P, P, P, P, P, P, Q, Q, Q, Q, 8, None), b"workspace")
    none = ctypes.byref(_problem(n_q=0, n_k=0))
    assert lib.igc_cross_attention(none, None, None, None, None, None, None, 0, None) == 0
    assert lib.igc_cross_attention_backward(none, None, None, None, None, None, None, None, None, None, None, 0, None) == 0


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import sparse_convolution_amd as igc
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="x must be a CUDA"):
        igc.layer_norm(x)
    with pytest.raises(ValueError, match="shape"):
        igc.layer_norm(torch.zeros(8))
    with pytest.raises(TypeError, match="unsupported dtype"):
        igc.checkpoint_pack(x.double())
    with pytest.raises(TypeError, match="codes must be a CUDA"):
        igc.Checkpoint8(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1))
    with pytest.raises(TypeError, match="unsupported dtype"):
        igc.Checkpoint8(torch.zeros(4, 8, dtype=torch.int8), torch.zeros(4, 1), torch.float16)
    with pytest.raises(TypeError, match="q must be a CUDA"):
        igc.cross_attention(torch.zeros(4, 2, 8), torch.zeros(4, 2, 8), torch.zeros(4, 2, 8))


@pytest.mark.gpu
def test_binding_refuses_wrong_device_operands():
    from tests._gpu import require_gpu
    require_gpu()
    import sparse_convolution_amd as igc
    x = torch.zeros(4, 8, device="cuda")
    with pytest.raises(ValueError, match="contiguous"):
        igc.layer_norm(x.t())
    with pytest.raises(ValueError, match="weight must have shape"):
        igc.layer_norm(x, torch.zeros(7, device="cuda"))
    with pytest.raises(TypeError, match="float32 or"):
        igc.layer_norm(x, torch.zeros(8, device="cuda", dtype=torch.bfloat16))
    with pytest.raises(TypeError, match="bias must have dtype"):
        igc.layer_norm(x.bfloat16(), torch.zeros(8, device="cuda"), torch.zeros(8, device="cuda", dtype=torch.bfloat16))
    y, mean, rstd = igc.layer_norm(x)
    with pytest.raises(TypeError, match="dy must have dtype"):
        igc.layer_norm_backward(x.bfloat16(), x, mean, rstd)
    with pytest.raises(ValueError, match="rstd must have shape"):
        igc.layer_norm_backward(x, x, mean, rstd[:2])
    with pytest.raises(ValueError, match="scales must have shape"):
        igc.Checkpoint8(torch.zeros(4, 80, dtype=torch.int8, device="cuda"), torch.zeros(4, 1, device="cuda"))
    q, k = torch.zeros(6, 4, 16, device="cuda"), torch.zeros(5, 2, 16, device="cuda")
    off = torch.tensor([0, 6], dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError, match="multiple"):
        igc.cross_attention(q[:, :3], k, k)
    with pytest.raises(ValueError, match="k and v must have shape"):
        igc.cross_attention(q, k, k[:, :1])
    with pytest.raises(ValueError, match="contiguous along"):
        igc.cross_attention(q.transpose(1, 2), k, k)
    with pytest.raises(ValueError, match="come together"):
        igc.cross_attention(q, k, k, q_offsets=off)
    with pytest.raises(TypeError, match="q_offsets must have dtype"):
        igc.cross_attention(q, k, k, off.long(), off)
    with pytest.raises(ValueError, match="key_mask must have shape"):
        igc.cross_attention(q, k, k, key_mask=torch.ones(4, dtype=torch.bool, device="cuda"))
    with pytest.raises(ValueError, match="out must have shape"):
        igc.cross_attention_backward(q, q, k, k, q[:3], torch.zeros(6, 4, device="cuda"))
    with pytest.raises(igc.IgcError, match="at most 128"):
        igc.cross_attention(torch.zeros(6, 1, 136, device="cuda"), torch.zeros(5, 1, 136, device="cuda"), torch.zeros(5, 1, 136, device="cuda"))
