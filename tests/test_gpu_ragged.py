"""Cross attention over offsets that leave rows out: before the first sequence, after the last one, or both.

Rows that no sequence covers take no part and their results are left unwritten; the rest equals the attention of the
covered slices alone, to the bounds of tests/test_gpu_attention.py.
"""
import ctypes

import pytest
import torch

from tests._gpu import require_gpu, say
from tests.test_gpu_attention import _case, _reference

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _offsets(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _lengths(off):
    o = off.tolist()
    return [b - a for a, b in zip(o, o[1:])]


# (query offsets, queries, key offsets, keys): single tokens, a few of them, tiles of the matrix kernels, a split key axis,
# a split query axis.
FIRST_ROWS = [([1, 2, 3], 3, [5, 70, 130], 130), ([4, 5, 6, 7], 7, [0, 20, 20, 60], 60), ([300, 400, 700], 700, [9, 80, 140], 140),
              ([257, 300], 300, [300, 420], 420), ([2, 3], 3, [1000, 4000], 4000), ([130, 200], 200, [1500, 4100], 4100),
              ([600, 4600], 4600, [31, 60], 60), ([0, 90, 200], 200, [129, 200, 300], 300)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("qo,nq,ko,nk", FIRST_ROWS)
def test_a_first_sequence_that_starts_late(qo, nq, ko, nk, dtype):
    import sparse_convolution_amd as igc
    say(f"attention offsets {qo} of {nq}, {ko} of {nk}, {dtype}")
    dev, _, _ = _case([nq], [nk], 4, 2, 32, dtype)
    q, k, v, do = dev
    qo, ko = _offsets(*qo), _offsets(*ko)
    out, lse = igc.cross_attention(q, k, v, qo, ko)
    dq, dk, dv = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko)
    torch.cuda.synchronize()
    qs, ks = slice(int(qo[0]), int(qo[-1])), slice(int(ko[0]), int(ko[-1]))
    r, b, rl = _reference([q[qs], k[ks], v[ks], do[qs]], _lengths(qo), _lengths(ko), None, 32 ** -0.5)
    got = lse[qs].double().cpu()
    fin = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(got), fin) and bool(((got - rl)[fin].abs() <= 2e-5 * (1 + rl[fin].abs())).all())
    for name, t in (("out", out[qs]), ("dq", dq[qs]), ("dk", dk[ks]), ("dv", dv[ks])):
        err = (t.double().cpu() - r[name]).abs()
        assert bool((err <= b[name]).all()), (name, float((err / b[name]).max()))


def _address(t):
    return ctypes.c_void_p(t.data_ptr())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,dim", [(4, 32), (2, 33)])
@pytest.mark.parametrize("qo,nq,ko,nk", FIRST_ROWS + [([0, 1], 4, [0, 2000], 2500), ([0, 60, 100], 150, [0, 900, 3000], 3300),
                                                      ([0, 3000], 3500, [0, 20], 50), ([0, 100], 160, [0, 90], 200), ([5, 5], 9, [3, 3], 7)])
def test_rows_of_no_sequence_are_left_unwritten(qo, nq, ko, nk, heads, dim, dtype):
    # Outputs filled with 7 and the workspace with NaN before the calls: what no sequence covers still holds 7, and
    # nothing else takes up the workspace's content.
    from sparse_convolution_amd import _lib
    lib = _lib.load()
    say(f"attention rows of no sequence, {qo} of {nq}, {ko} of {nk}, {heads} heads of {dim}, {dtype}")
    (q, k, v, do), _, _ = _case([nq], [nk], heads, 2, dim, dtype)
    qo, ko = _offsets(*qo), _offsets(*ko)
    pair = ctypes.c_int64 * 2
    p = _lib.Attention(dtype=int(dtype == BF16), batch=qo.numel() - 1, heads=heads, kv_heads=2, dim=dim, scale=dim ** -0.5, n_q=nq, n_k=nk,
                       q_stride=pair(heads * dim, dim), k_stride=pair(2 * dim, dim), v_stride=pair(2 * dim, dim),
                       d_q_offsets=qo.data_ptr(), d_kv_offsets=ko.data_ptr(), d_key_mask=None)

    def workspace(backward):
        size = ctypes.c_size_t(0)
        assert lib.igc_cross_attention_workspace(ctypes.byref(p), backward, ctypes.byref(size)) == 0
        return torch.full((size.value // 4 + 1,), float("nan"), device="cuda"), size.value

    out, lse = torch.full_like(q, 7), torch.full((nq, heads), 7.0, device="cuda")
    dq, dk, dv = torch.full_like(q, 7), torch.full_like(k, 7), torch.full_like(v, 7)
    stream = ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)
    ws, size = workspace(0)
    assert lib.igc_cross_attention(ctypes.byref(p), _address(q), _address(k), _address(v), _address(out), _address(lse), _address(ws), size,
                                   stream) == 0
    ws, size = workspace(1)
    assert lib.igc_cross_attention_backward(ctypes.byref(p), _address(q), _address(k), _address(v), _address(out), _address(lse),
                                            _address(do), _address(dq), _address(dk), _address(dv), _address(ws), size, stream) == 0
    torch.cuda.synchronize()
    for name, t, off in (("out", out, qo), ("lse", lse, qo), ("dq", dq, qo), ("dk", dk, ko), ("dv", dv, ko)):
        lo, hi = int(off[0]), int(off[-1])
        assert bool((t[:lo] == 7).all()) and bool((t[hi:] == 7).all()), name
        assert not bool(t[lo:hi].isnan().any()), name
