"""Cross attention over offsets that leave rows out: before the first sequence, after the last one, or both.

Rows that no sequence covers take no part; the rest equals the attention of the
covered slices alone, to the bounds of tests/test_gpu_attention.py.
"""
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
