"""Window attention rounds no probability to bf16: out and dv are as exact as their own rounding allows.

A probability enters its products as two bf16 parts. The first leaves at most half a step, 2^-8 of it, and the second
half a step of that: 2^-16. So out is off by its own rounding (2^-8 of its value), by 2^-16 sum p |v| and by the fp32 chain of scores,
exponentials and sums (F sum p |v|, as in tests/test_gpu_attention.py); dv the same with the rows' dout. One bf16 part
would add 2^-8 sum p |v|.
"""
import pytest
import torch

from tests._gpu import require_gpu, say
from tests.test_gpu_attention import F, _case
from tests.test_gpu_window import visible

pytestmark = pytest.mark.gpu

U = 2.0 ** -8
PARTS = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dim", [20, 32, 64, 96, 128])
@pytest.mark.parametrize("lengths,left,right,sinks,masked", [
    ([300, 77], 64, 64, 4, 0.0),       # few tiles: two waves on a row's axis
    ([2500], 1500, 0, 0, 0.2),         # the axis in parts
    ([9001, 9200], 40, 9, 2, 0.0),     # many tiles
    ([9001, 9200], 40, 0, 70, 0.2)])   # and sinks past the window
def test_out_and_dv_are_off_by_their_own_rounding_alone(lengths, left, right, sinks, masked, dim):
    import sparse_convolution_amd as igc
    heads, kv_heads = 4, 2
    say(f"window rounding {lengths} {left} {right} {sinks} masked={masked} dim={dim}")
    dev, (qo, ko), mask = _case(lengths, lengths, heads, kv_heads, dim, torch.bfloat16, masked=masked)
    q, k, v, do = dev
    out, lse = igc.window_attention(q, k, v, left, right, sinks, qo, ko, mask)
    _, _, dv = igc.window_attention_backward(do, q, k, v, out, lse, left, right, sinks, qo, ko, mask, need_dq=False)
    first = 0
    for n in lengths:
        rows = slice(first, first + n)
        see = visible(n, n, left, right, sinks)
        if mask is not None:
            see &= mask[rows].bool().cpu()
        first += n
        see = see.cuda()
        for kh in range(kv_heads):
            kk, vv = k[rows, kh].double(), v[rows, kh].double()
            grad, bound = torch.zeros_like(vv), torch.zeros_like(vv)
            for h in (2 * kh, 2 * kh + 1):
                s = (q[rows, h].double() @ kk.T * dim ** -0.5).masked_fill_(~see, -torch.inf)
                p = torch.softmax(s, 1).masked_fill_(~see.any(1, keepdim=True), 0.0)
                want, size, d = p @ vv, p @ vv.abs(), do[rows, h].double()
                err = (out[rows, h].double() - want).abs()
                assert bool((err <= U * want.abs() + (PARTS + F) * (1 + U) * size + 1e-9).all()), float((err / size).max())
                grad += p.T @ d
                bound += p.T @ d.abs()
            err = (dv[rows, kh].double() - grad).abs()
            assert bool((err <= U * grad.abs() + (PARTS + F) * (1 + U) * bound + 1e-9).all()), float((err / bound).max())
