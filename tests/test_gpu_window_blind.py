"""Rows that a key mask leaves without keys: whatever they hold, NaN and infinities too, they give zeros and -infinity, and nothing of them
reaches other rows or keys, forward or backward (left-padded batches, padded sequences)."""
import pytest
import torch

from tests._gpu import require_gpu, say
from tests.test_gpu_attention import _case

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _run(dev, args, qo, ko, mask):
    import sparse_convolution_amd as igc
    q, k, v, do = dev
    out, lse = igc.window_attention(q, k, v, *args, qo, ko, mask)
    return (out, lse, *igc.window_attention_backward(do, q, k, v, out, lse, *args, qo, ko, mask))


# Lengths and how many rows of padding each sequence starts with (all of them: a padded sequence).
BATCHES = [([300, 77, 40], [130, 5, 40]), ([9001, 9200], [3001, 64]), ([1] * 5, [0, 1, 0, 1, 0]), ([2500], [1100])]


@pytest.mark.parametrize("dim", [20, 32, 40, 64, 96, 128])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lengths,padding", BATCHES)
def test_left_padding_may_hold_anything(lengths, padding, dtype, dim):
    say(f"window blind {lengths[:4]} {padding[:4]} {dtype} dim={dim}")
    for heads, args in ((4, (60, 0, 3)), (2, (None, 0, 0)) if sum(lengths) < 5000 else (2, (40, 0, 0))):
        dev, (qo, ko), _ = _case(lengths, lengths, heads, 2, dim, dtype)
        blind = torch.cat([torch.arange(n) < p for n, p in zip(lengths, padding)]).cuda()
        clean = [t.clone() for t in dev]
        for t in clean:
            t[blind] = 0
        for bad in (float("nan"), float("inf"), -float("inf")):
            dirty = [t.clone() for t in dev]
            for t in dirty:
                t[blind] = bad
            got, want = _run(dirty, args, qo, ko, ~blind), _run(clean, args, qo, ko, ~blind)
            for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), got, want):
                assert torch.equal(a, b), (name, bad)
                assert bool((a[blind] == (0 if name != "lse" else -float("inf"))).all()), (name, bad)
                assert bool(torch.isfinite(a[~blind]).all()), (name, bad)


@pytest.mark.parametrize("dtype,dim", [(F32, 32), (F32, 128), (BF16, 64), (BF16, 128)])
def test_a_row_that_sees_keys_is_not_hidden(dtype, dim):
    # NaN in a query that sees a key is NaN in its row, and in no other's.
    import sparse_convolution_amd as igc
    say(f"window not hidden {dtype} dim={dim}")
    for n, left in ((200, 30), (9001, 30), (2500, 2000)):
        dev, _, mask = _case([n], [n], 2, 2, dim, dtype, masked=0.2)
        q, k, v, _ = dev
        out, lse = igc.window_attention(q, k, v, left, 0, 1, key_mask=mask)
        sees = torch.isfinite(lse).all(1).nonzero().flatten()
        row = int(sees[len(sees) // 2])
        for bad in (float("nan"), float("inf")):
            q2 = q.clone()
            q2[row, 1, 3] = bad
            out2, lse2 = igc.window_attention(q2, k, v, left, 0, 1, key_mask=mask)
            assert bool(torch.isnan(out2[row, 1]).all()) and bool(torch.isnan(lse2[row, 1]))
            out2[row, 1], lse2[row, 1] = out[row, 1], lse[row, 1]
            assert torch.equal(out2, out) and torch.equal(lse2, lse)
