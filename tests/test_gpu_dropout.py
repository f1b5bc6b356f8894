"""Dropout from a counter-based generator: the elements that stay against the generator in numpy, their values exactly or to
the fused sum's rounding."""
import numpy as np
import pytest
import torch

from tests._gpu import require_gpu, say

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _igc():
    import sparse_convolution_amd as igc
    return igc


def philox(counter, key):
    """Ten rounds on uint64 arrays [4, n] of 32-bit words."""
    c, (k0, k1) = [x.astype(np.uint64) for x in counter], key
    low = np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> np.uint64(32)) ^ c[1] ^ np.uint64(k0), b & low, (a >> np.uint64(32)) ^ c[3] ^ np.uint64(k1), a & low]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def bits(first, count, seed, offset):
    """16 bits of elements first .. first + count (first a multiple of 8)."""
    at = np.arange(first // 8, (first + count + 7) // 8, dtype=np.uint64)
    words = philox([at & np.uint64(0xFFFFFFFF), at >> np.uint64(32), np.full_like(at, offset & 0xFFFFFFFF), np.full_like(at, offset >> 32)],
                   (seed & 0xFFFFFFFF, seed >> 32))
    return np.stack([w >> np.uint64(s) & np.uint64(0xFFFF) for w in words for s in (0, 16)], 1).reshape(-1)[:count]


def test_generator_of_the_test_itself():
    # Known answers of the published generator (counter, key all zeros; all ones).
    for x, want in ((0, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"), (0xFFFFFFFF, "408f276d 41c83b0e a20bc7c6 6d5451fd")):
        got = philox([np.array([x], np.uint64)] * 4, (x, x))
        assert " ".join(f"{int(w[0]):08x}" for w in got) == want


def expected(x, p, seed, offset, residual):
    drop = round(65536 * p)
    keep = torch.from_numpy((bits(0, x.numel(), seed, offset) >= drop).reshape(x.shape))
    y = torch.where(keep, x.double().cpu() * (65536 / (65536 - drop) if drop < 65536 else 0.0), 0.0)
    return (y if residual is None else y + residual.double().cpu()), keep


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("shape", [(1,), (7,), (8,), (9, 1), (33, 5), (1000, 64), (4099, 33), (3, 5, 7), (300001,)])
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5, 0.999])
def test_values(shape, p, dtype):
    igc = _igc()
    say(f"dropout {shape} p={p} {dtype}")
    g = torch.Generator().manual_seed(sum(shape))
    x, r = torch.randn(shape, generator=g).to(dtype).cuda(), torch.randn(shape, generator=g).to(dtype).cuda()
    seed, offset = (1 << 63) + 12345, (1 << 40) + 7
    for residual in (None, r):
        want, keep = expected(x, p, seed, offset, residual)
        got = igc.dropout(x, p, seed, offset, residual)
        # The scale is rounded to fp32 and the product, or the fused sum, once: 2^-23 of the product; then the type's half step.
        size = want.abs() if residual is None else (want - residual.double().cpu()).abs()
        bound = 2.0 ** -23 * size + torch.finfo(dtype).eps / 2 * want.abs() * (1 + 2.0 ** -20)
        assert bool(((got.double().cpu() - want).abs() <= bound).all())
        if residual is None:
            assert bool((got.cpu()[~keep] == 0).all())
        else:
            assert torch.equal(got.cpu()[~keep], residual.cpu()[~keep])
    # The backward pass drops the same elements.
    assert torch.equal(igc.dropout_backward(x, p, seed, offset), igc.dropout(x, p, seed, offset))


def test_everything_dropped_and_special_values():
    igc = _igc()
    say("dropout special")
    x = torch.randn(1000).cuda()
    x[::3], x[1::3] = float("nan"), float("inf")
    assert bool((igc.dropout(x, 1.0, 5) == 0).all())
    r = torch.randn(1000).cuda()
    assert torch.equal(igc.dropout(x, 1.0, 5, residual=r), r)
    y, (_, keep) = igc.dropout(x, 0.5, 5).cpu(), expected(x, 0.5, 5, 0, None)
    assert bool((y[~keep] == 0).all()) and torch.equal(torch.isfinite(y[keep]), torch.isfinite(x.cpu()[keep]))
    assert torch.equal(igc.dropout(x[:0], 0.5, 5), x[:0])


def test_unaligned_addresses():
    igc = _igc()
    say("dropout unaligned")
    for dtype in (F32, BF16):
        base = torch.randn(5001, device="cuda").to(dtype)
        x = base[1:]
        assert torch.equal(igc.dropout(x, 0.3, 9, residual=x), igc.dropout(x.clone(), 0.3, 9, residual=x.clone()))


def test_seeds_offsets_and_rate():
    igc = _igc()
    say("dropout rates")
    x = torch.ones(1 << 20, device="cuda")
    kept = [igc.dropout(x, 0.25, s, o) > 0 for s, o in ((1, 0), (2, 0), (1, 1), ((1 << 32) + 1, 0), (1, 1 << 32))]
    for i, a in enumerate(kept):
        assert abs(float(a.float().mean()) - 0.75) < 5 * (0.25 * 0.75 / (1 << 20)) ** 0.5
        for b in kept[i + 1:]:  # independent: equal in 0.75^2 + 0.25^2 of the places
            assert abs(float((a == b).float().mean()) - 0.625) < 5 * (0.625 * 0.375 / (1 << 20)) ** 0.5


def test_count_on_the_device_in_a_graph():
    igc = _igc()
    say("dropout graph")
    x = torch.randn(10007, device="cuda").bfloat16()
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        igc.dropout(x, 0.2, 77, count)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = igc.dropout(x, 0.2, 77, count)
            dx = igc.dropout_backward(x, 0.2, 77, count)
            count += 1
    torch.cuda.synchronize()
    for step in range(4):
        graph.replay()
        torch.cuda.synchronize()
        eager = igc.dropout(x, 0.2, 77, step)
        assert torch.equal(y, eager) and torch.equal(dx, eager)
        assert int(count) == step + 1


def test_elements_past_2_to_the_32():
    igc = _igc()
    say("dropout of 2^32 + 4101 elements")
    n = (1 << 32) + 4101
    x = torch.ones(n, dtype=BF16, device="cuda")
    y = igc.dropout(x, 0.5, 3, 4)
    for first in (0, 1 << 31, (1 << 32) - 4096, (1 << 32)):
        count = min(4096, n - first)
        keep = torch.from_numpy(bits(first, count, 3, 4) >= 32768)
        assert torch.equal(y[first:first + count].cpu() > 0, keep)
    keep = torch.from_numpy(bits((1 << 32) + 4096, 5, 3, 4) >= 32768)
    assert torch.equal(y[-5:].cpu() > 0, keep)
