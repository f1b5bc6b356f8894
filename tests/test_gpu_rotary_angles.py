"""Rotations by far positions and high frequencies against angles in integers."""
import numpy as np
import pytest
import torch

from tests._gpu import require_gpu, say
from tests.test_gpu_qk import E

pytestmark = pytest.mark.gpu

PI = 31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679  # 10^100 pi
INVERSE = (10 ** 100 << 400) // (2 * PI)  # 2^400 / (2 pi)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _turned(exponents, seed):
    import sparse_convolution_amd as igc
    g = torch.Generator().manual_seed(seed)
    pos = torch.cat([torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31]), torch.randint(-2 ** 31, 2 ** 31 - 1, (295,), generator=g)]).int()
    freq = (2.0 ** torch.tensor(exponents).double() * (1 + torch.rand(len(exponents), generator=g).double())).float()
    x = torch.randn(300, 2, 2 * len(exponents), generator=g)
    return pos, freq, x, igc.rotary(x.cuda(), pos.cuda(), freq.cuda()).double().cpu()


def test_high_frequencies_of_far_positions():
    say("rotary of high frequencies")
    pos, freq, x, got = _turned([0, 10, 19, 20, 21, 22, 24, 28, 31, 35, 39], 3)
    n = freq.numel()
    turns = torch.empty(300, n, dtype=torch.float64)
    for j in range(n):
        m, e = np.frexp(np.float64(freq[j].item()))
        m, shift = int(m * 2 ** 24), 400 - (int(e) - 24)
        for i in range(300):
            turns[i, j] = (int(pos[i]) * m * INVERSE % (1 << shift)) / (1 << shift)
    c, s = torch.cos(2 * np.pi * turns)[:, None], torch.sin(2 * np.pi * turns)[:, None]
    a, b = x.double()[..., :n], x.double()[..., n:]
    r, size = torch.cat([a * c - b * s, b * c + a * s], 2), torch.cat([a.abs() + b.abs()] * 2, 2)
    # The bound of tests/test_gpu_qk.py: six roundings to fp32.
    assert bool(((got - r).abs() <= 6 * E * size).all()), float(((got - r).abs() / size).max() / E)


def test_frequencies_beyond_stay_rotations():
    # No angle is exact there, but a pair keeps its length (to six roundings) and is finite.
    say("rotary of frequencies beyond")
    _, freq, x, got = _turned([50, 70, 90, 120, 127], 4)
    n = freq.numel()
    was, now = x[..., :n].double() ** 2 + x[..., n:].double() ** 2, got[..., :n] ** 2 + got[..., n:] ** 2
    assert bool(torch.isfinite(got).all()) and bool(((now - was).abs() <= 4 * 6 * E * was).all()), float(((now - was).abs() / was).max() / E)
