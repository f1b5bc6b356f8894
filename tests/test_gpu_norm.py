"""Layer norm and its gradients against the formulas in float64.

Tolerances. Forward: the kernel sums a row in fp32 in a tree over at least four lanes' partial sums, so the
mean of values of magnitude m is off by at most about (c / lanes + 8) 2^-24 m, a few 1e-6 of the row's
largest value for these sizes; times rstd that is 1e-5 of (max |x| rstd + 1) max |w| with room. bf16 results
add their own rounding, 2^-8 of each value (8 significant bits). Input gradient: the same sums over g and g xhat, 1e-5 of
rstd (max |g|) (1 + max |xhat|)^2 of the row. Weight gradients: fp32 sums over the rows of a lane, then fp64:
an error of sqrt(rows) roundings at most, 1e-5 of the sum of the magnitudes.
"""
import numpy as np
import pytest
import torch

from tests._gpu import require_gpu, say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
HALF_ULP = {F32: 0.0, BF16: 2.0 ** -8}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _igc():
    import sparse_convolution_amd as igc
    return igc


def _inputs(n, c, dtype, wdtype, seed, shift=0.3, offset=0):
    g = torch.Generator().manual_seed(seed)

    def place(t):  # the same values at an address `offset` elements into an allocation
        t = t.to(dtype)
        buf = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
        out = buf[offset:].view(t.shape)
        out.copy_(t)
        return out

    x = place(torch.randn(n, c, generator=g) * (0.5 + torch.rand(c, generator=g)) + shift)
    dy = place(torch.randn(n, c, generator=g))
    w = (1 + 0.2 * torch.randn(c, generator=g)).to(wdtype).cuda() if wdtype else None
    b = (0.2 * torch.randn(c, generator=g)).to(wdtype).cuda() if wdtype else None
    return x, dy, w, b


def _forward64(x, w, b, eps):
    x = x.double().cpu()
    mu = x.mean(1, keepdim=True)
    rs = 1.0 / torch.sqrt((x - mu).square().mean(1, keepdim=True) + eps)
    h = (x - mu) * rs
    y = h * (1 if w is None else w.double().cpu()) + (0 if b is None else b.double().cpu())
    return y, mu[:, 0], rs[:, 0], h


def _backward64(dy, h, rs, w):
    dy = dy.double().cpu()
    g = dy * (1 if w is None else w.double().cpu())
    dx = rs[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    return dx, (dy * h).sum(0), dy.sum(0), g


def check_forward(x, w, b, eps, y, mean, rstd):
    r, mu, rs, h = _forward64(x, w, b, eps)
    big = (x.double().abs().amax(1).cpu() * rs + 1)[:, None] * (1.0 if w is None else float(w.abs().max()))
    err = (y.double().cpu() - r).abs()
    assert bool((err <= HALF_ULP[x.dtype] * r.abs() + 1e-5 * big).all()), float((err / big).max())
    assert bool(((mean.double().cpu() - mu).abs() <= 1e-5 * x.double().abs().amax(1).cpu()).all())
    assert bool(((rstd.double().cpu() - rs).abs() <= 1e-5 * rs * big[:, 0].clamp(min=1) ** 1).all())


def check_backward(dy, h, rs, w, dx, dw, db):
    r, rw, rb, g = _backward64(dy, h, rs, w)
    big = (rs * g.abs().amax(1) * (1 + h.abs().amax(1)) ** 2)[:, None]
    err = (dx.double().cpu() - r).abs()
    assert bool((err <= HALF_ULP[dy.dtype] * r.abs() + 1e-5 * big).all()), float((err / (big + 1e-30)).max())
    if dw is not None:
        d64 = dy.double().cpu()
        # xhat itself carries the forward's error, up to 1e-5 of its size
        assert bool(((dw.double().cpu() - rw).abs() <= 2e-5 * (d64.abs() * (h.abs() + 1)).sum(0) + 1e-30).all())
        assert bool(((db.double().cpu() - rb).abs() <= 1e-5 * d64.abs().sum(0) + 1e-30).all())


SHAPES = [(1, 1), (7, 1), (1, 8), (5, 3), (130, 7), (7130, 8), (1001, 20), (257, 36), (1025, 64), (77, 65), (33, 96), (513, 100),
          (999, 128), (300, 255), (1030, 256), (65, 300), (129, 512), (40, 516), (31, 1000), (17, 1024), (9, 1025), (21, 1032),
          (13, 2048), (6, 2049), (10, 4095), (5, 4096), (40003, 64), (20011, 33)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,c", SHAPES)
def test_forward_and_gradients(n, c, dtype):
    igc = _igc()
    say(f"layer norm n={n} c={c} {dtype}")
    x, dy, w, b = _inputs(n, c, dtype, dtype, n + c)
    y, mean, rstd = igc.layer_norm(x, w, b, eps=1e-5)
    dx, dw, db = igc.layer_norm_backward(dy, x, mean, rstd, w)
    torch.cuda.synchronize()
    assert y.dtype == dtype and dx.dtype == dtype and dw.dtype == F32 and db.shape == (c,)
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    check_backward(dy, h.cpu(), rstd.double().cpu(), w, dx, dw, db)


@pytest.mark.parametrize("dtype,wdtype", [(BF16, F32), (BF16, None), (F32, None)])
@pytest.mark.parametrize("c,offset", [(64, 0), (64, 1), (128, 4), (24, 2), (200, 3)])
def test_parameter_types_and_unaligned_rows(c, offset, dtype, wdtype):
    igc = _igc()
    say(f"layer norm c={c} offset={offset} {dtype} weights {wdtype}")
    x, dy, w, b = _inputs(301, c, dtype, wdtype, c, offset=offset)
    y, mean, rstd = igc.layer_norm(x, w, b)
    dx, dw, db = igc.layer_norm_backward(dy, x, mean, rstd, w)
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    h = (x.double() - mean.double()[:, None]) * rstd.double()[:, None]
    check_backward(dy, h.cpu(), rstd.double().cpu(), w, dx, dw, db)
    only, none_w, none_b = igc.layer_norm_backward(dy, x, mean, rstd, w, need_dweight=False)
    assert none_w is None and none_b is None and torch.equal(only, dx)


def test_rows_of_one_value_and_far_from_zero():
    # A constant row has variance 0: y = b, rstd = 1 / sqrt(eps), and only its own row is affected; a row
    # at 1000 times its spread keeps its variance (summed around the mean, not from squares).
    igc = _igc()
    x = torch.randn(64, 96, generator=torch.Generator().manual_seed(5))
    x[3] = 2.5
    x[10] = 1000.0 + x[10]
    x = x.cuda()
    b = torch.randn(96, generator=torch.Generator().manual_seed(6)).cuda()
    y, mean, rstd = igc.layer_norm(x, None, b, eps=1e-5)
    assert torch.equal(y[3], b) and abs(float(rstd[3]) - 1e-5 ** -0.5) < 1e-3
    check_forward(x, None, b, 1e-5, y, mean, rstd)


@pytest.mark.parametrize("c", [8, 64, 130, 1040])
def test_a_row_with_infinity_or_nan_stays_in_its_row(c):
    igc = _igc()
    x, dy, w, b = _inputs(70, c, F32, F32, 9)
    clean = igc.layer_norm(x, w, b)
    grads = igc.layer_norm_backward(dy, x, clean[1], clean[2], w)
    x[5, c // 2] = float("nan")
    x[6, 0] = float("inf")
    y, mean, rstd = igc.layer_norm(x, w, b)
    dx, _, _ = igc.layer_norm_backward(dy, x, mean, rstd, w)
    rest = [r for r in range(70) if r not in (5, 6)]
    assert torch.equal(y[rest], clean[0][rest]) and torch.equal(dx[rest], grads[0][rest])
    assert bool(torch.isnan(y[5:7]).all()) and bool(torch.isnan(dx[5:7]).all())


def test_no_rows():
    igc = _igc()
    x = torch.empty((0, 24), dtype=BF16, device="cuda")
    y, mean, rstd = igc.layer_norm(x)
    dx, dw, db = igc.layer_norm_backward(x, x, mean, rstd)
    assert y.shape == (0, 24) and dx.shape == (0, 24)
    assert bool((dw == 0).all()) and bool((db == 0).all()) and dw.shape == (24,)


def test_gradient_against_differences():
    # d/dt sum(y dy) along a direction u, central differences of the fp32 kernel summed in float64:
    # the step 2^-6 leaves an error of its square (2.4e-4) times third derivatives of order one, and
    # rounding of 2^-24 |y| sqrt(n c) / 2^-6, about 1e-4 here, against sums of order sqrt(n c) = 50.
    igc = _igc()
    n, c, t = 50, 48, 2.0 ** -6
    x, dy, w, b = _inputs(n, c, F32, F32, 21)
    _, mean, rstd = igc.layer_norm(x, w, b)
    dx, dw, db = igc.layer_norm_backward(dy, x, mean, rstd, w)

    def loss(xx, ww, bb):
        return float((igc.layer_norm(xx, ww, bb)[0].double() * dy.double()).sum())

    g = torch.Generator().manual_seed(22)
    u = torch.randn(n, c, generator=g).cuda()
    v = torch.randn(c, generator=g).cuda()
    for got, ref in (((dx.double() * u.double()).sum(), (loss(x + t * u, w, b) - loss(x - t * u, w, b)) / (2 * t)),
                     ((dw.double() * v.double()).sum(), (loss(x, w + t * v, b) - loss(x, w - t * v, b)) / (2 * t)),
                     ((db.double() * v.double()).sum(), (loss(x, w, b + t * v) - loss(x, w, b - t * v)) / (2 * t))):
        assert abs(float(got) - ref) <= 2e-3 * 50, (float(got), ref)


def test_other_stream_and_repeat_are_bit_identical():
    igc = _igc()
    x, dy, w, b = _inputs(30011, 96, BF16, BF16, 30)
    y, mean, rstd = igc.layer_norm(x, w, b)
    first = igc.layer_norm_backward(dy, x, mean, rstd, w)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        y2, mean2, rstd2 = igc.layer_norm(x, w, b)
        again = igc.layer_norm_backward(dy, x, mean2, rstd2, w)
    s.synchronize()
    assert torch.equal(y, y2)
    for a, e in zip(first, again):
        assert torch.equal(a, e)


def test_captured_in_a_graph():
    igc = _igc()
    x, dy, w, b = _inputs(5003, 64, BF16, F32, 31)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        igc.layer_norm_backward(dy, x, *igc.layer_norm(x, w, b)[1:], w)
    s.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y, mean, rstd = igc.layer_norm(x, w, b)
        dx, dw, db = igc.layer_norm_backward(dy, x, mean, rstd, w)
    for k in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(k)))
        g.replay()
        torch.cuda.synchronize()
        ry, rm, rr = igc.layer_norm(x, w, b)
        rx, rw, rb = igc.layer_norm_backward(dy, x, rm, rr, w)
        for a, e in ((y, ry), (dx, rx), (dw, rw), (db, rb)):
            assert torch.equal(a, e), k


def test_arrays_past_2_to_the_31_elements():
    igc = _igc()
    n, c = 2100001, 1024
    assert n * c > 2 ** 31
    x = torch.zeros(n, c, dtype=BF16, device="cuda")
    x[-500:] = torch.randn(500, c, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(BF16)
    y, mean, rstd = igc.layer_norm(x)
    yl, ml, rl = igc.layer_norm(x[-500:].contiguous())
    assert torch.equal(y[-500:], yl) and torch.equal(mean[-500:], ml) and torch.equal(rstd[-500:], rl)
    dx, dw, db = igc.layer_norm_backward(x, x, mean, rstd)
    dl, wl, bl = igc.layer_norm_backward(x[-500:].contiguous(), x[-500:].contiguous(), ml, rl)
    assert torch.equal(dx[-500:], dl)
    # All other rows are zero: the same sums, grouped differently (fp32 in a lane, fp64 across workgroups).
    assert float((dw - wl).abs().max()) <= 1e-5 * 500 and float((db - bl).abs().max()) <= 1e-5 * 500
    ck = igc.checkpoint_pack(x)
    assert torch.equal(igc.checkpoint_unpack(ck)[-500:], igc.checkpoint_unpack(igc.checkpoint_pack(x[-500:].contiguous())))


def test_more_rows_than_one_launch_has_threads_for():
    # 64 lanes a row and two rows a lane would be more than 2^32 threads, so the workgroups take more rows each (140 GB).
    igc = _igc()
    n, c, block = 135000003, 129, 1 << 20
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn(block, c, generator=g, device="cuda")
    x = torch.empty(n, c, device="cuda")
    for at in range(0, n, block):
        x[at:at + block] = rows[:min(block, n - at)]
    y, mean, rstd = igc.layer_norm(x)
    ry, rm, rr = igc.layer_norm(rows)
    last = (n - 1) // block * block
    for at in (0, last // 2 // block * block, last - block, last):
        k = min(block, n - at)
        assert torch.equal(y[at:at + k], ry[:k]) and torch.equal(mean[at:at + k], rm[:k]) and torch.equal(rstd[at:at + k], rr[:k])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("c", [1, 3, 8, 64, 130, 1040, 4096])
def test_statistics_of_a_row_with_infinity_or_nan(c, dtype):
    # By the definition: a NaN makes mean and rstd NaN; an infinity the mean infinite (of its sign) and rstd NaN, both signs
    # all NaN. The other rows keep theirs.
    igc = _igc()
    x, _, w, b = _inputs(40, c, dtype, dtype, 13)
    clean = igc.layer_norm(x, w, b)
    nan, inf = float("nan"), float("inf")
    x[3, c // 2], x[5, 0], x[8, c - 1] = nan, inf, -inf
    both = c > 1
    if both:
        x[9, 0], x[9, c - 1] = inf, -inf
    y, mean, rstd = igc.layer_norm(x, w, b)
    y8, ck, rstd8 = igc.layer_norm_checkpoint(x, w, b)
    bad = [3, 5, 8] + [9] * both
    assert bool(mean[3].isnan()) and float(mean[5]) == inf and float(mean[8]) == -inf and (not both or bool(mean[9].isnan()))
    for t in (rstd, rstd8, y, y8, igc.checkpoint_unpack(ck)):
        assert bool(t[bad].isnan().all())
    rest = [r for r in range(40) if r not in bad]
    assert torch.equal(mean[rest], clean[1][rest]) and torch.equal(rstd[rest], clean[2][rest]) and torch.equal(rstd8[rest], clean[2][rest])
