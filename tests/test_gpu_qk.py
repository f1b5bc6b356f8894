"""Norm of queries and keys with the rotation by positions, and its gradients, against the formulas in float64.

Tolerances bound each element, counted in roundings of fp32 (e = 2^-24). u is half a step of the data's type.
  y:  the sum of squares takes up to 12 e (8 in a lane, 4 across lanes), halved by the root, which adds 2; two products for z; cosine and
      sine 2 e each, the amplitude one, two for the pair's sum: below 16 e of amplitude (|z1| + |z2|), plus u |y|.
  dx: rstd (h - xhat m), m = mean(h xhat): g 5 e, the dot product 12, rstd 8 and its products: below 64 e of
      rstd (|h| + |xhat| mean(|h| |xhat|)) with |h| formed from |dy1| + |dy2|, plus u |dx|.
  dw: 13 e a term, up to 40 sums in a lane and 8 across lanes and waves: below 64 e of the sum of magnitudes.
"""
import numpy as np
import pytest
import torch

from tests._gpu import require_gpu, say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
E = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _igc():
    import sparse_convolution_amd as igc
    return igc


def u(dtype):
    return torch.finfo(dtype).eps / 2


def turn(z, positions, frequencies, layout, amplitude, back=False, size=False):
    """The rotation in float64; size: magnitudes instead of sums."""
    if frequencies is None:
        return z.abs() if size else z
    f = frequencies.double().cpu()
    angle = torch.stack([positions.double().cpu()[:, a, None] * f[a] for a in range(f.shape[0])], 1).reshape(len(z), 1, -1)
    c, s = torch.cos(angle) * amplitude, torch.sin(angle) * amplitude * (-1 if back else 1)
    p = f.numel()
    i, j = (slice(0, p), slice(p, 2 * p)) if layout == "half" else (slice(0, 2 * p, 2), slice(1, 2 * p, 2))
    y = z.abs() if size else z.clone()
    if size:
        y[..., i] = y[..., j] = abs(amplitude) * (z[..., i].abs() + z[..., j].abs())
    else:
        y[..., i], y[..., j] = z[..., i] * c - z[..., j] * s, z[..., j] * c + z[..., i] * s
    return y


def case(n, heads, kv_heads, dim, axes, pairs, dtype, wdtype=F32, packed=True, reach=3000, seed=0, weights=True):
    g = torch.Generator().manual_seed(seed * 101 + n + 7 * dim + heads)
    if packed:  # slices of one projection, between values that must not be read
        buf = torch.full((n, heads + kv_heads + 1, dim + (3 if packed == "odd" else 0)), float("nan"), dtype=dtype)
        buf[:, :heads + kv_heads, :dim] = torch.randn(n, heads + kv_heads, dim, generator=g).to(dtype)
        buf = buf.cuda()
        q, k = buf[:, :heads, :dim], buf[:, heads:heads + kv_heads, :dim]
    else:
        q, k = torch.randn(n, heads, dim, generator=g).to(dtype).cuda(), torch.randn(n, kv_heads, dim, generator=g).to(dtype).cuda()
    pos = torch.randint(-reach, reach, (n, axes), generator=g, dtype=torch.int64).int().cuda() if axes else None
    freq = torch.stack([10000.0 ** (-torch.arange(pairs) / pairs) * (1 + 0.3 * a) for a in range(axes)]).float().cuda() if axes else None
    w = [(1 + 0.2 * torch.randn(dim, generator=g)).to(wdtype).cuda() if weights else None for _ in range(2)]
    dy = [torch.randn(n, h, dim, generator=g).to(dtype).cuda() for h in (heads, kv_heads)]
    return q, k if kv_heads else None, pos, freq, w, dy


def check(n, heads, kv_heads, dim, axes, pairs, dtype, layout="half", amplitude=1.0, eps=1e-6, **kw):
    igc = _igc()
    say(f"qk n={n} heads={heads}/{kv_heads} dim={dim} axes={axes}x{pairs} {layout} {dtype} {kw}")
    q, k, pos, freq, w, dy = case(n, heads, kv_heads, dim, axes, pairs, dtype, **kw)
    got = igc.qk_norm_rotary(q, k, pos, freq, w[0], w[1], eps, layout, amplitude)
    grads = igc.qk_norm_rotary_backward(dy[0], dy[1] if kv_heads else None, q, k, pos, freq, w[0], w[1], eps, layout, amplitude)
    torch.cuda.synchronize()
    for t, x in enumerate((q, k)):
        if x is None:
            assert got[t] is None and grads[t] is None and grads[2 + t] is None
            continue
        assert got[t].is_contiguous() and got[t].dtype == dtype and got[t].shape == x.shape
        xd, wd = x.double().cpu(), torch.ones(dim, dtype=torch.float64) if w[t] is None else w[t].double().cpu()
        r = (xd.square().mean(2, keepdim=True) + eps).rsqrt()
        y = turn(xd * r * wd, pos, freq, layout, amplitude)
        bound = 16 * E * turn(xd * r * wd, pos, freq, layout, amplitude, size=True) + u(dtype) * y.abs()
        err = (got[t].double().cpu() - y).abs()
        assert bool((err <= bound + 1e-30).all()), (t, float((err / bound).max()))
        d = dy[t].double().cpu()
        g, size = turn(d, pos, freq, layout, amplitude, back=True), turn(d, pos, freq, layout, amplitude, size=True)
        h, xhat = g * wd, xd * r
        dx = r * (h - xhat * (h * xhat).mean(2, keepdim=True))
        hs = size * wd.abs()
        bound = 64 * E * r * (hs + xhat.abs() * (hs * xhat.abs()).mean(2, keepdim=True)) + u(dtype) * dx.abs()
        err = (grads[t].double().cpu() - dx).abs()
        assert grads[t].is_contiguous() and bool((err <= bound + 1e-30).all()), (t, float((err / bound).max()))
        err = (grads[2 + t].double().cpu() - (g * xhat).sum((0, 1))).abs()
        bound = 64 * E * (size * xhat.abs()).sum((0, 1))
        assert grads[2 + t].dtype == F32 and bool((err <= bound + 1e-30).all()), (t, float((err / bound).max()))
    return got, grads


SHAPES = [(1, 0, 0), (2, 1, 1), (3, 1, 1), (7, 1, 3), (8, 1, 4), (8, 3, 1), (16, 1, 8), (20, 3, 3), (32, 3, 5), (33, 1, 16), (40, 1, 20),
          (40, 2, 10), (64, 3, 10), (64, 1, 16), (96, 3, 16), (100, 1, 33), (126, 1, 63), (127, 2, 31), (128, 1, 64), (128, 3, 21)]


@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("dim,axes,pairs", SHAPES)
def test_head_shapes(dim, axes, pairs, dtype, layout):
    check(67, 3, 2, dim, axes, pairs, dtype, layout, amplitude=1.25)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,heads,kv_heads", [(1, 1, 1), (1, 8, 2), (2, 70, 1), (31, 1, 0), (33, 4, 4), (257, 8, 8), (5001, 2, 1), (4099, 16, 4)])
def test_rows_and_heads(n, heads, kv_heads, dtype):
    check(n, heads, kv_heads, 64, 3, 10, dtype)
    check(n, heads, kv_heads, 32, 1, 16, dtype, "interleaved")


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("kw", [dict(packed="odd"), dict(packed=False), dict(wdtype=None), dict(weights=False)])
def test_strides_and_weights(kw, dtype):
    if "wdtype" in kw:
        kw = dict(wdtype=dtype)
    check(130, 4, 2, 64, 1, 32, dtype, **kw)
    check(130, 4, 2, 40, 1, 10, dtype, "interleaved", **kw)


@pytest.mark.parametrize("eps", [0.0, 1e-6, 0.1])
def test_norm_alone(eps):
    check(300, 2, 2, 48, 0, 0, BF16, eps=eps)
    check(301, 1, 3, 24, 0, 0, F32, eps=eps)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotation_alone(layout, dtype):
    igc = _igc()
    for dim, axes, pairs in ((48, 3, 8), (64, 1, 11), (9, 1, 4)):
        say(f"rotary dim={dim} {layout} {dtype}")
        q, _, pos, freq, _, dy = case(1003, 3, 1, dim, axes, pairs, dtype, packed="odd")
        y, dx = igc.rotary(q, pos, freq, layout, 1.5), igc.rotary_backward(dy[0], pos, freq, layout, 1.5)
        for got, x, back in ((y, q, False), (dx, dy[0], True)):
            r = turn(x.double().cpu(), pos, freq, layout, 1.5, back)
            bound = 6 * E * turn(x.double().cpu(), pos, freq, layout, 1.5, size=True) + u(dtype) * r.abs()
            assert bool(((got.double().cpu() - r).abs() <= bound).all())


def test_far_positions_and_any_frequency():
    # Angles of up to 2^31 * 3 radians and beyond, reduced exactly; 1-d positions and frequencies.
    igc = _igc()
    say("rotary of far positions")
    g = torch.Generator().manual_seed(5)
    pos = torch.tensor([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 1, 123456789], dtype=torch.int32)
    pos = torch.cat([pos, torch.randint(-2 ** 31, 2 ** 31 - 1, (993,), generator=g).int()])
    freq = torch.cat([torch.tensor([1.0, 3.0, 0.5, 1e-4, 1e-8, 700.0]), torch.rand(10, generator=g) * 2]).float()
    x = torch.randn(1000, 2, 32, generator=g)
    got = igc.rotary(x.cuda(), pos.cuda(), freq.cuda()).double().cpu()
    # The angle in integers: frequency = m 2^e exactly, position * m below 2^55, taken modulo a turn with 1 / (2 pi) to 200 bits.
    pi = 31415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679  # 10^100 pi
    inverse = (10 ** 100 << 400) // (2 * pi)  # 2^400 / (2 pi)
    turns = torch.empty(1000, 16, dtype=torch.float64)
    for j in range(16):
        m, e = np.frexp(np.float64(freq[j].item()))
        m, e = int(m * 2 ** 24), int(e) - 24
        for i in range(1000):
            t = int(pos[i]) * m * inverse
            shift = 400 - e
            turns[i, j] = (t % (1 << shift)) / (1 << shift)
    c, s = torch.cos(2 * np.pi * turns)[:, None], torch.sin(2 * np.pi * turns)[:, None]
    a, b = x.double()[..., :16], x.double()[..., 16:]
    r = torch.cat([a * c - b * s, b * c + a * s], 2)
    size = torch.cat([a.abs() + b.abs()] * 2, 2)
    assert bool(((got - r).abs() <= 6 * E * size).all()), float(((got - r).abs() / size).max() / E)


def test_rows_of_zeros_and_not_finite():
    igc = _igc()
    say("qk special rows")
    x = torch.randn(40, 2, 16)
    x[3] = 0
    x[5, 1, 2] = float("inf")
    x[6, 0, 3] = float("nan")
    w = torch.ones(16).cuda()
    freq = igc.rotary_frequencies(8).cuda()
    pos = torch.arange(40, dtype=torch.int32).cuda()
    y, _ = igc.qk_norm_rotary(x.cuda(), None, pos, freq, w)
    assert bool((y[3] == 0).all())
    bad = torch.zeros(40, 2, dtype=torch.bool)
    bad[5, 1] = bad[6, 0] = True
    assert torch.equal(torch.isfinite(y.cpu()).all(2), ~bad)  # no other head, and no row beside them
    # Without the norm channels behind the pairs pass whatever they hold, and the pairs beside them stay finite.
    for layout in ("half", "interleaved"):
        x[7, 0, 8], x[7, 0, 15] = float("inf"), float("-inf")
        z = igc.rotary(x.cuda(), pos, freq, layout).cpu()
        assert torch.equal(z[7, 0, 8:], x[7, 0, 8:]) and bool(torch.isfinite(z[7, 0, :8]).all())


def test_eps_zero_and_a_ragged_last_tile():
    # Rows behind the last one add nothing to the weights' gradient, not even 0 * infinity.
    igc = _igc()
    say("qk eps 0")
    x, dy = torch.randn(5, 1, 8).cuda(), torch.randn(5, 1, 8).cuda()
    _, _, dw, _ = igc.qk_norm_rotary_backward(dy, None, x, None, eps=0.0)
    assert bool(torch.isfinite(dw).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_rows_behind_the_last_do_not_meet_what_other_kernels_left(dtype):
    # Tables full of NaN, left by a call with such frequencies on every CU, and then tiles whose last rows have no table.
    igc = _igc()
    say(f"qk stale tables {dtype}")
    many, pos = torch.randn(200000, 1, 64, device="cuda").to(dtype), torch.ones(200000, dtype=torch.int32, device="cuda")
    for n in (5, 4099):
        q, k, p, freq, w, dy = case(n, 16, 4, 64, 3, 10, dtype)
        igc.rotary(many, pos, torch.full((32,), float("nan"), device="cuda"))
        grads = igc.qk_norm_rotary_backward(dy[0], dy[1], q, k, p, freq, w[0], w[1])
        y = igc.qk_norm_rotary(q, k, p, freq, w[0], w[1])
        assert all(bool(torch.isfinite(t).all()) for t in grads + y)


def test_no_rows():
    igc = _igc()
    x = torch.empty(0, 2, 16, device="cuda")
    y, k = igc.qk_norm_rotary(x, x)
    assert y.shape == k.shape == (0, 2, 16)
    dq, dk, dw, dkw = igc.qk_norm_rotary_backward(x, x, x, x)
    assert dq.shape == (0, 2, 16) and bool((dw == 0).all()) and bool((dkw == 0).all())
    torch.cuda.synchronize()


def test_gradient_against_differences():
    # Central differences of sum(y * dy) in fp32 along random directions: y is off by about 2e-7 of itself, the
    # difference over 2 * 2^-7 by 2e-7 * 64 of the sum's parts, and the step's own error is (2^-7)^2 / 6 of third derivatives.
    igc = _igc()
    say("qk differences")
    q, k, pos, freq, w, dy = case(50, 2, 1, 24, 3, 4, F32)
    dq, dk, dqw, dkw = igc.qk_norm_rotary_backward(dy[0], dy[1], q, k, pos, freq, w[0], w[1])

    def value(q, k, w0, w1):
        a, b = igc.qk_norm_rotary(q, k, pos, freq, w0, w1)
        return float((a.double() * dy[0].double()).sum() + (b.double() * dy[1].double()).sum())

    g, h = torch.Generator(device="cuda").manual_seed(3), 2.0 ** -7
    for _ in range(4):
        t = [torch.randn(x.shape, generator=g, device="cuda") for x in (q, k, w[0], w[1])]
        slope = sum(float((x.double() * y.double()).sum()) for x, y in zip(t, (dq, dk, dqw, dkw)))
        up, down = [value(*[x + s * h * y for x, y in zip((q, k, w[0], w[1]), t)]) for s in (1, -1)]
        assert abs((up - down) / (2 * h) - slope) < 2e-3 * (1 + abs(slope)) + 0.05


def test_reruns_streams_and_graphs():
    igc = _igc()
    say("qk graph")
    q, k, pos, freq, w, dy = case(3001, 4, 2, 64, 3, 10, BF16)

    def step():
        y = igc.qk_norm_rotary(q, k, pos, freq, w[0], w[1])
        return (*y, *igc.qk_norm_rotary_backward(dy[0], dy[1], q, k, pos, freq, w[0], w[1]))

    first = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            caught = step()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, other))
    for _ in range(3):
        q.normal_()
        dy[0].normal_()
        eager = step()
        for t in caught:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, caught))


def test_frequencies():
    igc = _igc()
    f = igc.rotary_frequencies(64, 10000.0)
    assert f.shape == (1, 32) and f.dtype == F32 and f[0, 0] == 1
    assert abs(float(f[0, 16]) - 0.01) < 1e-8
    assert igc.rotary_frequencies(64, axes=3).shape == (3, 10)
    assert torch.allclose(igc.rotary_frequencies(64, scaling="linear", factor=4.0) * 4, f)
    g = igc.rotary_frequencies(64, scaling="base", factor=4.0)
    assert g[0, 0] == 1 and abs(float(g[0, -1] * 4 / f[0, -1]) - 1) < 1e-5
    p = igc.rotary_frequencies(64, scaling="parts", factor=4.0, original=4096)
    assert torch.equal(p[0, :8], f[0, :8]) and torch.allclose(p[0, -3:] * 4, f[0, -3:]) and bool((p <= f).all()) and bool((p >= f / 4.001).all())


def test_broadcast_operands():
    # One head, or one row, seen many times (strides of 0): results and gradients as for copies.
    igc = _igc()
    say("qk broadcast")
    g = torch.Generator(device="cuda").manual_seed(2)
    x, dy = torch.randn(50, 1, 24, generator=g, device="cuda"), torch.randn(50, 4, 24, generator=g, device="cuda")
    freq, pos = igc.rotary_frequencies(24).cuda(), torch.arange(50, dtype=torch.int32, device="cuda")
    for q in (x.expand(50, 4, 24), x[:1].expand(50, 4, 24)):
        a, b = igc.qk_norm_rotary(q, None, pos, freq), igc.qk_norm_rotary(q.contiguous(), None, pos, freq)
        assert a[0].is_contiguous() and torch.equal(a[0], b[0])
        a, b = [igc.qk_norm_rotary_backward(dy, None, t, None, pos, freq) for t in (q, q.contiguous())]
        assert torch.equal(a[0], b[0]) and torch.equal(a[2], b[2])
