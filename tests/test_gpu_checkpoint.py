"""8-bit activation checkpoints: their format, the layer norm that writes and reads them, and the
convolution's weight gradient from them.

The format is exact: codes and scales equal the fp32 formula, and each value is within half a step (the
group's largest magnitude / 254) of what was packed, plus the fp32 rounding of a product, 2^-22. The
checkpoint of a normalised row is a rounding of a computed value: within half a step of the float64 value
plus the forward pass's own error (1e-5, as in the layer norm's tests). Gradients from a checkpoint are
those of the values it stands for, at the tolerances of the gradients from features.
"""
import numpy as np
import pytest
import torch

import oracle
import workloads
from tests._gpu import normwise_error, require_gpu, say, to_dev
from tests.test_gpu_norm import _forward64, _inputs, check_backward, check_forward

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _igc():
    import sparse_convolution_amd as igc
    return igc


def _pack32(x):
    """Codes and scales of float32 rows by the fp32 formula."""
    n, c = x.shape
    g = -(-c // 64)
    codes, scales = np.zeros((n, c), np.int8), np.zeros((n, g), np.float32)
    for k in range(g):
        part = x[:, 64 * k:64 * k + 64]
        a = np.abs(part).max(1)
        with np.errstate(all="ignore"):
            zero, bad = a < np.float32(2.0 ** -100), ~np.isfinite(a)
            inv = np.where(zero | bad, np.float32(0), (np.float32(1) / a) * np.float32(127)).astype(np.float32)
            q = np.rint(part * inv[:, None])
        codes[:, 64 * k:64 * k + 64] = np.where(inv[:, None] == 0, 0, q).astype(np.int8)
        scales[:, k] = np.where(zero, 0, np.where(bad, np.nan, a * (np.float32(1) / np.float32(127))))
    return codes, scales


def _values64(ck):
    s = ck.scales.double().cpu().repeat_interleave(64, 1)[:, :ck.shape[1]]
    return ck.codes.double().cpu() * s


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,c,offset", [(1, 1, 0), (3, 5, 0), (1000, 8, 0), (501, 16, 0), (333, 63, 0), (400, 64, 0), (77, 65, 0),
                                        (129, 100, 0), (90, 128, 0), (55, 200, 1), (31, 257, 0), (11, 1024, 0), (3, 4096, 0), (7, 4095, 0),
                                        (64, 32, 4), (100003, 24, 0)])
def test_pack_and_unpack(n, c, offset, dtype):
    igc = _igc()
    say(f"checkpoint n={n} c={c} offset={offset} {dtype}")
    x = _inputs(n, c, dtype, None, n + c, offset=offset)[0]
    x[0, 0] *= 50
    ck = igc.checkpoint_pack(x)
    codes, scales = _pack32(x.float().cpu().numpy())
    assert np.array_equal(ck.codes.cpu().numpy(), codes)
    assert np.array_equal(ck.scales.cpu().numpy(), scales)
    step = torch.from_numpy(scales).double().repeat_interleave(64, 1)[:, :c]
    x64 = x.double().cpu()
    assert bool(((_values64(ck) - x64).abs() <= 0.5 * step + 2.0 ** -22 * x64.abs() + step * 1e-5).all())
    exact32 = torch.from_numpy(codes.astype(np.float32)) * torch.from_numpy(scales).repeat_interleave(64, 1)[:, :c]
    assert torch.equal(igc.checkpoint_unpack(ck, F32).cpu(), exact32)
    assert torch.equal(igc.checkpoint_unpack(ck).cpu(), exact32.to(dtype))
    assert ck.nbytes == n * c + 4 * n * -(-c // 64)


def test_zero_tiny_infinite_and_nan_groups():
    igc = _igc()
    x = torch.randn(6, 200, generator=torch.Generator().manual_seed(1))
    x[0, :64] = 0
    x[1, 64:128] = 2.0 ** -110
    x[2, 70] = float("inf")
    x[3, 199] = float("nan")
    x[4, :] = 3e38
    ck = igc.checkpoint_pack(x.cuda())
    v = igc.checkpoint_unpack(ck).cpu()
    assert bool((v[0, :64] == 0).all()) and bool((v[1, 64:128] == 0).all())
    assert bool(torch.isnan(v[2, 64:128]).all()) and bool(torch.isfinite(v[2, :64]).all()) and bool(torch.isfinite(v[2, 128:]).all())
    assert bool(torch.isnan(v[3, 192:]).all()) and bool(torch.isfinite(v[3, :192]).all())
    assert bool(((v[4] / 3e38 - 1).abs() < 1e-6).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("n,c", [(1, 1), (9, 3), (501, 8), (1000, 20), (777, 64), (90, 96), (1003, 128), (301, 255), (129, 256), (65, 300),
                                 (33, 512), (40, 520), (21, 1000), (9, 1024), (7, 1100), (5, 2048), (3, 4095), (3, 4096), (30011, 32)])
def test_norm_with_checkpoint(n, c, dtype):
    igc = _igc()
    say(f"layer norm checkpoint n={n} c={c} {dtype}")
    x, dy, w, b = _inputs(n, c, dtype, dtype, 3 * n + c)
    y, ck, rstd = igc.layer_norm_checkpoint(x, w, b)
    yp, mean, rp = igc.layer_norm(x, w, b)
    assert torch.equal(y, yp) and torch.equal(rstd, rp)  # the checkpoint changes neither
    check_forward(x, w, b, 1e-5, y, mean, rstd)
    h = _forward64(x, w, b, 1e-5)[3]
    v = _values64(ck)
    step = ck.scales.double().cpu().repeat_interleave(64, 1)[:, :c]
    big = (x.double().abs().amax(1).cpu() * rstd.double().cpu() + 1)[:, None]
    assert bool(((v - h).abs() <= 0.5 * step + 1e-5 * big).all())
    dx, dw, db = igc.layer_norm_checkpoint_backward(dy, ck, rstd, w)
    check_backward(dy, v, rstd.double().cpu(), w, dx, dw, db)
    only, none_w, _ = igc.layer_norm_checkpoint_backward(dy, ck, rstd, w, need_dweight=False)
    assert none_w is None and torch.equal(only, dx)


def test_norm_checkpoint_of_no_rows():
    igc = _igc()
    x = torch.empty((0, 24), dtype=BF16, device="cuda")
    y, ck, rstd = igc.layer_norm_checkpoint(x)
    dx, dw, db = igc.layer_norm_checkpoint_backward(x, ck, rstd)
    assert dx.shape == (0, 24) and bool((dw == 0).all()) and bool((db == 0).all())
    assert igc.checkpoint_unpack(igc.checkpoint_pack(x)).shape == (0, 24)


def test_norm_checkpoint_gradient_is_near_the_full_one():
    # The stored rows are off by at most 1/254 of a group's largest value, about 1.2% of one standard
    # deviation here (largest of 64 normal values: 2.4 to 3.5); the gradient's term in xhat moves by that
    # times mean(g xhat), itself about 1/sqrt(c) of g.
    igc = _igc()
    x, dy, w, b = _inputs(4001, 128, F32, F32, 8)
    y, ck, rstd = igc.layer_norm_checkpoint(x, w, b)
    _, mean, _ = igc.layer_norm(x, w, b)
    full, fw, fb = igc.layer_norm_backward(dy, x, mean, rstd, w)
    got, gw, gb = igc.layer_norm_checkpoint_backward(dy, ck, rstd, w)
    assert float((got - full).norm() / full.norm()) < 0.02 / 128 ** 0.5 * 2
    assert float((gw - fw).norm() / fw.norm()) < 0.02 and torch.equal(gb, fb)


@pytest.mark.parametrize("dtype,cin,cout", [(BF16, 128, 128), (BF16, 64, 64), (BF16, 32, 64), (BF16, 192, 64), (BF16, 256, 128),
                                            (BF16, 20, 36), (BF16, 4, 32), (F32, 8, 16), (F32, 16, 8), (F32, 40, 48)])
def test_conv_weight_gradient_from_a_checkpoint(dtype, cin, cout):
    igc = _igc()
    say(f"conv backward from a checkpoint {dtype} {cin}->{cout}")
    rng = np.random.default_rng(cin + cout)
    cube = np.stack(np.meshgrid(*[np.arange(18)] * 3, indexing="ij"), -1).reshape(-1, 3)
    coords = np.concatenate([cube[rng.random(cube.shape[0]) < 0.3] + o for o in ([0, 0, 0], [40, -7, 3])]).astype(np.int32)
    g = igc.grid_build(to_dev(coords))
    m = igc.kernel_map(g)
    n = g.n_voxels
    f = torch.from_numpy(workloads.make_features(n, cin, 5100)).to("cuda", dtype)
    w = torch.from_numpy(workloads.make_weights(cin, cout, 6100, 0.05)).to("cuda", dtype)
    dy = torch.from_numpy(workloads.make_features(n, cout, 7100)).to("cuda", dtype)
    ck = igc.checkpoint_pack(f)
    v = igc.checkpoint_unpack(ck)
    dx, dw = igc.sparse_conv_backward(g, ck, w, dy, m)
    rx, rw = igc.sparse_conv_backward(g, v, w, dy, m)
    assert torch.equal(dx, rx) and torch.equal(dw, rw)  # the same sums over the same values
    ref = oracle.conv_wgrad(m.cpu().numpy(), v.float().cpu().numpy(), dy.float().cpu().numpy())
    assert normwise_error(dw.cpu().numpy(), ref) <= 1e-5
    alone = igc.sparse_conv_backward(g, ck, w, dy, m, need_dfeats=False)
    assert alone[0] is None and torch.equal(alone[1], dw)


def test_conv_weight_gradient_from_codes_at_an_odd_address():
    igc = _igc()
    cube = np.stack(np.meshgrid(*[np.arange(9)] * 3, indexing="ij"), -1).reshape(-1, 3).astype(np.int32)
    g = igc.grid_build(to_dev(cube))
    m = igc.kernel_map(g)
    f = torch.from_numpy(workloads.make_features(g.n_voxels, 64, 1)).to("cuda", BF16)
    w = torch.zeros(27, 64, 64, dtype=BF16, device="cuda")
    dy = torch.from_numpy(workloads.make_features(g.n_voxels, 64, 2)).to("cuda", BF16)
    ck = igc.checkpoint_pack(f)
    buf = torch.empty(ck.codes.numel() + 3, dtype=torch.int8, device="cuda")
    moved = buf[3:].view(ck.codes.shape)
    moved.copy_(ck.codes)
    odd = igc.Checkpoint8(moved, ck.scales, BF16)
    assert torch.equal(igc.sparse_conv_backward(g, odd, w, dy, m)[1], igc.sparse_conv_backward(g, ck, w, dy, m)[1])
    assert torch.equal(igc.checkpoint_unpack(odd), igc.checkpoint_unpack(ck))


@pytest.mark.parametrize("cin,cout,side,blocks", [(128, 128, 46, (9, 24)), (128, 128, 63, (25, 99)), (256, 256, 32, (9, 24)),
                                                  (256, 256, 41, (25, 99)), (256, 128, 44, (9, 24)), (128, 256, 55, (25, 99))])
def test_conv_weight_gradient_from_a_checkpoint_on_larger_grids(cin, cout, side, blocks):
    # The block of the weight gradient that a workgroup computes grows with the grid: up to 8 blocks of 128 x 128 for each 11 tiles
    # of 256 rows it is 64 x 64, up to 24 it is 64 x 128, beyond 128 x 128. The row order and the chunks are those of the
    # features' gradient at these sizes, so the sums are the same to the bit.
    igc = _igc()
    rng = np.random.default_rng(side)
    cube = np.stack(np.meshgrid(*[np.arange(side)] * 3, indexing="ij"), -1).reshape(-1, 3)
    g = igc.grid_build(to_dev(cube[rng.random(cube.shape[0]) < 0.3].astype(np.int32)))
    m, n = igc.kernel_map(g), g.n_voxels
    say(f"conv backward from a checkpoint {cin}->{cout}, {n} voxels")
    count = -(-n // (11 * 256)) * (cin // 128) * (cout // 128)
    assert blocks[0] <= count <= blocks[1], count
    f = torch.from_numpy(workloads.make_features(n, cin, 5200)).to("cuda", BF16)
    dy = torch.from_numpy(workloads.make_features(n, cout, 7200)).to("cuda", BF16)
    w = torch.zeros(27, cin, cout, dtype=BF16, device="cuda")
    ck = igc.checkpoint_pack(f)
    v = igc.checkpoint_unpack(ck)
    dw = igc.sparse_conv_backward(g, ck, w, dy, m, need_dfeats=False)[1]
    assert torch.equal(dw, igc.sparse_conv_backward(g, v, w, dy, m, need_dfeats=False)[1])
    ref = oracle.conv_wgrad(m.cpu().numpy(), v.float().cpu().numpy(), dy.float().cpu().numpy())
    assert normwise_error(dw.cpu().numpy(), ref) <= 1e-5
