"""Cross attention and its gradients against the formulas in float64, one sequence and head at a time.

Tolerances are bounds on each element, from sums of magnitudes formed beside the reference. u is the relative
rounding to the data's type (2^-8 for bf16, which has 8 significant bits; fp32's is within f) and f = 2e-5
covers the fp32 chain: scores of size up to 30 are off by about 2^-22 of that, exp turns the absolute error of
its argument into a relative one of up to 1e-5, sums add a few 2^-24.
  out: probabilities are rounded to u before the product with v, the result is rounded once more:
       (u + f) sum_j p |v| + u |out|
  dv:  the same with dout: (u + f) sum_i p |dout| + u |dv|
  dq, dk: ds = p (dp - delta) is rounded to u; delta comes from the rounded `out`, off by u sum |dout out|; in fp32
       the difference is off by f of its parts: scale sum (u |ds| + p (u e + f (e + g))) |k or q| + u |result|, with
       e = sum |dout out| and g = sum |dout v|.
"""
import numpy as np
import pytest
import torch

from tests._gpu import require_gpu, say

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
U = {F32: 0.0, BF16: 2.0 ** -8}
F = 2e-5


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _igc():
    import sparse_convolution_amd as igc
    return igc


def _case(lq, lk, heads, kv_heads, dim, dtype, seed=0, masked=0.0, packed=False, std=1.0, offset=0):
    """Operands of ragged sequences: `packed` gives q, k and v as slices with strides of their own, offset an
    address that is no multiple of 16 bytes."""
    g = torch.Generator().manual_seed(1000 * seed + 17 * sum(lq) + sum(lk) + dim)
    nq, nk = sum(lq), sum(lk)
    q, k, v = torch.randn(nq, heads, dim, generator=g) * std, torch.randn(nk, kv_heads, dim, generator=g), torch.randn(nk, kv_heads, dim, generator=g)
    do = torch.randn(nq, heads, dim, generator=g)
    mask = (torch.rand(nk, generator=g) >= masked) if masked else None
    dev = [t.to(dtype).cuda() for t in (q, k, v, do)]
    if packed:
        kv = torch.full((nk, kv_heads, 2, dim + 3 * (packed == "odd")), float("nan"), dtype=dtype, device="cuda")
        kv[:, :, 0, :dim], kv[:, :, 1, :dim] = dev[1], dev[2]
        dev[1], dev[2] = kv[:, :, 0, :dim], kv[:, :, 1, :dim]
        qq = torch.full((heads, nq, dim), float("nan"), dtype=dtype, device="cuda").transpose(0, 1)
        qq.copy_(dev[0])
        dev[0] = qq
    if offset:
        for i in range(4):
            buf = torch.empty(dev[i].numel() + offset, dtype=dtype, device="cuda")[offset:].view(dev[i].shape)
            buf.copy_(dev[i])
            dev[i] = buf
    off = [torch.tensor(np.concatenate([[0], np.cumsum(x)]), dtype=torch.int32).cuda() for x in (lq, lk)] if len(lq) > 1 else [None, None]
    return dev, off, None if mask is None else mask.cuda()


def _reference(dev, lq, lk, mask, scale):
    """Results and bounds in float64 (u and f filled in by the caller's dtype)."""
    dtype = dev[0].dtype
    u = U[dtype]
    q, k, v, do = [t.double().cpu() for t in dev]
    h, hk = q.shape[1], k.shape[1]
    r = {n: torch.zeros_like(t) for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", k))}
    b = {n: torch.zeros_like(t) for n, t in r.items()}
    lse = torch.full(q.shape[:2], -np.inf, dtype=torch.float64)
    qa = ka = 0
    for nq, nk in zip(lq, lk):
        rows, keys = torch.arange(qa, qa + nq), torch.arange(ka, ka + nk)
        qa, ka = qa + nq, ka + nk
        if mask is not None:
            keys = keys[mask.cpu()[keys]]
        if not keys.numel() or not nq:
            continue
        for i in range(h):
            j = i * hk // h
            qq, kk, vv, dd = q[rows, i], k[keys, j], v[keys, j], do[rows, i]
            s = scale * qq @ kk.T
            lse[rows, i] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1)
            o = p @ vv
            e, dp = (dd.abs() * o.abs()).sum(1, keepdim=True), dd @ vv.T
            ds = p * (dp - (dd * o).sum(1, keepdim=True))
            w = scale * (u * ds.abs() + p * (u * e + F * (e + dd.abs() @ vv.abs().T)))
            r["out"][rows, i], b["out"][rows, i] = o, (u + F) * p @ vv.abs()
            r["dq"][rows, i], b["dq"][rows, i] = scale * ds @ kk, w @ kk.abs()
            r["dk"][keys, j] += scale * ds.T @ qq
            b["dk"][keys, j] += w.T @ qq.abs()
            r["dv"][keys, j] += p.T @ dd
            b["dv"][keys, j] += (u + F) * p.T @ dd.abs()
    for n in r:
        b[n] += u * r[n].abs() + 1e-9
    return r, b, lse


def check(lq, lk, heads, kv_heads, dim, dtype, scale=None, **kw):
    igc = _igc()
    say(f"attention q={lq[:4]}.. k={lk[:4]}.. heads={heads}/{kv_heads} dim={dim} {dtype} {kw}")
    dev, (qo, ko), mask = _case(lq, lk, heads, kv_heads, dim, dtype, **kw)
    q, k, v, do = dev
    out, lse = igc.cross_attention(q, k, v, qo, ko, mask, scale)
    dq, dk, dv = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko, mask, scale)
    torch.cuda.synchronize()
    r, b, rl = _reference(dev, lq, lk, mask, dim ** -0.5 if scale is None else scale)
    got = lse.double().cpu()
    assert torch.equal(torch.isinf(got), torch.isinf(rl))
    fin = torch.isfinite(rl)
    assert bool(((got - rl)[fin].abs() <= F * (1 + rl[fin].abs())).all())
    for name, t in (("out", out), ("dq", dq), ("dk", dk), ("dv", dv)):
        assert t.dtype == dtype and t.is_contiguous()
        err = (t.double().cpu() - r[name]).abs()
        assert bool((err <= b[name]).all()), (name, float((err / b[name]).max()), float(err.max()))
    return out, lse, (dq, dk, dv)


DIMS = [(1, 1, 1), (2, 2, 8), (1, 1, 20), (2, 1, 32), (4, 2, 40), (4, 4, 64), (1, 1, 96), (3, 1, 128), (2, 2, 100)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,kv_heads,dim", DIMS)
def test_head_layouts(heads, kv_heads, dim, dtype):
    check([37, 70], [65, 130], heads, kv_heads, dim, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([1], [64]), ([3], [63]), ([128], [65]), ([129], [128]), ([256], [32]), ([257], [33]), ([300], [1]),
                                   ([5, 0, 7], [9, 4, 0]), ([0, 0, 4], [3, 1, 70]), ([130, 1, 260, 31], [7, 100, 1, 64]),
                                   ([1] * 20, list(range(20))), ([40] * 9, [3] * 9)])
def test_lengths(lq, lk, dtype):
    check(lq, lk, 2, 2, 32, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lq,lk,heads,kv_heads,dim", [([2], [5003], 2, 2, 64), ([1, 1, 1], [3000, 17, 1500], 4, 1, 32), ([6001], [41], 2, 2, 32),
                                                      ([3000, 2000], [90, 33], 2, 1, 64), ([100], [2500], 1, 1, 128),
                                                      ([1] * 8, [700] * 8, 8, 8, 64), ([2, 1], [1025, 3000], 6, 2, 128), ([4], [900], 3, 3, 20)])
def test_long_axes(lq, lk, heads, kv_heads, dim, dtype):
    check(lq, lk, heads, kv_heads, dim, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("packed", ["even", "odd"])
@pytest.mark.parametrize("dim", [24, 64, 128])
def test_strided_operands(dim, packed, dtype):
    check([50, 90], [77, 40], 4, 2, dim, dtype, packed=packed)
    check([1, 1], [1200, 40], 4, 2, dim, dtype, packed=packed)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_operands_at_odd_addresses(dtype):
    check([50, 90], [77, 40], 2, 2, 32, dtype, offset=1)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lq,lk", [([60, 200], [100, 150]), ([1, 1], [1500, 900]), ([3000], [50])])
def test_masked_keys(lq, lk, dtype):
    check(lq, lk, 2, 1, 64, dtype, masked=0.4)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lq,lk", [([70, 30, 200], [90, 64, 130]), ([1, 1, 2], [600, 1300, 20])])
def test_masked_places_may_hold_anything_and_masks_may_leave_nothing(lq, lk, dtype):
    igc = _igc()
    dev, (qo, ko), mask = _case(lq, lk, 2, 2, 32, dtype, masked=0.3)
    mask[lk[0]:lk[0] + lk[1]] = False  # the second sequence has no key left
    q, k, v, do = dev
    base = igc.cross_attention(q, k, v, qo, ko, mask)
    grads = igc.cross_attention_backward(do, q, k, v, *base, qo, ko, mask)
    rows = slice(lq[0], lq[0] + lq[1])
    assert bool((base[0][rows] == 0).all()) and bool((base[1][rows] == -np.inf).all()) and bool((grads[0][rows] == 0).all())
    k2, v2 = k.clone(), v.clone()
    k2[~mask], v2[~mask] = float("nan"), float("inf")
    again = igc.cross_attention(q, k2, v2, qo, ko, mask)
    grads2 = igc.cross_attention_backward(do, q, k2, v2, *again, qo, ko, mask)
    for x, y in zip(base + grads, again + grads2):
        assert torch.equal(x, y)
    assert bool((grads[1][~mask] == 0).all()) and bool((grads[2][~mask] == 0).all())
    r, b, _ = _reference(dev, lq, lk, mask, 32 ** -0.5)
    for name, t in (("out", base[0]), ("dq", grads[0]), ("dk", grads[1]), ("dv", grads[2])):
        assert bool(((t.double().cpu() - r[name]).abs() <= b[name]).all()), name


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_large_scores_and_given_scale(dtype):
    # Scores of several hundred: only differences from the maximum may be exponentiated. The argument's own
    # rounding grows with the scores, so this looks at rows with one clear winner.
    igc = _igc()
    n, d = 64, 32
    k = torch.eye(n, d).repeat(1, 1).view(n, 1, d)
    k[32:] = -k[:32]
    q = (k * 40).to(dtype).cuda()
    kk = (k * 10).to(dtype).cuda()
    v = torch.randn(n, 1, d, generator=torch.Generator().manual_seed(3)).to(dtype).cuda()
    out, lse = igc.cross_attention(q, kk, v, scale=1.0)
    assert torch.equal(out, v) and bool(((lse - 400).abs() < 1e-3).all())
    check([40], [50], 1, 1, 64, dtype, scale=0.03)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows", [1, 2, 70])
@pytest.mark.parametrize("step,first", [(3.0, 0.0), (40.0, 0.0), (-5.0, 0.0), (400.0, -200.0)])
def test_scores_that_grow_or_fall_along_the_keys(step, first, rows, dtype):
    # Scores first + step * (block of 50 keys) + noise, up to several thousand: the running reference must follow them,
    # within a tile and from one to the next. q has one channel of 1 and keys carry the ramp there, so the ramp is exact
    # in bf16 (multiples of the step below 2^8 steps); the rest are small values. The ramp's fp32 rounding in exp's
    # argument is up to 2^-22 of the largest score, 1e-3 here: rows are compared at 4e-3 of the largest value.
    igc = _igc()
    n, d = 400, 32
    g = torch.Generator().manual_seed(5)
    q = torch.randn(rows, 1, d, generator=g)
    k = torch.randn(n, 1, d, generator=g)
    v = torch.randn(n, 1, d, generator=g)
    q[:, :, 0] = 1.0
    k[:, 0, 0] = (first + step * (torch.arange(n) // 50)).to(BF16).float()
    q, k, v = [t.to(dtype).cuda() for t in (q, k, v)]
    out, lse = igc.cross_attention(q, k, v, scale=1.0)
    s = q[:, 0].double().cpu() @ k[:, 0].double().cpu().T
    ref = torch.softmax(s, 1) @ v[:, 0].double().cpu()
    assert bool(((lse[:, 0].double().cpu() - torch.logsumexp(s, 1)).abs() <= 1e-3 + 2.0 ** -22 * s.abs().max()).all())
    assert bool(((out[:, 0].double().cpu() - ref).abs() <= (4e-3 + 2 * U[dtype]) * v.double().abs().max().cpu()).all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_nan_and_infinite_queries_stay_in_their_rows(dtype):
    igc = _igc()
    for lq, lk in (([150], [90]), ([2], [900])):
        (q, k, v, do), _, _ = _case(lq, lk, 2, 2, 32, dtype)
        base, _ = igc.cross_attention(q, k, v)
        q2 = q.clone()
        q2[1, 0, 3] = float("nan")
        out, lse = igc.cross_attention(q2, k, v)
        assert bool(torch.isnan(out[1, 0]).all()) and bool(torch.isnan(lse[1, 0]))
        out[1, 0] = base[1, 0]
        assert torch.equal(out, base)


def test_no_queries_or_no_keys():
    igc = _igc()
    for dtype in (F32, BF16):
        q, k = torch.randn(5, 2, 16, device="cuda", dtype=dtype), torch.randn(7, 1, 16, device="cuda", dtype=dtype)
        out, lse = igc.cross_attention(q, k[:0], k[:0])
        assert bool((out == 0).all()) and bool((lse == -np.inf).all())
        dq, dk, dv = igc.cross_attention_backward(q, q, k[:0], k[:0], out, lse)
        assert bool((dq == 0).all()) and dk.shape == (0, 1, 16)
        out, lse = igc.cross_attention(q[:0], k, k)
        assert out.shape == (0, 2, 16) and lse.shape == (0, 2)
        dq, dk, dv = igc.cross_attention_backward(q[:0], q[:0], k, k, out, lse)
        assert dq.shape == (0, 2, 16) and bool((dk == 0).all()) and bool((dv == 0).all())


def test_offsets_past_the_arrays_are_clamped():
    igc = _igc()
    (q, k, v, do), (qo, ko), _ = _case([40, 30], [50, 20], 2, 2, 32, BF16)
    far, kfar = qo.clone(), ko.clone()
    far[2], kfar[2], kfar[0] = 1 << 30, 1 << 30, -5
    base = igc.cross_attention(q, k, v, qo, ko)
    got = igc.cross_attention(q, k, v, far, kfar)
    assert torch.equal(base[0], got[0]) and torch.equal(base[1], got[1])
    for a, b in zip(igc.cross_attention_backward(do, q, k, v, *base, qo, ko), igc.cross_attention_backward(do, q, k, v, *base, far, kfar)):
        assert torch.equal(a, b)


def test_gradients_one_side_at_a_time():
    igc = _igc()
    for lq, lk in (([90, 20], [70, 100]), ([2], [1500]), ([4000], [30])):
        (q, k, v, do), (qo, ko), _ = _case(lq, lk, 4, 2, 64, BF16)
        out, lse = igc.cross_attention(q, k, v, qo, ko)
        dq, dk, dv = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko)
        a = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko, need_dkv=False)
        b = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko, need_dq=False)
        assert a[1] is None and a[2] is None and b[0] is None
        assert torch.equal(a[0], dq) and torch.equal(b[1], dk) and torch.equal(b[2], dv)


def test_gradient_against_differences():
    # Central differences along random directions with step 2^-5: the fp32 forward's error, about 1e-6 of sums of
    # 60 x 2 x 16 terms of order one, divided by the step (3e-3 in all), and the step's square (1e-3) times third
    # derivatives of order one times the sums' size (about 40).
    igc = _igc()
    t = 2.0 ** -5
    (q, k, v, do), (qo, ko), _ = _case([40, 20], [30, 25], 2, 1, 16, F32)
    out, lse = igc.cross_attention(q, k, v, qo, ko)
    grads = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko)

    def loss(*x):
        return float((igc.cross_attention(*x, qo, ko)[0].double() * do.double()).sum())

    for i, g in enumerate(grads):
        u = torch.randn(g.shape, generator=torch.Generator().manual_seed(i)).cuda()
        hi, lo = [q, k, v], [q, k, v]
        hi[i], lo[i] = hi[i] + t * u, lo[i] - t * u
        ref = (loss(*hi) - loss(*lo)) / (2 * t)
        assert abs(float((g.double() * u.double()).sum()) - ref) <= 0.06, i


@pytest.mark.parametrize("lq,lk", [([300, 500], [100, 90]), ([1, 1], [2000, 1500])])
def test_other_stream_repeat_and_graph_are_bit_identical(lq, lk):
    igc = _igc()
    (q, k, v, do), (qo, ko), mask = _case(lq, lk, 4, 2, 64, BF16, masked=0.1)

    def both():
        out, lse = igc.cross_attention(q, k, v, qo, ko, mask)
        return (out, lse) + igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko, mask)

    first = both()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        second = both()
    s.synchronize()
    for a, b in zip(first, second):
        assert torch.equal(a, b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kept = both()
    for n in range(4):
        q.copy_(torch.randn(q.shape, generator=torch.Generator().manual_seed(n)))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, both()):
            assert torch.equal(a, b), n


@pytest.mark.parametrize("rows", [1, 300])
def test_caches_past_2_to_the_31_elements(rows):
    # The states of the last sequence lie beyond element 2^31 of k and v (4.4 GB each); the same states in a
    # small tensor of their own give the same bits.
    igc = _igc()
    heads, dim, nk, last = 8, 128, 2150000, 900
    k = torch.zeros(nk, heads, dim, dtype=BF16, device="cuda")
    v = torch.zeros(nk, heads, dim, dtype=BF16, device="cuda")
    assert (nk - last) * heads * dim > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(4)
    k[-last:] = torch.randn(last, heads, dim, generator=g, device="cuda").to(BF16)
    v[-last:] = torch.randn(last, heads, dim, generator=g, device="cuda").to(BF16)
    q = torch.randn(rows, heads, dim, generator=g, device="cuda").to(BF16)
    do = torch.randn(rows, heads, dim, generator=g, device="cuda").to(BF16)
    kl, vl = k[-last:].clone(), v[-last:].clone()
    # Two empty sequences around one, so that the number of parts is decided from the same averages.
    qo = torch.tensor([0, 0, rows], dtype=torch.int32, device="cuda")
    ko = torch.tensor([0, nk - last, nk], dtype=torch.int32, device="cuda")
    out, lse = igc.cross_attention(q, k, v, qo, ko)
    ref, rlse = igc.cross_attention(q, kl, vl)
    # Other parts of the key axis, so equal up to their order: fp32 sums and one rounding to bf16.
    assert float((lse - rlse).abs().max()) < 1e-4
    assert float((out.float() - ref.float()).abs().max()) <= 2 * U[BF16] * float(ref.float().abs().max())
    dq, dk, dv = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko)
    rq, rk, rv = igc.cross_attention_backward(do, q, kl, vl, out, lse)
    assert bool((dk[:nk - last] == 0).all()) and bool((dv[:nk - last] == 0).all())
    for a, b in ((dq, rq), (dk[-last:], rk), (dv[-last:], rv)):
        assert float((a.float() - b.float()).abs().max()) <= 4 * U[BF16] * float(b.float().abs().max())


@pytest.mark.parametrize("dtype", [torch.float32, BF16])
def test_masked_keys_get_zeros_whatever_the_output_gradient_holds(dtype):
    igc = _igc()
    g = torch.Generator(device="cuda").manual_seed(8)
    q, do = (torch.randn(150, 2, 64, generator=g, device="cuda").to(dtype) for _ in range(2))
    k, v = (torch.randn(300, 2, 64, generator=g, device="cuda").to(dtype) for _ in range(2))
    mask = torch.rand(300, generator=g, device="cuda") > 0.3
    do[7, 0, 5], do[11, 1, 3] = float("nan"), float("inf")
    out, lse = igc.cross_attention(q, k, v, key_mask=mask)
    _, dk, dv = igc.cross_attention_backward(do, q, k, v, out, lse, key_mask=mask)
    assert bool((dk[~mask] == 0).all()) and bool((dv[~mask] == 0).all())
    # The gradients of the kept keys carry the NaN of each head's one channel, and dv nothing else.
    assert bool(dk[mask].isnan().any()) and bool(dv[mask][:, 0, 5].isnan().all())
    rest = dv[mask][:, 0].clone()
    rest[:, 5] = 0
    assert bool(rest.isfinite().all())


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("lq,heads,dim", [([1], 1, 33), ([1], 1, 1), ([3], 3, 45), ([41], 1, 99)])
def test_a_split_key_axis_with_odd_sizes(lq, heads, dim, dtype):
    # 3 parts: an odd number of partial results before the statistics.
    check(lq, [1000], heads, heads, dim, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,keys", [(1, 90), (40, 90), (300, 90), (40, 3000)])
def test_a_scale_near_zero(rows, keys, dtype):
    # With a scale below the smallest normal number all scores are 0 to 2^-100: out is the mean of v and lse log(keys).
    igc = _igc()
    (q, k, v, do), _, _ = _case([rows], [keys], 2, 2, 32, dtype)
    out, lse = igc.cross_attention(q, k, v, scale=1e-38)
    mean = v.double().mean(0).cpu()
    assert bool(((lse.double().cpu() - np.log(keys)).abs() <= F * (1 + np.log(keys))).all())
    # Probabilities are 1 or 1 / keys: exact or one rounding; sums and the result's rounding as in the bounds above.
    assert bool(((out.double().cpu() - mean).abs() <= (U[dtype] + F) * v.double().abs().mean(0).cpu() + U[dtype] * mean.abs()).all())
    _, _, dv = igc.cross_attention_backward(do, q, k, v, out, lse, scale=1e-38)
    ref, mag = do.double().sum(0).cpu() / keys, do.double().abs().sum(0).cpu() / keys
    assert bool(((dv.double().cpu() - ref).abs() <= (U[dtype] + F) * mag + U[dtype] * ref.abs()).all())


def _off_by(lk, seqs, rows=256):
    """rms errors of dq, and of dk sequence by sequence, against float64, as multiples of the error that rounding the exact
    results to bf16 makes. The reference's delta comes from the rounded `out`, as the kernel's does."""
    igc = _igc()
    lq, lk = [rows] * seqs, lk if isinstance(lk, list) else [lk] * seqs
    dev, (qo, ko), _ = _case(lq, lk, 2, 2, 64, BF16)
    q, k, v, do = dev
    out, lse = igc.cross_attention(q, k, v, qo, ko)
    dq, dk, _ = igc.cross_attention_backward(do, q, k, v, out, lse, qo, ko)
    q, k, v, do, out, dq, dk = [t.double().cpu() for t in (q, k, v, do, out, dq, dk)]
    rq, rk = torch.zeros_like(q), torch.zeros_like(k)
    a = b = 0
    for nq, nk in zip(lq, lk):
        for h in range(2):
            qq, kk, vv, dd, oo = q[a:a + nq, h], k[b:b + nk, h], v[b:b + nk, h], do[a:a + nq, h], out[a:a + nq, h]
            p = torch.softmax(qq @ kk.T / 8, 1)
            ds = p * (dd @ vv.T - (dd * oo).sum(1, keepdim=True))
            rq[a:a + nq, h], rk[b:b + nk, h] = ds @ kk / 8, ds.T @ qq / 8
        a, b = a + nq, b + nk
    res, b = [], 0
    for nk in lk:
        s = slice(b, b + nk)
        res.append(float((dk[s] - rk[s]).norm() / (rk[s].bfloat16().double() - rk[s]).norm()))
        b += nk
    return float((dq - rq).norm() / (rq.bfloat16().double() - rq).norm()), res


@pytest.mark.parametrize("lk", [30, 100, 256, 400, 1500, [30, 900], [900, 30]])
def test_bf16_score_gradients_are_not_rounded_once(lk):
    # ds in two bf16 parts carries 16 bits: what is left is the result's own rounding, with the fp32 chain and the order of
    # sums far below it. Rounded once, each term is off by as much of itself as the result's rounding is of the result, and the
    # terms cancel: both errors are independent and at least as large, sqrt(2) in all. Halfway between 1 and 1.5.
    dq, dk = _off_by(lk, 2)
    say(f"lk={lk}: dq {dq:.3f}, dk {dk}")
    assert dq < 1.25 and max(dk) < 1.25


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 96), (4, 2, 128), (8, 2, 100), (3, 1, 72), (4, 1, 65)])
def test_a_few_rows_of_wide_heads(heads, kv_heads, dim, dtype):
    # 1 to 4 rows that share a key head: one part and several parts of the key axis, a sequence without keys.
    check([1, 1, 1], [90, 0, 1300], heads, kv_heads, dim, dtype)
    check([1], [3001], heads, kv_heads, dim, dtype, masked=0.3)
