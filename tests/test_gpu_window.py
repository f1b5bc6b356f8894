"""Window attention with sinks and its gradients against the formulas in float64, one sequence and head at a time.

The bounds are those of tests/test_gpu_attention.py, with the visible keys of each row in place of all: u half a step of the
data's type (2^-8 for bf16; fp32's is within f), f = 2e-5 for the fp32 chain of scores, exponentials and sums.
"""
import numpy as np
import pytest
import torch

from tests._gpu import require_gpu, say
from tests.test_gpu_attention import F, U, _case

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _igc():
    import sparse_convolution_amd as igc
    return igc


def visible(lq, lk, left, right, sinks):
    p, j = torch.arange(lq)[:, None] + lk - lq, torch.arange(lk)[None]
    see = torch.ones(lq, lk, dtype=torch.bool)
    if right is not None:
        see &= j <= p + right
    if left is not None:
        see &= (j >= p - left) | (j < sinks)
    return see


def reference(dev, lq, lk, mask, scale, left, right, sinks, q_first=0, k_first=0):
    """Results and bounds in float64."""
    u = U[dev[0].dtype]
    q, k, v, do = [t.double().cpu() for t in dev]
    h, hk = q.shape[1], k.shape[1]
    r = {n: torch.zeros_like(t) for n, t in (("out", q), ("dq", q), ("dk", k), ("dv", k))}
    b = {n: torch.zeros_like(t) for n, t in r.items()}
    lse = torch.full(q.shape[:2], -np.inf, dtype=torch.float64)
    qa, ka = q_first, k_first
    for nq, nk in zip(lq, lk):
        rows, keys = slice(qa, qa + nq), slice(ka, ka + nk)
        see = visible(nq, nk, left, right, sinks)
        if mask is not None:
            see = see & mask.cpu()[keys]
        qa, ka = qa + nq, ka + nk
        if not nq or not nk:
            continue
        blind = ~see.any(1, keepdim=True)
        for i in range(h):
            j = i * hk // h
            qq, kk, vv, dd = q[rows, i], k[keys, j], v[keys, j], do[rows, i]
            s = (scale * qq @ kk.T).masked_fill(~see, -np.inf)
            lse[rows, i] = torch.logsumexp(s, 1)
            p = torch.softmax(s, 1).masked_fill(blind, 0.0)
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


def compare(out, lse, grads, r, b, rl, rows=slice(None), keys=slice(None)):
    got = lse.double().cpu()[rows]
    rl = rl[rows]
    fin = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(got), fin) and bool((got[~fin] == -np.inf).all())
    assert bool(((got - rl)[fin].abs() <= F * (1 + rl[fin].abs())).all())
    for name, t, at in (("out", out, rows), ("dq", grads[0], rows), ("dk", grads[1], keys), ("dv", grads[2], keys)):
        assert t.is_contiguous()
        err = (t.double().cpu() - r[name]).abs()[at]
        assert bool((err <= b[name][at]).all()), (name, float((err / b[name][at]).max()), float(err.max()))


def check(lq, lk, heads, kv_heads, dim, dtype, left, right, sinks, scale=None, **kw):
    igc = _igc()
    say(f"window q={lq[:4]} k={lk[:4]} heads={heads}/{kv_heads} dim={dim} {dtype} left={left} right={right} sinks={sinks} {kw}")
    dev, (qo, ko), mask = _case(lq, lk, heads, kv_heads, dim, dtype, **kw)
    q, k, v, do = dev
    out, lse = igc.window_attention(q, k, v, left, right, sinks, qo, ko, mask, scale)
    grads = igc.window_attention_backward(do, q, k, v, out, lse, left, right, sinks, qo, ko, mask, scale)
    torch.cuda.synchronize()
    compare(out, lse, grads, *reference(dev, lq, lk, mask, dim ** -0.5 if scale is None else scale, left, right, sinks))


TYPES = pytest.mark.parametrize("dtype", [F32, BF16])
WINDOWS = [(0, 0, 0), (0, 0, 3), (5, 0, 0), (5, 0, 1), (0, 7, 2), (64, 64, 4), (31, 100, 40), (200, 0, 70), (None, 0, 0), (None, 33, 5), (40, None, 3),
           (1000, 1000, 10), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1), (3, 0, 2 ** 31 - 1), (None, None, 4)]


@TYPES
@pytest.mark.parametrize("left,right,sinks", WINDOWS)
def test_windows(left, right, sinks, dtype):
    check([300, 77], [300, 77], 2, 1, 32, dtype, left, right, sinks)


@TYPES
@pytest.mark.parametrize("heads,kv_heads,dim", [(1, 1, 1), (2, 2, 8), (3, 1, 20), (4, 2, 40), (4, 4, 64), (6, 2, 64), (2, 1, 96), (1, 1, 100), (3, 1, 128)])
def test_head_layouts(heads, kv_heads, dim, dtype):
    check([150, 201], [150, 201], heads, kv_heads, dim, dtype, 60, 9, 2)


@TYPES
@pytest.mark.parametrize("lq,lk", [([1], [1]), ([2], [2]), ([33], [33]), ([129], [129]), ([257], [257]), ([0, 5, 0, 90], [0, 5, 0, 90]), ([40] * 9, [40] * 9),
                                   ([0, 7], [3, 9]), ([7, 0], [0, 4])])
@pytest.mark.parametrize("left,right,sinks", [(16, 0, 1), (20, 20, 4)])
def test_lengths(lq, lk, left, right, sinks, dtype):
    check(lq, lk, 2, 2, 32, dtype, left, right, sinks)


@TYPES
@pytest.mark.parametrize("lq,lk,heads,kv_heads,dim", [([1], [900], 2, 2, 64), ([1] * 7, [5, 0, 800, 64, 1, 1700, 33], 4, 2, 32), ([1, 1], [3000, 2500], 8, 2, 128),
                                                      ([2, 1, 3], [600, 40, 900], 1, 1, 64), ([1] * 3, [500, 20, 77], 3, 1, 33), ([40, 70], [500, 100], 4, 2, 64),
                                                      ([130], [2000], 1, 1, 128)])
@pytest.mark.parametrize("left,right,sinks", [(255, 0, 4), (1500, 0, 0), (20, 0, 90), (None, 0, 0)])
def test_new_rows_behind_a_cache(lq, lk, heads, kv_heads, dim, left, right, sinks, dtype):
    check(lq, lk, heads, kv_heads, dim, dtype, left, right, sinks)


@TYPES
@pytest.mark.parametrize("lq,lk,room,heads,kv_heads,dim", [([1] * 5, [5, 1, 800, 0, 64], 900, 4, 2, 64), ([1, 1], [300, 2000], 4096, 8, 2, 128),
                                                           ([40, 0, 130], [500, 60, 130], 600, 2, 1, 32), ([1] * 90, [37] * 90, 64, 2, 2, 64)])
@pytest.mark.parametrize("left,right,sinks", [(255, 0, 4), (None, 0, 0), (30, 9, 0), (None, None, 0)])
def test_caches_with_room(lq, lk, room, heads, kv_heads, dim, left, right, sinks, dtype):
    # Each sequence's keys lie at the start of `room` rows whose rest holds NaN.
    igc = _igc()
    say(f"window caches with room {lq[:4]} {lk[:4]} {dtype}")
    dev, (qo, _), _ = _case(lq, lk, heads, kv_heads, dim, dtype)
    q, k, v, do = dev
    cache = [torch.full((len(lk) * room, kv_heads, dim), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
    first = 0
    for b, n in enumerate(lk):
        for c, t in zip(cache, (k, v)):
            c[b * room:b * room + n] = t[first:first + n]
        first += n
    ko = (torch.arange(len(lk) + 1) * room).int().cuda()
    lengths = torch.tensor(lk, dtype=torch.int32).cuda()
    out, lse = igc.window_attention(q, *cache, left, right, sinks, qo, ko, kv_lengths=lengths)
    r, b, rl = reference(dev, lq, lk, None, dim ** -0.5, left, right, sinks)
    got = lse.double().cpu()
    fin = torch.isfinite(rl)
    assert torch.equal(torch.isfinite(got), fin) and bool(((got - rl)[fin].abs() <= F * (1 + rl[fin].abs())).all())
    assert bool(((out.double().cpu() - r["out"]).abs() <= b["out"]).all())
    # Lengths beyond the rows are the rows, negative ones none.
    full = igc.window_attention(q, *[c.nan_to_num(0.0) for c in cache], left, right, sinks, qo, ko, kv_lengths=torch.full_like(lengths, 2 ** 31 - 1))
    same = igc.window_attention(q, *[c.nan_to_num(0.0) for c in cache], left, right, sinks, qo, ko, kv_lengths=torch.full_like(lengths, room))
    assert torch.equal(full[0], same[0])
    none = igc.window_attention(q, *cache, left, right, sinks, qo, ko, kv_lengths=torch.full_like(lengths, -5))
    assert bool((none[0] == 0).all()) and bool((none[1] == -np.inf).all())


@TYPES
def test_more_queries_than_keys(dtype):
    # The first queries stand before the first key: without a look ahead they see nothing.
    for right in (0, 30):
        check([200, 50], [90, 50], 2, 2, 32, dtype, 40, right, 3)


@TYPES
@pytest.mark.parametrize("n,left,right,sinks", [(3000, 64, 64, 8), (2500, 300, 0, 130), (4001, 20, 3, 1), (2000, None, 0, 0), (1500, 700, None, 300)])
def test_long_sequences(n, left, right, sinks, dtype):
    check([n], [n], 2, 1, 64, dtype, left, right, sinks)


# More than 512 tiles of 64 rows (and keys): the kernels in which no two waves share a row's axis.
MANY = [510, 33, 700, 64, 0, 129, 1] * 12


@TYPES
@pytest.mark.parametrize("heads,kv_heads,dim", [(2, 2, 32), (4, 2, 64), (3, 3, 20), (2, 2, 40), (2, 2, 96), (4, 2, 128)])
@pytest.mark.parametrize("left,right,sinks", [(60, 9, 2), (100, 0, 70), (None, 0, 0)])
def test_many_tiles(heads, kv_heads, dim, left, right, sinks, dtype):
    assert len(MANY) * -(-(sum(MANY) // len(MANY)) // 64) * kv_heads > 512
    check(MANY, MANY, heads, kv_heads, dim, dtype, left, right, sinks)


@TYPES
@pytest.mark.parametrize("dim", [32, 64, 96, 128])
def test_many_tiles_masked_and_strided(dim, dtype):
    check(MANY, MANY, 2, 2, dim, dtype, 60, 9, 5, masked=0.3)
    check(MANY, MANY, 4, 2, dim, dtype, 40, 40, 3, packed="odd")


@pytest.mark.parametrize("dim", [40, 64])
@pytest.mark.parametrize("left,right,sinks", [(60, 9, 2), (100, 0, 70)])
def test_between_256_and_512_tiles(dim, left, right, sinks):
    # fp32 heads of 33 to 64 channels have a form of eight waves there.
    lengths = [510, 33, 700, 64, 0, 129, 1] * 6
    assert 256 < len(lengths) * -(-(sum(lengths) // len(lengths)) // 64) * 2 <= 512
    check(lengths, lengths, 2, 2, dim, F32, left, right, sinks)
    check(lengths, lengths, 4, 2, dim, F32, left, right, sinks, masked=0.3, packed="odd")


@TYPES
def test_many_tiles_of_new_rows_behind_caches(dtype):
    # Chunks of queries over longer caches, more far parts than one.
    lk = [n + 300 for n in MANY]
    check(MANY, lk, 2, 2, 64, dtype, 200, 0, 9)


@TYPES
def test_many_sequences_with_sinks(dtype):
    # More rows of sinks than keys: the far parts go by the keys themselves. And far parts of ragged sequences.
    check([3, 0, 17, 40, 1, 90] * 3, [3, 0, 17, 40, 1, 90] * 3, 2, 2, 32, dtype, 8, 0, 64)
    check([2000, 40, 1300], [2000, 40, 1300], 1, 1, 32, dtype, 30, 30, 200)


@TYPES
@pytest.mark.parametrize("packed", ["even", "odd"])
@pytest.mark.parametrize("dim", [24, 64])
def test_strided_operands(dim, packed, dtype):
    check([150, 90], [150, 90], 4, 2, dim, dtype, 40, 11, 3, packed=packed)
    check([1, 1], [1200, 40], 4, 2, dim, dtype, 700, 0, 3, packed=packed)


@TYPES
def test_operands_at_odd_addresses(dtype):
    check([50, 190], [50, 190], 2, 2, 32, dtype, 40, 0, 3, offset=1)


@TYPES
@pytest.mark.parametrize("lq,lk", [([160, 200], [160, 200]), ([1, 1], [1500, 900]), ([3, 60], [400, 80])])
def test_masked_keys(lq, lk, dtype):
    check(lq, lk, 2, 1, 64, dtype, 50, 0, 5, masked=0.4)


@TYPES
def test_masks_that_leave_rows_empty(dtype):
    igc = _igc()
    say(f"window masks {dtype}")
    lq = lk = [300, 200]
    dev, (qo, ko), mask = _case(lq, lk, 2, 2, 32, dtype, masked=0.2)
    mask[:3] = False
    mask[60:140] = False   # rows whose whole window is masked, and the sinks with it
    mask[300:500] = False  # a sequence without keys
    q, k, v, do = dev
    k[~mask], v[~mask] = float("nan"), float("inf")
    out, lse = igc.window_attention(q, k, v, 30, 0, 3, qo, ko, mask)
    grads = igc.window_attention_backward(do, q, k, v, out, lse, 30, 0, 3, qo, ko, mask)
    clean = [q, torch.where(mask[:, None, None], k, 0), torch.where(mask[:, None, None], v, 0), do]
    compare(out, lse, grads, *reference(clean, lq, lk, mask, 32 ** -0.5, 30, 0, 3))
    blind = ~(visible(300, 300, 30, 0, 3) & mask.cpu()[:300]).any(1)
    assert int(blind.sum()) >= 50 and bool((out[:300][blind] == 0).all()) and bool((grads[0][:300][blind] == 0).all())
    assert bool((grads[1][~mask] == 0).all()) and bool((grads[2][~mask] == 0).all())


@TYPES
@pytest.mark.parametrize("qo,nq,ko,nk", [([30, 200, 290], 300, [30, 200, 290], 300), ([1, 2, 3], 5, [9, 500, 900], 950), ([257, 300], 310, [0, 200], 300)])
@pytest.mark.parametrize("sinks", [0, 4, 500])
def test_rows_of_no_sequence_are_left(qo, nq, ko, nk, sinks, dtype):
    igc = _igc()
    say(f"window offsets {qo} of {nq}, {ko} of {nk}, sinks {sinks}, {dtype}")
    dev, _, _ = _case([nq], [nk], 4, 2, 32, dtype)
    q, k, v, do = dev
    a, b = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in (qo, ko)]
    lq, lk = [[y - x for x, y in zip(o, o[1:])] for o in (qo, ko)]
    out, lse = igc.window_attention(q, k, v, 50, 7, sinks, a, b)
    grads = igc.window_attention_backward(do, q, k, v, out, lse, 50, 7, sinks, a, b)
    rows, keys = slice(qo[0], qo[-1]), slice(ko[0], ko[-1])
    compare(out, lse, grads, *reference(dev, lq, lk, None, 32 ** -0.5, 50, 7, sinks, qo[0], ko[0]), rows, keys)
    # Through the C ABI into prepared arrays: rows outside stay as they were.
    import ctypes

    from sparse_convolution_amd import _lib
    from sparse_convolution_amd._block import _problem
    p, _ = _problem(q, k, v, a, b, None, None)
    lib, size, s = _lib.load(), ctypes.c_size_t(0), torch.cuda.current_stream().cuda_stream
    mark = [torch.full_like(t, 7.0) for t in (q, lse, q, k, v)]
    for back in (0, 1):
        _lib.check(lib.igc_window_attention_workspace(p, 50, 7, sinks, back, ctypes.byref(size)))
        ws = torch.empty(max(16, size.value), dtype=torch.uint8, device="cuda")
        if back:
            _lib.check(lib.igc_window_attention_backward(p, 50, 7, sinks, q.data_ptr(), k.data_ptr(), v.data_ptr(), out.data_ptr(), lse.data_ptr(),
                                                         do.data_ptr(), *[t.data_ptr() for t in mark[2:]], ws.data_ptr(), size.value, s))
        else:
            _lib.check(lib.igc_window_attention(p, 50, 7, sinks, None, q.data_ptr(), k.data_ptr(), v.data_ptr(), mark[0].data_ptr(), mark[1].data_ptr(),
                                                ws.data_ptr(), size.value, s))
    torch.cuda.synchronize()
    for t, want, at in zip(mark, (out, lse, *grads), (rows, rows, rows, keys, keys)):
        assert torch.equal(t[at], want[at])
        rest = torch.ones(t.shape[0], dtype=torch.bool)
        rest[at] = False
        assert bool((t[rest] == 7).all())


def test_offsets_past_the_arrays_are_clamped():
    igc = _igc()
    say("window offsets past the arrays")
    (q, k, v, do), (qo, ko), _ = _case([90, 70], [90, 70], 2, 2, 32, BF16)
    far = qo.clone()
    far[2] = 1 << 30
    base = igc.window_attention(q, k, v, 20, 5, 3, qo, ko)
    got = igc.window_attention(q, k, v, 20, 5, 3, far, far)
    assert torch.equal(base[0], got[0]) and torch.equal(base[1], got[1])
    for a, b in zip(igc.window_attention_backward(do, q, k, v, *base, 20, 5, 3, qo, ko), igc.window_attention_backward(do, q, k, v, *base, 20, 5, 3, far, far)):
        assert torch.equal(a, b)


def test_without_limits_it_is_cross_attention():
    igc = _igc()
    say("window without limits")
    (q, k, v, do), (qo, ko), mask = _case([90, 70], [50, 170], 4, 2, 64, BF16, masked=0.2)
    a, b = igc.cross_attention(q, k, v, qo, ko, mask), igc.window_attention(q, k, v, q_offsets=qo, kv_offsets=ko, key_mask=mask)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(igc.cross_attention_backward(do, q, k, v, *a, qo, ko, mask),
                    igc.window_attention_backward(do, q, k, v, *a, q_offsets=qo, kv_offsets=ko, key_mask=mask)):
        assert torch.equal(x, y)


@TYPES
def test_scores_outside_the_window_do_not_matter_however_large(dtype):
    # A key far above all others, seen by rows 50 to 60 only, and the same key without it: the other rows' results and the other
    # keys' gradients lie within the same bounds of the same exact values. (Their bits may differ: where some row of a wave raises its
    # reference, the others raise theirs to their own maxima, which changes roundings and nothing else.)
    igc = _igc()
    say(f"window large scores {dtype}")
    dev, _, _ = _case([200], [200], 1, 1, 32, dtype)
    q, k, v, do = dev
    q[:, :, 0] = 1.0
    k2 = k.clone()
    k2[50, :, 0] = 30000.0
    rest = torch.ones(200, dtype=torch.bool)
    rest[50:61] = False
    r, b, rl = reference([q, k, v, do], [200], [200], None, 32 ** -0.5, 10, 0, 2)
    r2, b2, _ = reference([q, k2, v, do], [200], [200], None, 32 ** -0.5, 10, 0, 2)
    for name in ("out", "dq"):
        assert torch.equal(r[name][rest], r2[name][rest])
    out, lse = igc.window_attention(q, k2, v, 10, 0, 2)
    grads = igc.window_attention_backward(do, q, k2, v, out, lse, 10, 0, 2)
    keys = torch.ones(200, dtype=torch.bool)
    keys[50] = False
    compare(out, lse, grads, r2, b2, rl, rest, keys)
    assert bool(((out[50:61] - v[50]).abs() <= 2.0 ** -20).all())
    assert all(bool(torch.isfinite(g).all()) for g in grads)


@TYPES
def test_broadcast_keys(dtype):
    # One key head seen as two (a stride of 0) gives what two copies of it give; its gradient is per copy.
    igc = _igc()
    say(f"window broadcast {dtype}")
    (q, k, v, do), _, _ = _case([300], [300], 2, 1, 32, dtype)
    wide = [t.expand(300, 2, 32) for t in (k, v)]
    a, b = igc.window_attention(q, *wide, 40, 0, 3), igc.window_attention(q, *[t.contiguous() for t in wide], 40, 0, 3)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for x, y in zip(igc.window_attention_backward(do, q, *wide, *a, 40, 0, 3),
                    igc.window_attention_backward(do, q, *[t.contiguous() for t in wide], *a, 40, 0, 3)):
        assert x.is_contiguous() and torch.equal(x, y)


def test_no_queries_or_no_keys():
    igc = _igc()
    for dtype in (F32, BF16):
        q, k = torch.randn(5, 2, 16, device="cuda", dtype=dtype), torch.randn(7, 1, 16, device="cuda", dtype=dtype)
        out, lse = igc.window_attention(q, k[:0], k[:0], 3, 0, 2)
        assert bool((out == 0).all()) and bool((lse == -np.inf).all())
        dq, dk, dv = igc.window_attention_backward(q, q, k[:0], k[:0], out, lse, 3, 0, 2)
        assert bool((dq == 0).all()) and dk.shape == (0, 1, 16)
        out, lse = igc.window_attention(q[:0], k, k, 3, 0, 2)
        dq, dk, dv = igc.window_attention_backward(q[:0], q[:0], k, k, out, lse, 3, 0, 2)
        assert dq.shape == (0, 2, 16) and bool((dk == 0).all()) and bool((dv == 0).all())


def test_gradients_one_side_at_a_time():
    igc = _igc()
    for lq, lk in (([90, 300], [90, 300]), ([2], [1500]), ([4000], [4000])):
        (q, k, v, do), (qo, ko), _ = _case(lq, lk, 4, 2, 64, BF16)
        out, lse = igc.window_attention(q, k, v, 60, 0, 5, qo, ko)
        dq, dk, dv = igc.window_attention_backward(do, q, k, v, out, lse, 60, 0, 5, qo, ko)
        a = igc.window_attention_backward(do, q, k, v, out, lse, 60, 0, 5, qo, ko, need_dkv=False)
        b = igc.window_attention_backward(do, q, k, v, out, lse, 60, 0, 5, qo, ko, need_dq=False)
        assert a[1] is None and a[2] is None and b[0] is None
        assert torch.equal(a[0], dq) and torch.equal(b[1], dk) and torch.equal(b[2], dv)


def test_gradient_against_differences():
    # As for cross attention: the fp32 forward's error over the step (3e-3 in all), and the step's square (1e-3) times third
    # derivatives of order one times the sums' size (about 40).
    igc = _igc()
    t = 2.0 ** -5
    (q, k, v, do), (qo, ko), _ = _case([40, 20], [40, 20], 2, 1, 16, F32)
    where = (9, 2, 3, qo, ko)
    out, lse = igc.window_attention(q, k, v, *where)
    grads = igc.window_attention_backward(do, q, k, v, out, lse, *where)

    def loss(*x):
        return float((igc.window_attention(*x, *where)[0].double() * do.double()).sum())

    for i, g in enumerate(grads):
        u = torch.randn(g.shape, generator=torch.Generator().manual_seed(i)).cuda()
        hi, lo = [q, k, v], [q, k, v]
        hi[i], lo[i] = hi[i] + t * u, lo[i] - t * u
        assert abs(float((g.double() * u.double()).sum()) - (loss(*hi) - loss(*lo)) / (2 * t)) <= 0.06, i


@pytest.mark.parametrize("lq,lk,left,sinks", [([300, 500], [300, 500], 70, 4), ([1, 1], [2000, 1500], 1200, 4), ([60, 2500], [60, 2500], 20, 150)])
def test_other_stream_repeat_and_graph_are_bit_identical(lq, lk, left, sinks):
    igc = _igc()
    say(f"window graph {lq}")
    (q, k, v, do), (qo, ko), mask = _case(lq, lk, 4, 2, 64, BF16, masked=0.1)

    def both():
        out, lse = igc.window_attention(q, k, v, left, 0, sinks, qo, ko, mask)
        return (out, lse) + igc.window_attention_backward(do, q, k, v, out, lse, left, 0, sinks, qo, ko, mask)

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


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("masked", [0.0, 0.3])
@pytest.mark.parametrize("heads,kv_heads,dim", [(4, 2, 40), (4, 4, 64), (2, 1, 96), (1, 1, 100), (3, 1, 128)])
def test_repeats_between_other_kernels_are_bit_identical(heads, kv_heads, dim, masked, dtype):
    """What other kernels leave in registers and shared memory is in no result: cross attention runs between the calls."""
    igc = _igc()
    (q, k, v, do), (qo, ko), m = _case([150, 201], [150, 201], heads, kv_heads, dim, dtype, masked=masked)
    win = 60, 9, 2
    first = None
    for _ in range(20):
        igc.cross_attention(q, k, v, qo, ko)
        out, lse = igc.window_attention(q, k, v, *win, qo, ko, m)
        got = [out, lse, *igc.window_attention_backward(do, q, k, v, out, lse, *win, qo, ko, m)]
        first = first or got
        for name, a, b in zip(("out", "lse", "dq", "dk", "dv"), got, first):
            assert torch.equal(a, b), name


@pytest.mark.parametrize("rows", [1, 300])
def test_caches_past_2_to_the_31_elements(rows):
    # The cache's end, and with it the window, lies beyond element 2^31 of k and v (4.4 GB each), its sinks at the start:
    # the same keys in a small tensor of their own give the same up to the order of sums.
    igc = _igc()
    say(f"window past 2^31, {rows} rows")
    heads, dim, nk, left, sinks = 8, 128, 2150000, 700, 5
    assert (nk - rows - left) * heads * dim > 2 ** 31
    last = rows + left
    g = torch.Generator(device="cuda").manual_seed(4)
    k, v = (torch.zeros(nk, heads, dim, dtype=BF16, device="cuda") for _ in range(2))
    for t in (k, v):
        for part in (slice(0, sinks), slice(nk - last, nk)):
            t[part] = torch.randn(t[part].shape, generator=g, device="cuda").to(BF16)
    q, do = (torch.randn(rows, heads, dim, generator=g, device="cuda").to(BF16) for _ in range(2))
    kl, vl = [torch.cat([t[:sinks], t[-last:]]) for t in (k, v)]
    out, lse = igc.window_attention(q, k, v, left, 0, sinks)
    ref, rlse = igc.window_attention(q, kl, vl, left, 0, sinks)
    assert float((lse - rlse).abs().max()) < 1e-4
    assert float((out.float() - ref.float()).abs().max()) <= 2 * U[BF16] * float(ref.float().abs().max())
    dq, dk, dv = igc.window_attention_backward(do, q, k, v, out, lse, left, 0, sinks)
    rq, rk, rv = igc.window_attention_backward(do, q, kl, vl, out, lse, left, 0, sinks)
    assert bool((dk[sinks:nk - last] == 0).all()) and bool((dv[sinks:nk - last] == 0).all())
    for a, b in ((dq, rq), (torch.cat([dk[:sinks], dk[-last:]]), rk), (torch.cat([dv[:sinks], dv[-last:]]), rv)):
        assert float((a.float() - b.float()).abs().max()) <= 4 * U[BF16] * float(b.float().abs().max())
