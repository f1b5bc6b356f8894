"""The example of norm, rotation, window attention and dropout together: output and gradients against the same block in float32
torch with autograd, a captured training step against eager ones, and the block read row by row against the block read at once.

The example computes in bf16 (half a step 2^-8 a rounding). The forward pass rounds seven times on its longest chain (norm,
projection, rotation, probabilities, attention, projection, sum), independently of each other: sqrt(7) 2^-8 = 1.0%; scores of up to 8 that
are off by 2^-8 of |q| |k| / sqrt(dim) over sqrt(dim) channels, below 0.4%, come on top: 1.5% in norm. The backward pass doubles
the chain and its weight gradients are products rounded to bf16 once more: sqrt(15) 2^-8 = 1.5%, with the forward pass's values
in it: 3% in norm.
"""
import os
import sys

import pytest
import torch

from tests._gpu import require_gpu, say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def _reference(block, x, ijk, offsets, keep, dy):
    import window_block as ex
    p = {k: v.float().detach().clone().requires_grad_() for k, v in block.p.items()}
    x = x.float().requires_grad_()
    n, h, hk, d = x.shape[0], block.heads, block.kv_heads, block.dim
    t = (torch.nn.functional.layer_norm(x, (x.shape[1],), p["nw"], p["nb"]) @ p["qkv"]).view(n, h + 2 * hk, d)
    angle = torch.cat([ijk[:, a:a + 1].double() * block.frequencies[a].double() for a in range(3)], 1)[:, None]
    c, s, m = torch.cos(angle).float(), torch.sin(angle).float(), angle.shape[2]

    def turned(z, w):
        z = z * torch.rsqrt(z.square().mean(2, keepdim=True) + 1e-6) * w
        a, b = z[..., :m], z[..., m:2 * m]
        return torch.cat([a * c - b * s, b * c + a * s, z[..., 2 * m:]], 2)

    q, k, v = turned(t[:, :h], p["qw"]), turned(t[:, h:h + hk], p["kw"]), t[:, h + hk:]
    rows, o = [], offsets.tolist()
    for first, last in zip(o, o[1:]):
        at = torch.arange(last - first, device="cuda")
        near = (at <= at[:, None] + block.right) & ((at >= at[:, None] - block.left) | (at < ex.TOKENS))
        kk, vv = [z[first:last].repeat_interleave(h // hk, 1).transpose(0, 1).contiguous() for z in (k, v)]
        sc = q[first:last].transpose(0, 1).contiguous() @ kk.transpose(1, 2).contiguous() * d ** -0.5
        rows.append((torch.softmax(sc.masked_fill(~near, -torch.inf), 2) @ vv).transpose(0, 1))
    y = x + torch.where(keep, torch.cat(rows).reshape(n, -1) @ p["wo"], 0.0) * (65536 / (65536 - round(65536 * block.drop)))
    y.backward(dy.float())
    return y.detach(), x.grad, {k: v.grad for k, v in p.items()}


def _case(left, right, seed=2, channels=128):
    import window_block as ex
    ijk, offsets = ex.scene(3, 1500)
    n = ijk.shape[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    x, dy = [torch.randn(n, channels, generator=g, device="cuda").bfloat16() for _ in range(2)]
    return ex.WindowBlock(channels, 4, 2, left, right, 0.25), ijk, offsets, x, dy


@pytest.mark.parametrize("left,right", [(60, 60), (200, 0)])
def test_block_against_float32_autograd(left, right):
    import sparse_convolution_amd as igc
    say(f"window block against autograd, {left} {right}")
    block, ijk, offsets, x, dy = _case(left, right)
    y = block.forward(x, ijk, offsets, 5)
    dx, grads = block.backward(dy, ijk, offsets)
    keep = igc.dropout(torch.ones_like(x), block.drop, block.seed, 5) > 0
    ry, rdx, rgrads = _reference(block, x, ijk, offsets, keep, dy)

    def off(a, b):
        return float((a.float().reshape(b.shape) - b).norm() / b.norm())

    assert off(y, ry) < 0.015
    assert off(dx, rdx) < 0.03
    for name, r in rgrads.items():
        assert off(grads[name], r) < 0.03, (name, off(grads[name], r))


def test_a_captured_step_of_training():
    # The step's number lives on the device and counts in the graph, so that every replay drops other elements.
    say("window block captured")
    block, ijk, offsets, x, dy = _case(60, 60)
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block.forward(x, ijk, offsets, count)
        block.backward(dy, ijk, offsets)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            y = block.forward(x, ijk, offsets, count)
            dx, grads = block.backward(dy, ijk, offsets)
            count += 1
    torch.cuda.synchronize()
    for step in range(3):
        graph.replay()
        torch.cuda.synchronize()
        ey = block.forward(x, ijk, offsets, step)
        edx, egrads = block.backward(dy, ijk, offsets)
        assert torch.equal(y, ey) and torch.equal(dx, edx)
        assert all(torch.equal(grads[k], egrads[k]) for k in grads)
        x.copy_(x.flip(0))


def test_rows_one_by_one_behind_a_cache():
    import window_block as ex
    say("window block row by row")
    block, _, _, _, _ = _case(20, 0)
    block.drop = 0.0
    g = torch.Generator(device="cuda").manual_seed(7)
    lengths = [70, 33, 51]
    offsets = torch.tensor([0] + lengths).cumsum(0).int().cuda()
    n = sum(lengths)
    x = torch.randn(n, 128, generator=g, device="cuda").bfloat16()
    ijk = torch.randint(-50, 50, (n, 3), generator=g, device="cuda").int()
    whole = block.forward(x, ijk, offsets)
    ck = torch.full((3, 80, block.kv_heads, block.dim), float("nan"), dtype=torch.bfloat16, device="cuda")
    cv, used = ck.clone(), torch.zeros(3, dtype=torch.int32, device="cuda")
    for t in range(min(lengths)):
        rows = offsets[:-1].long() + t
        y = block.step(x[rows], ijk[rows].contiguous(), ck, cv, used)
        # The same values up to the roundings of p, of out and of the sum.
        assert float((y.float() - whole[rows].float()).norm() / whole[rows].float().norm()) < 4 * 2.0 ** -8
    assert used.tolist() == [33] * 3


def test_example_trains():
    import window_block as ex
    say("window example")
    losses = ex.train(steps=3, channels=64, heads=2, voxels=3000, window=40, say=say)
    assert len(losses) == 3 and all(x == x and x < 1e3 for x in losses)
