"""The example block (norm, cross attention, norm, convolution) end to end: its output and gradients against the same
block in float32 torch with autograd, and a few steps of training.

The example computes in bf16 (2^-8 a rounding, a dozen roundings on the longest chain, independent of each other:
3.5 x 2^-8 = 1.4%) and its backward pass reads 8-bit checkpoints (rows off by up to 1/254 of their largest of 64 values, rms
0.7% of one standard deviation): gradients agree within 4% in norm.
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


def _reference(block, kmap, offsets, x, states, state_offsets, mask, dy):
    p = {k: v.float().detach().clone().requires_grad_() for k, v in block.p.items()}
    x = x.float().requires_grad_()
    n, c = x.shape
    h, d = block.heads, c // block.heads
    ln = torch.nn.functional.layer_norm
    q = (ln(x, (c,), p["n1w"], p["n1b"]) @ p["wq"]).view(n, h, d)
    kv = (states.float() @ p["wkv"]).view(-1, 2, h, d)
    rows = []
    o, s = offsets.tolist(), state_offsets.tolist()
    for b in range(len(o) - 1):
        keys = torch.arange(s[b], s[b + 1], device="cuda")
        keys = keys[mask[keys]]
        sc = torch.einsum("qhd,khd->hqk", q[o[b]:o[b + 1]], kv[keys, 0]) * d ** -0.5
        rows.append(torch.einsum("hqk,khd->qhd", torch.softmax(sc, 2), kv[keys, 1]))
    x1 = x + torch.cat(rows).reshape(n, c) @ p["wo"]
    y2 = ln(x1, (c,), p["n2w"], p["n2b"])
    y = x1
    for t in range(27):
        src = kmap[t].long()
        y = y + (y2[src.clamp(min=0)] * (src >= 0)[:, None]) @ p["conv"][t]
    y.backward(dy.float())
    return y.detach(), x.grad, {k: v.grad for k, v in p.items()}


def test_block_against_float32_autograd():
    import conditioned_block as ex
    say("conditioned block against autograd")
    grid, kmap, offsets = ex.scene(3, 2500)
    n, c = grid.n_voxels, 128
    assert int(offsets[-1]) == n
    g = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(n, c, generator=g, device="cuda").bfloat16()
    dy = torch.randn(n, c, generator=g, device="cuda").bfloat16()
    lengths = [40, 7, 90]
    so = torch.tensor([0] + lengths).cumsum(0).int().cuda()
    states = torch.randn(sum(lengths), 96, generator=g, device="cuda").bfloat16()
    mask = torch.rand(sum(lengths), generator=g, device="cuda") > 0.2
    block = ex.ConditionedBlock(c, 4, 96)
    y = block.forward(grid, kmap, offsets, x, states, so, mask)
    dx, grads = block.backward(grid, kmap, offsets, dy, states, so, mask)
    ry, rdx, rgrads = _reference(block, kmap, offsets, x, states, so, mask, dy)

    def off(a, b):
        return float((a.float().reshape(b.shape) - b).norm() / b.norm())

    assert off(y, ry) < 0.014
    assert off(dx, rdx) < 0.04
    for name, r in rgrads.items():
        assert off(grads[name], r) < 0.04, (name, off(grads[name], r))


def test_training_reduces_the_loss():
    import conditioned_block as ex
    losses = ex.train(steps=6, channels=64, heads=2, voxels=3000, say=say)
    assert losses[-1] < 0.9 * losses[0] and all(b < a for a, b in zip(losses, losses[1:]))
