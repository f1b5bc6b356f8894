"""A voxel block that attends to an encoder's states, trained with its activations kept in 8 bits.

    python examples/conditioned_block.py [--steps 20] [--channels 128] [--heads 4] [--voxels 20000]

Several scenes share one grid (each in a root tile of its own, so their rows are contiguous), and each has a set
of states of its own length (tokens, image patches). With x the voxels' features and c the states:

    h = layer_norm(x)            kept as an 8-bit checkpoint of the normalised rows
    x = x + cross_attention(h Wq, c Wk, c Wv) Wo
    g = layer_norm(x)            kept as an 8-bit checkpoint
    y = x + sparse_conv(g)       its input g kept as an 8-bit checkpoint

The backward pass reads the checkpoints: layer_norm_checkpoint_backward for the norms, sparse_conv_backward for the
convolution's weights, checkpoint_unpack for the projection's input. The attention keeps out and lse. The linear
projections are plain torch products.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_convolution_amd as igc  # noqa: E402


def scene(n_scenes: int, voxels: int, seed: int = 0):
    """(grid, kernel map, row offsets of the scenes) of rough sheets, scene s in root tile i >> 12 = s."""
    g = torch.Generator().manual_seed(seed)
    parts, side = [], max(2, int((voxels / n_scenes) ** 0.5))
    for s in range(n_scenes):
        i, j = torch.meshgrid(torch.arange(side + s), torch.arange(side), indexing="ij")
        k = (30 + 8 * torch.sin(i * 0.2 + s) + 6 * torch.cos(j * 0.15) + torch.rand(i.shape, generator=g)).long()
        parts.append(torch.stack([i + 4096 * s, j, k], -1).reshape(-1, 3))
    grid = igc.grid_build(torch.cat(parts).int().cuda())
    offsets = torch.tensor([0] + [p.shape[0] for p in parts]).cumsum(0).int().cuda()
    return grid, igc.kernel_map(grid), offsets


class ConditionedBlock:
    """Parameters (bf16, norms' in fp32) with the forward and backward pass above; `saved` holds what the forward pass keeps."""

    def __init__(self, channels: int, heads: int, state_channels: int, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        c, self.heads = channels, heads

        def weight(*shape, fan):
            return (torch.randn(*shape, generator=g) / fan ** 0.5).bfloat16().cuda()

        self.p = {"n1w": torch.ones(c).cuda(), "n1b": torch.zeros(c).cuda(), "n2w": torch.ones(c).cuda(), "n2b": torch.zeros(c).cuda(),
                  "wq": weight(c, c, fan=c), "wkv": weight(state_channels, 2 * c, fan=state_channels), "wo": weight(c, c, fan=c),
                  "conv": weight(27, c, c, fan=27 * c)}
        self.saved: dict = {}

    def forward(self, grid, kmap, offsets, x, states, state_offsets, state_mask=None):
        p, (n, c), h = self.p, x.shape, self.heads
        y1, ck1, r1 = igc.layer_norm_checkpoint(x, p["n1w"], p["n1b"])
        q = (y1 @ p["wq"]).view(n, h, c // h)
        kv = (states @ p["wkv"]).view(-1, 2, h, c // h)
        out, lse = igc.cross_attention(q, kv[:, 0], kv[:, 1], offsets, state_offsets, state_mask)
        x = x + out.view(n, c) @ p["wo"]
        y2, ck2, r2 = igc.layer_norm_checkpoint(x, p["n2w"], p["n2b"])
        y = x + igc.sparse_conv(grid, y2, p["conv"], kmap=kmap)
        self.saved = {"norm1": (ck1, r1), "norm2": (ck2, r2), "conv": igc.checkpoint_pack(y2), "q": q, "kv": kv, "out": out, "lse": lse}
        return y

    def backward(self, grid, kmap, offsets, dy, states, state_offsets, state_mask=None):
        """(gradient of x, gradients of the parameters) for the output gradient dy."""
        p, s, d = self.p, self.saved, {}
        n, c = dy.shape
        dg, d["conv"] = igc.sparse_conv_backward(grid, s["conv"], p["conv"], dy, kmap)
        dx, d["n2w"], d["n2b"] = igc.layer_norm_checkpoint_backward(dg, *s["norm2"], p["n2w"])
        dx = dx + dy
        d["wo"] = s["out"].view(n, c).t() @ dx
        dout = (dx @ p["wo"].t()).view(s["out"].shape)
        dq, dk, dv = igc.cross_attention_backward(dout, s["q"], s["kv"][:, 0], s["kv"][:, 1], s["out"], s["lse"], offsets, state_offsets,
                                                  state_mask)
        d["wkv"] = states.t() @ torch.stack([dk, dv], 1).view(states.shape[0], 2 * c)
        ck1, r1 = s["norm1"]
        y1 = (igc.checkpoint_unpack(ck1, torch.float32) * p["n1w"] + p["n1b"]).bfloat16()
        d["wq"] = y1.t() @ dq.view(n, c)
        dh, d["n1w"], d["n1b"] = igc.layer_norm_checkpoint_backward(dq.view(n, c) @ p["wq"].t(), ck1, r1, p["n1w"])
        return dx + dh, d

    def kept_bytes(self) -> int:
        def size(v):
            if isinstance(v, (tuple, list)):
                return sum(size(x) for x in v)
            return v.nbytes if isinstance(v, igc.Checkpoint8) else v.numel() * v.element_size()

        return sum(size(v) for v in self.saved.values())


def train(steps: int = 20, channels: int = 128, heads: int = 4, voxels: int = 20000, rate: float = 0.01, say=print) -> list[float]:
    grid, kmap, offsets = scene(3, voxels)
    n = grid.n_voxels
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, channels, generator=g, device="cuda").bfloat16()
    target = torch.randn(n, channels, generator=g, device="cuda")
    lengths = [77, 31, 130]
    state_offsets = torch.tensor([0] + lengths).cumsum(0).int().cuda()
    states = torch.randn(sum(lengths), 96, generator=g, device="cuda").bfloat16()
    mask = torch.rand(sum(lengths), generator=g, device="cuda") > 0.1  # padded states
    block, losses = ConditionedBlock(channels, heads, 96), []
    for step in range(steps):
        y = block.forward(grid, kmap, offsets, x, states, state_offsets, mask)
        diff = y.float() - target
        losses.append(float(diff.square().mean()))
        _, grads = block.backward(grid, kmap, offsets, (2 * diff / diff.numel() * 1e3).bfloat16(), states, state_offsets, mask)
        for name, grad in grads.items():
            w = block.p[name]
            w.copy_(w.float() - rate * grad.float().view(w.shape))
        say(f"step {step}: loss {losses[-1]:.4f}")
    say(f"{n} voxels, {channels} channels: the forward pass keeps {block.kept_bytes() / 1e6:.1f} MB")
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--channels", type=int, default=128)
    a.add_argument("--heads", type=int, default=4)
    a.add_argument("--voxels", type=int, default=20000)
    train(**vars(a.parse_args()))
