"""A self-attention block over voxels in grid order, trained, and read row by row.

    python examples/window_block.py [--steps 20] [--channels 128] [--heads 4] [--voxels 20000] [--window 128]

Several scenes share one grid (each in a root tile of its own, so their rows are contiguous and neighbours in space are mostly
neighbours in order). A few tokens stand before each scene's voxels: every later row sees them besides its window. With x the rows'
features and ijk their coordinates (0 for tokens):

    q, k, v = layer_norm(x) Wqkv
    q, k    = qk_norm_rotary(q, k, ijk)                      each head normed, turned by three axes of positions
    y       = x + dropout(window_attention(q, k, v) Wo)      the mask is computed again in the backward pass

`step` is the same block for one new row of each sequence behind a cache of keys and values (windows that look back only). The
linear projections are plain torch products.
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import sparse_convolution_amd as igc  # noqa: E402

TOKENS = 4


def scene(n_scenes: int, voxels: int, seed: int = 0):
    """(coordinates int32 [rows, 3], row offsets of the scenes): TOKENS rows of zeros, then a scene's voxels in the grid's order."""
    g = torch.Generator().manual_seed(seed)
    parts, side = [], max(2, int((voxels / n_scenes) ** 0.5))
    for s in range(n_scenes):
        i, j = torch.meshgrid(torch.arange(side + s), torch.arange(side), indexing="ij")
        k = (30 + 8 * torch.sin(i * 0.2 + s) + 6 * torch.cos(j * 0.15) + torch.rand(i.shape, generator=g)).long()
        parts.append(torch.stack([i + 4096 * s, j, k], -1).reshape(-1, 3))
    ijk = igc.grid_build(torch.cat(parts).int().cuda()).active_ijk()
    rows, first = [], 0
    for p in parts:
        rows += [torch.zeros(TOKENS, 3, dtype=torch.int32, device="cuda"), ijk[first:first + p.shape[0]]]
        first += p.shape[0]
    offsets = torch.tensor([0] + [p.shape[0] + TOKENS for p in parts]).cumsum(0).int().cuda()
    return torch.cat(rows).contiguous(), offsets


class WindowBlock:
    """Parameters (bf16, norms' in fp32) with the forward and backward pass above; `saved` holds what the forward pass keeps. right 0:
    no row looks ahead."""

    def __init__(self, channels: int, heads: int, kv_heads: int, left: int, right: int, drop: float = 0.1, seed: int = 0):
        g = torch.Generator().manual_seed(seed)
        c, self.heads, self.kv_heads, self.dim = channels, heads, kv_heads, channels // heads
        self.left, self.right, self.drop, self.seed = left, right, drop, seed

        def weight(*shape):
            return (torch.randn(*shape, generator=g) / shape[0] ** 0.5).bfloat16().cuda()

        self.p = {"nw": torch.ones(c).cuda(), "nb": torch.zeros(c).cuda(), "qkv": weight(c, (heads + 2 * kv_heads) * self.dim), "wo": weight(c, c),
                  "qw": torch.ones(self.dim).cuda(), "kw": torch.ones(self.dim).cuda()}
        self.frequencies = igc.rotary_frequencies(self.dim, base=1000.0, axes=3).cuda()
        self.saved: dict = {}

    def _heads(self, h):
        """Queries, keys and values of normed rows: slices of one product."""
        t = (h @ self.p["qkv"]).view(h.shape[0], self.heads + 2 * self.kv_heads, self.dim)
        return t[:, :self.heads], t[:, self.heads:self.heads + self.kv_heads], t[:, self.heads + self.kv_heads:]

    def forward(self, x, ijk, offsets, count=0):
        """count numbers the steps of training: each drops other elements."""
        p, n = self.p, x.shape[0]
        h, mean, rstd = igc.layer_norm(x, p["nw"], p["nb"])
        q, k, v = self._heads(h)
        qr, kr = igc.qk_norm_rotary(q, k, ijk, self.frequencies, p["qw"], p["kw"])
        out, lse = igc.window_attention(qr, kr, v, self.left, self.right, TOKENS, offsets, offsets)
        y = igc.dropout(out.view(n, -1) @ p["wo"], self.drop, self.seed, count, residual=x)
        self.saved = {"x": x, "h": h, "norm": (mean, rstd), "q": q, "k": k, "v": v, "qr": qr, "kr": kr, "out": out, "lse": lse, "count": count}
        return y

    def backward(self, dy, ijk, offsets):
        """(gradient of x, gradients of the parameters) for the output gradient dy."""
        p, s, d, n = self.p, self.saved, {}, dy.shape[0]
        dz = igc.dropout_backward(dy, self.drop, self.seed, s["count"])
        d["wo"] = s["out"].view(n, -1).t() @ dz
        dout = (dz @ p["wo"].t()).view(s["out"].shape)
        dq, dk, dv = igc.window_attention_backward(dout, s["qr"], s["kr"], s["v"], s["out"], s["lse"], self.left, self.right, TOKENS, offsets,
                                                   offsets)
        dq, dk, d["qw"], d["kw"] = igc.qk_norm_rotary_backward(dq, dk, s["q"], s["k"], ijk, self.frequencies, p["qw"], p["kw"])
        dqkv = torch.cat([dq, dk, dv], 1).view(n, -1)
        d["qkv"] = s["h"].t() @ dqkv
        dx, d["nw"], d["nb"] = igc.layer_norm_backward(dqkv @ p["qkv"].t(), s["x"], *s["norm"], p["nw"])
        return dx + dy, d

    def step(self, x, ijk, cache_k, cache_v, lengths):
        """One new row of each sequence, x [batch, channels], behind the `lengths` (int32 [batch]) rows in use of caches [batch, room,
        kv_heads, dim]: the block's output without dropout. Adds the row to the caches and to lengths."""
        p, (batch, room) = self.p, cache_k.shape[:2]
        h, _, _ = igc.layer_norm(x, p["nw"], p["nb"])
        q, k, v = self._heads(h)
        q, k = igc.qk_norm_rotary(q, k, ijk, self.frequencies, p["qw"], p["kw"])
        one = torch.arange(batch + 1, dtype=torch.int32, device=x.device)
        at = (one[:-1], lengths.long())
        cache_k[at], cache_v[at] = k, v
        lengths += 1
        out, _ = igc.window_attention(q, cache_k.flatten(0, 1), cache_v.flatten(0, 1), self.left, 0, TOKENS, one, one * room, kv_lengths=lengths)
        return x + out.view(batch, -1) @ p["wo"]


def train(steps: int = 20, channels: int = 128, heads: int = 4, voxels: int = 20000, window: int = 128, rate: float = 0.01, say=print) -> list[float]:
    ijk, offsets = scene(3, voxels)
    n = ijk.shape[0]
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(n, channels, generator=g, device="cuda").bfloat16()
    target = torch.randn(n, channels, generator=g, device="cuda")
    block, losses = WindowBlock(channels, heads, heads // 2 or 1, window, window), []
    for step in range(steps):
        diff = block.forward(x, ijk, offsets, step).float() - target
        losses.append(float(diff.square().mean()))
        _, grads = block.backward((2 * diff / diff.numel() * 1e3).bfloat16(), ijk, offsets)
        for name, grad in grads.items():
            w = block.p[name]
            w.copy_(w.float() - rate * grad.float().view(w.shape))
        say(f"step {step}: loss {losses[-1]:.4f}")
    say(f"{n} rows, {channels} channels")
    return losses


if __name__ == "__main__":
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--channels", type=int, default=128)
    a.add_argument("--heads", type=int, default=4)
    a.add_argument("--voxels", type=int, default=20000)
    a.add_argument("--window", type=int, default=128)
    train(**vars(a.parse_args()))
