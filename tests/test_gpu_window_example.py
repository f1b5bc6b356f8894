"""The example's training step applies its gradients: each parameter moves against its gradient by the rate, and by nothing else."""
import os
import sys

import pytest
import torch

from tests._gpu import require_gpu, say

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def test_updates_are_applied(monkeypatch):
    require_gpu()
    import window_block as ex
    say("window example's updates")
    seen = []

    class Watched(ex.WindowBlock):
        def backward(self, *args):
            dx, grads = super().backward(*args)
            seen.append((self, {k: v.clone() for k, v in self.p.items()}, grads))
            return dx, grads

    monkeypatch.setattr(ex, "WindowBlock", Watched)
    rate = 0.02
    ex.train(steps=2, channels=64, heads=2, voxels=3000, window=40, rate=rate, say=say)
    assert len(seen) == 2
    block, before, grads = seen[0]
    after = seen[1][1]
    assert before.keys() == grads.keys()
    for name, w in before.items():
        assert bool((grads[name] != 0).any()) and not torch.equal(after[name], w), name
        assert torch.equal(after[name], (w.float() - rate * grads[name].float().view(w.shape)).to(w.dtype)), name
    # The last step's update reaches the block too.
    for name, w in seen[1][1].items():
        assert not torch.equal(block.p[name], w), name
