"""Several calls of dropout in one captured step share a counter on the device and differ by their offsets."""
import numpy as np
import pytest
import torch

from tests._gpu import require_gpu, say
from tests.test_gpu_dropout import bits

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_two_calls_of_a_captured_step_drop_other_elements(dtype):
    import sparse_convolution_amd as igc
    say(f"dropout counter {dtype}")
    n, p, seed, offsets = 10007, 0.25, 77, (0, 1 << 32, (1 << 64) - 1)
    x, r = [torch.randn(n, device="cuda").to(dtype) for _ in range(2)]
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step():
        return [(igc.dropout(x, p, seed, o, r, counter), igc.dropout(x, p, seed, o, counter=counter),
                 igc.dropout_backward(x, p, seed, o, counter)) for o in offsets]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
            counter += 1
    torch.cuda.synchronize()
    counter.fill_(5)
    for count in range(5, 9):
        graph.replay()
        torch.cuda.synchronize()
        kept = []
        for o, (y, z, dx) in zip(offsets, got):
            at = (o + count) % (1 << 64)
            assert torch.equal(y, igc.dropout(x, p, seed, at, r)) and torch.equal(z, igc.dropout(x, p, seed, at)) and torch.equal(dx, z)
            kept.append(bits(0, n, seed, at) >= round(65536 * p))
            assert torch.equal((z == 0).cpu() | (x == 0).cpu(), torch.from_numpy(~kept[-1]) | (x == 0).cpu())
        # Independent masks agree in p^2 + (1 - p)^2 of the places.
        for i, j in ((0, 1), (0, 2), (1, 2)):
            assert abs(float(np.mean(kept[i] == kept[j])) - 0.625) < 5 * (0.625 * 0.375 / n) ** 0.5
        assert int(counter) == count + 1


def test_refusals():
    import sparse_convolution_amd as igc
    say("dropout counter refusals")
    x, one = torch.zeros(4, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="offset is a number"):
        igc.dropout(x, 0.1, 3, one, counter=one)
    with pytest.raises(TypeError, match="counter must have dtype"):
        igc.dropout(x, 0.1, 3, counter=one.int())
    with pytest.raises(ValueError, match="counter must have shape"):
        igc.dropout_backward(x, 0.1, 3, counter=torch.zeros(2, dtype=torch.int64, device="cuda"))
    with pytest.raises(TypeError, match="counter must be a CUDA"):
        igc.dropout(x, 0.1, 3, counter=one.cpu())
    with pytest.raises(ValueError, match="seed and offset"):
        igc.dropout(x, 0.1, 3, -1, counter=one)
