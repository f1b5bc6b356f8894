"""Window attention over batches of short sequences, whose launches have more workgroups than rows fill: results and gradients
against the formulas in float64, on either side of each choice of shapes (see tests/test_gpu_window.py for the bounds)."""
import pytest
import torch

from tests._gpu import require_gpu
from tests.test_gpu_window import check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


BATCHES = [(200, 64), (135, 64), (130, 40), (100, 100), (68, 100), (64, 128), (45, 192), (34, 256), (64, 192), (300, 17)]


@pytest.mark.parametrize("sequences,rows", BATCHES)
@pytest.mark.parametrize("dtype,dim", [(torch.float32, 32), (torch.float32, 40), (torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 128)])
def test_short_sequences(sequences, rows, dtype, dim):
    check([rows] * sequences, [rows] * sequences, 2, 2, dim, dtype, 50, 0, 3)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_short_sequences_of_many_lengths(dtype):
    lengths = [(37 * i) % 130 for i in range(150)]  # some empty, up to 129 rows
    check(lengths, lengths, 4, 2, 64, dtype, 30, 30, 70, masked=0.2)
    check([max(1, n // 3) for n in lengths], lengths, 4, 2, 64, dtype, 30, 0, 5)
