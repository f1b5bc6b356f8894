"""Single tokens behind caches with a workgroup or more for every CU: their windows are read whole up to some rounds of keys, in parts
beyond (see tests/test_gpu_window.py for the bounds)."""
import pytest
import torch

from tests import test_gpu_window as window
from tests._gpu import require_gpu

pytestmark = pytest.mark.gpu
F32, BF16 = torch.float32, torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


@pytest.mark.parametrize("left,sinks", [(700, 4), (2600, 0)])
@pytest.mark.parametrize("group", [1, 2, 4])
@pytest.mark.parametrize("dtype,dim", [(F32, 32), (F32, 64), (F32, 128), (BF16, 64)])
def test_many_tokens(dtype, dim, group, left, sinks):
    # 280 workgroups; caches of 0 to 3,312 keys, an average of 1,656.
    keys = [48 * i for i in range(70)]
    window.check([1] * 70, keys, 4 * group, 4, dim, dtype, left, 0, sinks)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("left", [300, 1900])
def test_many_masked_tokens(dtype, left):
    window.check([1] * 130, [(997 * i) % 2200 for i in range(130)], 4, 2, 64, dtype, left, 0, 6, masked=0.3)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("left,right,sinks", [(255, 0, 4), (1700, 0, 0)])
def test_many_tokens_in_caches_with_room(dtype, left, right, sinks):
    window.test_caches_with_room([1] * 130, [(997 * i) % 2200 for i in range(130)], 2200, 4, 2, 64, left, right, sinks, dtype)
