"""The layer's operators on batches of 2^32 threads and more, which one dimension of a launch does not take."""

import pytest
import torch

import routing_fp8_grouped_amd as moe
from tests.gpu_util import DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs an MI355X")


def test_quant():
    """2^28 tiles and some (2^32 threads of 16 a tile): the tiles that are not zeros, and that all others are."""
    rows = (1 << 28) + 5
    at = torch.tensor([0, 1, 17, rows // 2, (1 << 28) - 1, 1 << 28, rows - 1], device=DEV)
    x = torch.zeros(rows, 128, dtype=torch.bfloat16, device=DEV)
    few = (torch.randn(len(at), 128, generator=torch.Generator().manual_seed(5)) * 3).bfloat16().to(DEV)
    x[at] = few
    q, s = torch.full((rows, 128), 7, dtype=torch.uint8, device=DEV), torch.full((rows, 1), 7.0, device=DEV)
    moe.fp8_quant_1x128(x, q, s)
    q2, s2 = torch.empty(len(at), 128, dtype=torch.uint8, device=DEV), torch.empty(len(at), 1, device=DEV)
    moe.fp8_quant_1x128(few, q2, s2)
    assert torch.equal(q[at], q2) and torch.equal(s[at], s2)
    q[at], s[at] = 0, 1.0
    assert not q.view(torch.int64).any() and (s == 1).all()
    del x, q, s
    torch.cuda.empty_cache()
