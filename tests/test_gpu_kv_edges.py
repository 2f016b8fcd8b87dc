"""The key/value cache's calls where they can go wrong: what the plain tests of
test_gpu_kv.py do not reach. GPU only."""
import pytest
import torch

from operator_reference import gen
from test_gpu_kv import check_evict

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------- evict


@pytest.mark.parametrize("middle", [1, 2, 33, 63, 64, 65, 96, 127, 128])
def test_evict_short_middles(middle):
    """Few rows to choose from, no two weights alike: waves without a row of their own."""
    def distinct(shape):
        order = torch.stack([torch.randperm(shape[-1], generator=gen(i)) for i in range(shape[0] * shape[1])])
        return ((order + 1).float() * 2.0 ** -7).view(shape)

    n, sinks, recent = middle + 24, 4, 20
    for budget in sorted({sinks + recent, n - 1, sinks + recent + middle // 2}):
        check_evict([n, n + 1], 64, 64, 16, budget, sinks, recent, seed=middle, acc=distinct)
