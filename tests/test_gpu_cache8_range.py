"""The 8-bit cache's operators at the ends of their ranges: sizes and counts beyond the capacity, blocks
whose scales lie far apart, scores far outside fp16, against tests/cache8_ref.py."""
import numpy as np
import pytest
import torch

from cache8_ref import f64
from test_gpu_cache8 import equal_cache, filled, memory

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("budget,recent", [(2 ** 31 - 1, 2 ** 31 - 1), (2 ** 31 - 1, 2 ** 31 - 64),
                                           (257, 257), (256, 256), (200, 200)])
def test_evict_with_budgets_beyond_the_capacity(budget, recent, in_place):
    """Any budget and recent up to 2^31 - 1 are accepted; beyond the capacity they keep every row."""
    from top_document_sparse_b200 import msa
    mem, _ = memory(torch.bfloat16, 2, 64)
    cache, ref = filled(mem, 3, 256, 64, "int8", [256, 201, 0], seed=3, track=True)
    cache.weights.copy_(torch.rand(cache.weights.shape, device="cuda"))
    ref.load(cache)
    ws = msa.workspace(cache.evict_workspace_size() + 4096)
    used = cache.evict_workspace_size()
    ws.fill_(0x5A)
    got = cache if in_place else msa.Cache8(mem, 3, 256, 64, "int8", track_weights=True)
    cache.evict(budget, recent, ws[:used], out=None if in_place else got)
    ref.evict(min(budget, 256), min(recent, 256))
    equal_cache(got, ref)
    for b in range(3):
        n = int(ref.lens[b])
        assert np.array_equal(f64(got.weights[b, :, :n]), ref.w[b, :, :n])
    assert torch.all(ws[used:] == 0x5A)
    assert msa.device_error() == 0
