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


# ---------------------------------------------------------------- attention
# dtype, D, tokens, heads of a group: one MMA column tile, two, four, tcgen05, fp32 of one and two
PATHS = [("bf16", 128, 1, 4), ("bf16", 64, 3, 4), ("bf16", 64, 20, 2), ("bf16", 128, 30, 2), ("bf16", 128, 150, 1),
         ("f32", 64, 1, 2), ("f32", 128, 6, 2)]


def torch_dtype(dt):
    return torch.bfloat16 if dt == "bf16" else torch.float32


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(map(str, p)))
def test_attend_of_far_scores(path):
    """Scores of 2^16 to 2^110 where fp32 resolves no small difference: the row whose score is twice
    the others' takes all the weight (its score's error is 2^-16 of it at most), so O is its V."""
    from top_document_sparse_b200 import msa
    dt, D, T, G = path
    mem, content = memory(torch_dtype(dt), 1, D)
    g = torch.Generator(device="cuda").manual_seed(2)
    n, win = 200 + T, 77
    K = torch.zeros(1, n, 1, D, device="cuda")
    K[..., 0] = 0.5
    K[:, win, :, 0] = 1.0
    V = torch.randn(1, n, 1, D, generator=g, device="cuda").to(mem.dtype)
    cache = msa.Cache8(mem, 1, 512, 16, "int8", track_weights=True)
    cache.append(K.to(mem.dtype), V)
    want = cache.read(None, n)[1][0, win].double()
    ws = msa.workspace(cache.attend_workspace_size(T, 0, G))
    for e in list(range(16, 40)) + [64, 110]:
        for f in (1.0, 1.375, 1.75):
            Q = torch.zeros(1, T, G, D, dtype=mem.dtype, device="cuda")
            Q[..., 0] = f * 2.0 ** e
            O = torch.empty_like(Q)
            cache.attend(None, None, Q, O, ws, weight_decay=0.0)
            # one weight of 1, rounded to fp16 (2^-11) or its head and tail, over its own sum
            err = (O.double() - want).abs()
            assert torch.all(err <= 2.0 ** -8 * want.abs() if dt == "bf16" else err <= 2.0 ** -20 * want.abs()), (e, f)
            w = cache.weights[0, 0, :n].clone()
            assert abs(float(w[win]) - T * G) <= 2.0 ** -10 * T * G, (e, f)
            w[win] = 0.0
            assert torch.all(w == 0), (e, f)
    assert msa.device_error() == 0
