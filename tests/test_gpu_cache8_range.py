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


# ---------------------------------------------------------------- attention, bounds by row
U = 2.0 ** -23
QMAX = {"int8": 127.0, "e4m3": 448.0}


def expected(ref, mem_rows, Q, n, bf16):
    """O, lse, weights and their bounds in fp64.  First order in u = 2^-23, for each column by itself:
      ds_j = (D + 17) u sum_d |q_d k_jd| / sqrt(D)  (sums on the tensor cores may truncate)
             + sum_d (lost(q_d) |k_jd| + [memory row] 2^6 lost(k_jd) |q_d|) / sqrt(D)
      lost : 2^-25 of a row's largest element for elements whose bits reach below fp16's smallest
             step there: bf16's 8 bits below 2^-16 of the largest, fp32's all (zeros lose nothing);
             a memory row of K shares a power of two with rows up to 2^6 larger
      dl   = sum_j p_j ds_j + (rows + 8) u                        of the log-sum
      O    : sum_j p_j |v_j| (ds_j + dl + w + (rows + 16) u), w the rounding of a weight: 2^-11 to
             fp16 (bf16 queries), 2^-22 to its head and tail (fp32)
             + 2^-28 P sum_j |v_j| / s_j: weights below fp16's normal range, half its smallest step
             2^-25 against weights times scales kept at 2^11 2^-8 of P = max_j p_j s_j or above
    (memory rows: V and a weight's head and tail are bf16, nothing is below their normal range).
    A block or a row of little weight enters by that weight alone, however large its values are."""
    B, T, Hq, D = Q.shape

    def lost(x, below=1.0):
        a = np.abs(x)
        top = below * a.max(-1, initial=0.0, keepdims=True)
        return np.where((a > 0) & ((a < 2.0 ** -16 * top) | (not bf16)), 2.0 ** -25 * top, 0.0)

    G, w = Hq // ref.H, 2.0 ** -11 if bf16 else 2.0 ** -22
    O, tol = np.zeros(Q.shape), np.zeros(Q.shape)
    lse, tl = np.zeros((B, T, Hq)), np.zeros((B, T, Hq))
    W, tw = np.zeros((B, ref.H, ref.cap)), np.zeros((B, ref.H, ref.cap))
    for b in range(B):
        ln = int(ref.lens[b])
        for g in range(ref.H):
            M = mem_rows[b][0].shape[0]
            K = np.concatenate([mem_rows[b][0][:, g], ref.values(b, g, "k")])
            V = np.concatenate([mem_rows[b][1][:, g], ref.values(b, g, "v")])
            s = np.concatenate([np.zeros(M), np.repeat(ref.vs[b, g], ref.bl)[:ln]])
            vq = np.where(s[:, None] > 0, np.abs(V) / np.where(s > 0, s, 1.0)[:, None], 0.0)
            kl = np.concatenate([lost(K[:M], 64.0), np.zeros((ln, D))])
            for t in range(int(n[b])):
                seen = M + max(0, ln - int(n[b]) + t + 1)
                rows = seen
                for h in range(g * G, (g + 1) * G):
                    q = Q[b, t, h]
                    if seen == 0:
                        lse[b, t, h] = -np.inf
                        continue
                    z = K[:seen] @ q / D ** 0.5
                    ds = ((D + 17) * U * (np.abs(K[:seen]) @ np.abs(q)) + np.abs(K[:seen]) @ lost(q)
                          + kl[:seen] @ np.abs(q)) / D ** 0.5
                    p = np.exp(z - z.max())
                    lse[b, t, h] = z.max() + np.log(p.sum())
                    p /= p.sum()
                    dl = p @ ds + (rows + 8) * U
                    a = np.abs(V[:seen])
                    O[b, t, h] = p @ V[:seen]
                    tol[b, t, h] = ((p * (ds + dl + w + (rows + 16) * U)) @ a
                                    + 2.0 ** -28 * (p * s[:seen]).max() * vq[:seen].sum(0))
                    tl[b, t, h] = dl + 4 * U * abs(lse[b, t, h])
                    W[b, g, :seen - M] += p[M:]
                    tw[b, g, :seen - M] += p[M:] * (ds[M:] + tl[b, t, h] + 16 * U)
    if bf16:
        tol = tol + 2.0 ** -8 * (np.abs(O) + tol)
    return O, tol, lse, tl, W, tw


def check_attend(mem, content, cache, Q, ids=None):
    from top_document_sparse_b200 import msa
    import cache8_ref as R
    B, T, Hq, D = Q.shape
    ref = R.RefCache(B, mem.n_kv_heads, cache.capacity, D, cache.block_len, cache.fmt).load(cache)
    rows = R.content_rows(mem, content, ids) if ids is not None else \
        [(np.zeros((0, mem.n_kv_heads, D)),) * 2] * B
    k = 0 if ids is None else ids.shape[1]
    O, lse = torch.empty_like(Q), torch.empty(B, T, Hq, device="cuda")
    cache.attend(content, ids, Q, O, msa.workspace(cache.attend_workspace_size(T, k, Hq)), lse=lse,
                 weight_decay=None if cache.weights is None else 0.0)
    want, tol, wl, tl, W, tw = expected(ref, rows, f64(Q), [T] * B, Q.dtype == torch.bfloat16)
    err = np.abs(f64(O) - want)
    assert np.all(err <= tol), f"O off by {np.nanmax(err / np.maximum(tol, 1e-300)):.3g} times its bound"
    assert np.all(np.abs(f64(lse) - wl) <= tl)
    if cache.weights is not None:
        for b in range(B):
            n = int(ref.lens[b])
            assert np.all(np.abs(f64(cache.weights[b, :, :n]) - W[b, :, :n]) <= tw[b, :, :n] + 2.0 ** -100)
    assert msa.device_error() == 0


# dtype, D, tokens, heads of a group: one MMA column tile, two, four, tcgen05, fp32 of one and two
PATHS = [("bf16", 128, 1, 4), ("bf16", 64, 3, 4), ("bf16", 64, 20, 2), ("bf16", 128, 30, 2), ("bf16", 128, 150, 1),
         ("f32", 64, 1, 2), ("f32", 128, 6, 2)]


def torch_dtype(dt):
    return torch.bfloat16 if dt == "bf16" else torch.float32


def rows_and_queries(dt, D, T, G, n, seed):
    """K, V of n rows and T x G queries; dimension 0 of every query is 8, dimension 1 is 0."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    kv = torch.randn(2, 1, n, 1, D, generator=g, device="cuda")
    Q = torch.randn(1, T, G, D, generator=g, device="cuda")
    kv[0, ..., :2] = 0.0
    Q[..., 0], Q[..., 1] = 8.0, 0.0
    return kv, Q


def light(K, rows, D, log2_weight=60.0):
    """K[rows] such that every query gives them 2^-log2_weight of an ordinary row's weight."""
    K[:, rows, :, 0] = -log2_weight * 0.6931 * D ** 0.5 / 8.0


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("r", [0, 16, 24, 28, 60])
def test_attend_after_a_light_block_of_huge_values(path, fmt, r):
    """Blocks whose V is 2^r times the others' and whose weight is nothing, each followed by an
    ordinary one, so that every warp of every split meets both, the light one first."""
    from top_document_sparse_b200 import msa
    dt, D, T, G = path
    mem, content = memory(torch_dtype(dt), 1, D)
    n = 8192
    kv, Q = rows_and_queries(dt, D, T, G, n, seed=r + D)
    for x in range(0, n, 128):
        light(kv[0], slice(x, x + 64), D)
        kv[1, :, x:x + 64] *= 2.0 ** r
    cache = msa.Cache8(mem, 1, n, 64, fmt)
    cache.append(kv[0].to(mem.dtype), kv[1].to(mem.dtype))
    check_attend(mem, content, cache, Q.to(mem.dtype))


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("small", [2.0 ** -27, 2.0 ** -100])
def test_attend_after_a_block_of_zeros(path, small):
    """All-zero rows (they carry weight) before and among rows of small V."""
    from top_document_sparse_b200 import msa
    dt, D, T, G = path
    mem, content = memory(torch_dtype(dt), 1, D)
    kv, Q = rows_and_queries(dt, D, T, G, 192 + T, seed=D)
    kv[1] *= small
    kv[:, :, :64] = 0.0
    kv[:, :, 80:96] = 0.0
    cache = msa.Cache8(mem, 1, 512, 16, "int8")
    cache.append(kv[0].to(mem.dtype), kv[1].to(mem.dtype))
    check_attend(mem, content, cache, Q.to(mem.dtype))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("r", [12, 18, 24, 25, 26, 60])
def test_attend_blocks_of_16_rows_far_apart(path, fmt, r):
    """Neighbouring blocks whose K and V scales are 2^r apart: K by a dimension that no query has, V
    in rows of no weight."""
    from top_document_sparse_b200 import msa
    dt, D, T, G = path
    mem, content = memory(torch_dtype(dt), 1, D)
    kv, Q = rows_and_queries(dt, D, T, G, 160 + T, seed=r + D)
    light(kv[0], slice(0, 16), D)
    kv[1, :, :16] *= 2.0 ** r
    kv[0, :, 48:64, :, 1] = 2.0 ** r
    light(kv[0], slice(96, 112), D)
    kv[1, :, 96:112] *= 2.0 ** r
    kv[0, :, 96:112, :, 1] = 2.0 ** r
    cache = msa.Cache8(mem, 1, 512, 16, fmt, track_weights=True)
    cache.append(kv[0].to(mem.dtype), kv[1].to(mem.dtype))
    check_attend(mem, content, cache, Q.to(mem.dtype))


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("r", [0, 12, 24, 60])
def test_attend_memory_rows_far_apart(path, r):
    """One memory row with V 2^r times the others' and no weight, one with K 2^r larger in a
    dimension that no query has, rows of zeros; few and tiny local rows."""
    from top_document_sparse_b200 import msa
    dt, D, T, G = path
    mem, content = memory(torch_dtype(dt), 1, D, docs=(64 * 40, 64 * 3))
    kv, Q = rows_and_queries(dt, D, T, G, mem.n_chunks, seed=r)
    kv = kv[:, 0]
    light(kv[0][None], slice(3, 4), D)
    kv[1, 3] *= 2.0 ** r
    kv[0, 7, :, 1] = 2.0 ** r
    kv[:, 11] = 0.0
    content.copy_(kv.transpose(0, 1).to(mem.dtype))
    cache = msa.Cache8(mem, 1, 256, 16, "int8")
    loc = torch.randn(2, 1, T, 1, D, device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    cache.append(loc[0].to(mem.dtype), (loc[1] * 2.0 ** -r).to(mem.dtype))
    ids = torch.tensor([[0, 1]], dtype=torch.int32, device="cuda")
    check_attend(mem, content, cache, Q.to(mem.dtype), ids)


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


@pytest.mark.parametrize("path", PATHS, ids=lambda p: "-".join(map(str, p)))
@pytest.mark.parametrize("r", [1, 3, 10])
def test_attend_of_far_scores_in_smaller_blocks(path, r):
    """The same where V of the row that takes all the weight is 2^r below the other blocks', which its
    warp has met before it."""
    from top_document_sparse_b200 import msa
    dt, D, T, G = path
    mem, content = memory(torch_dtype(dt), 1, D)
    g = torch.Generator(device="cuda").manual_seed(2)
    n, win = 8192, 77
    K = torch.zeros(1, n, 1, D, device="cuda")
    K[..., 0] = 0.5
    K[:, win, :, 0] = 1.0
    V = torch.randn(1, n, 1, D, generator=g, device="cuda") * 2.0 ** r
    V[:, 64:80] *= 2.0 ** -r
    cache = msa.Cache8(mem, 1, n, 16, "int8")
    cache.append(K.to(mem.dtype), V.to(mem.dtype))
    want = cache.read(None, n)[1][0, win].double()
    ws = msa.workspace(cache.attend_workspace_size(T, 0, G))
    for e in list(range(16, 40)) + [64, 110]:
        for f in (1.0, 1.375, 1.75):
            Q = torch.zeros(1, T, G, D, dtype=mem.dtype, device="cuda")
            Q[..., 0] = f * 2.0 ** e
            O = torch.empty_like(Q)
            cache.attend(None, None, Q, O, ws)
            err = (O.double() - want).abs()
            assert torch.all(err <= 2.0 ** -8 * want.abs() if dt == "bf16" else err <= 2.0 ** -20 * want.abs()), (e, f)
    assert msa.device_error() == 0
