"""The 8-bit local cache on the GPU against its plain 64-bit restatement (tests/cache8_ref.py).

Stored values, scales and lengths have to be equal: dividing by a power of two is exact, so the
rounding is the same in any precision.  Attention bounds, per output, first order in
u = 2^-23 (tensor-core sums may truncate):
  ds  = (D + 16) u A, A = max_j sum_d |q_d k_jd| / sqrt(D)          error of a score
  lse : ds + (rows + 8) u + 4 u |lse|
  O   : (2 ds + w + (rows + 16) u) sum_j p_j |v_j| + rows 2^-28 max|v|,
        w the rounding of a weight, 2^-11 to fp16 (bf16 queries) and 2^-22 to an fp16 head and
        tail (fp32 queries, whose Q is split alike: 2^-22 again, inside ds), the last term weights below fp16's normal
        range: half its smallest step, 2^-25, against weights kept at 2^11 2^(s - m) with m at
        most 8 above the largest score, 2^-25 2^-11 2^8 = 2^-28 of the largest weight;
        a bf16 output adds half a step, 2^-8 |O|
  weights : (ds + lse's bound + 16 u) w a token."""
import numpy as np
import pytest
import torch

import cache8_ref as R
from cache8_ref import f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -23
BAD_DOC_ID = 0x1


def memory(dtype, H, D, docs=(70, 1, 64, 200, 129, 33)):
    from top_document_sparse_b200 import msa
    off = np.concatenate([[0], np.cumsum(docs)])
    mem = msa.Memory(off, 64, H, D, 8, 128, dtype, 1e6, 64)
    g = torch.Generator(device="cuda").manual_seed(7)
    content = (torch.randn(mem.n_chunks, 2, H, D, generator=g, device="cuda") * 0.5).to(dtype)
    return mem, content


def equal_cache(cache, ref, what=""):
    assert np.array_equal(cache.cache_len.cpu().numpy(), ref.lens), what
    for b in range(ref.B):
        n = int(ref.lens[b])
        nb = -(-n // ref.bl)
        for its, mine, s, ms in ((cache.k, ref.k, cache.k_scale, ref.ks), (cache.v, ref.v, cache.v_scale, ref.vs)):
            assert np.array_equal(f64(s[b, :, :nb]), ms[b, :, :nb]), f"{what} scales of query {b}"
            assert np.array_equal(f64(its[b, :, :n].float()), mine[b, :, :n]), f"{what} rows of query {b}"


def poison(cache):
    """Bytes, scales and weights that no kernel may use: NaN everywhere (0x7f is e4m3's NaN)."""
    cache.k.view(torch.int8).fill_(0x7F)
    cache.v.view(torch.int8).fill_(0x7F)
    cache.k_scale.fill_(float("nan"))
    cache.v_scale.fill_(float("nan"))
    if cache.weights is not None:
        cache.weights.fill_(float("nan"))


def filled(mem, B, cap, bl, fmt, lens, seed, track=False, spread=0.0):
    """A poisoned cache with lens[b] appended rows, and its reference."""
    from top_document_sparse_b200 import msa
    cache = msa.Cache8(mem, B, cap, bl, fmt, track_weights=track)
    poison(cache)
    H, D, T = mem.n_kv_heads, mem.head_dim, max(max(lens), 1)
    g = torch.Generator(device="cuda").manual_seed(seed)
    kv = torch.randn(2, B, T, H, D, generator=g, device="cuda")
    if spread:  # blocks of very different magnitude
        kv = kv * torch.exp2(spread * torch.randn(2, 1, T, 1, 1, generator=g, device="cuda"))
    kv = kv.to(mem.dtype)
    cache.append(kv[0], kv[1], n_tokens=torch.tensor(lens, dtype=torch.int32, device="cuda"))
    return cache, R.RefCache(B, H, cap, D, bl, fmt).load(cache)


# ---------------------------------------------------------------- append and read
@pytest.mark.parametrize("dt,fmt,D,H,bl", [("bf16", "int8", 128, 2, 64), ("bf16", "e4m3", 64, 3, 16),
                                           ("f32", "int8", 64, 1, 32), ("f32", "e4m3", 128, 2, 128)])
def test_append_token_by_token_chunks_and_rollback(dt, fmt, D, H, bl):
    from top_document_sparse_b200 import msa
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    mem, _ = memory(dtype, H, D)
    B, cap = 3, 256
    cache = msa.Cache8(mem, B, cap, bl, fmt, track_weights=True)
    poison(cache)
    ref = R.RefCache(B, H, cap, D, bl, fmt)
    rng = np.random.default_rng(3)
    g = torch.Generator(device="cuda").manual_seed(5)
    lens = np.zeros(B, dtype=np.int64)
    flags = 0
    for i, T in enumerate([1, 1, 1, bl - 3, 1, 1, 37, 1, 2 * bl + 5, 1, 3]):
        n = rng.integers(0, T + 1, B) if i % 3 == 2 else np.full(B, T)
        start = None
        if i in (5, 9):  # drop some rows first, once to a block's first row
            start = np.maximum(lens - [1, 5, 9], 0)
            start[0] = start[0] // bl * bl
        # growing magnitudes: later rows force larger scales of partly filled blocks
        kv = torch.randn(B, T, 2 * H * D, generator=g, device="cuda") * 2.0 ** rng.integers(-4, 4 + i)
        kv = kv.to(dtype)
        K, V = kv[..., :H * D].view(B, T, H, D), kv[..., H * D:].view(B, T, H, D)
        i32 = lambda x: None if x is None else torch.tensor(x, dtype=torch.int32, device="cuda")
        cache.append(K, V, n_tokens=i32(n) if i % 3 == 2 else None, start=i32(start))
        ref.append(f64(K), f64(V), n, start)
        if np.any((lens if start is None else start) + n > cap):
            flags = msa.DEVERR_CACHE_OVERFLOW  # 2 * 128 + 5 new rows do not fit
        lens = ref.lens.copy()
        equal_cache(cache, ref, f"step {i}")
        for b in range(B):
            assert torch.all(cache.weights[b, :, :lens[b]] == 0)
        begin = np.array([0, max(0, lens[1] - 7), 3])
        Kr, Vr = cache.read(i32(begin), 40)
        for out, which in ((Kr, "k"), (Vr, "v")):
            want = np.zeros((B, 40, H, D))
            for b in range(B):
                for h in range(H):
                    x = ref.values(b, h, which)[begin[b]:begin[b] + 40]
                    want[b, :len(x), h] = x
            assert np.array_equal(f64(out), want)
    assert msa.device_error() == flags


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_special_values(fmt):
    """Zero blocks, tiny and huge values, NaN and infinities, in place of a scale border."""
    from top_document_sparse_b200 import msa
    mem, _ = memory(torch.float32, 1, 64)
    cache = msa.Cache8(mem, 1, 64, 16, fmt)
    ref = R.RefCache(1, 1, 64, 64, 16, fmt)
    q = R.QMAX[fmt]
    x = np.zeros((1, 61, 1, 64), dtype=np.float32)
    x[0, 16, 0, :4] = [1e-30, -2e-38, 1e-45, 0]                 # a tiny block
    x[0, 32, 0, :5] = [3e38, -1e38, np.inf, -np.inf, np.nan]    # a huge one
    x[0, 48, 0, :3] = [q * 2.0 ** -7, -q * 2.0 ** -7, 0.5]      # exactly at a scale's border
    x[0, 49, 0, :3] = [2.5 * 2.0 ** -7, 3.5 * 2.0 ** -7, 0.5 * 2.0 ** -7]  # ties
    t = torch.from_numpy(x).cuda()
    cache.append(t, -t)
    ref.append(x, -x)
    equal_cache(cache, ref)
    y = np.zeros((1, 1, 1, 64), dtype=np.float32)
    y[..., 0] = np.nextafter(np.float32(q * 2.0 ** -7), np.float32(1e9))  # one step past the border
    cache.append(torch.from_numpy(y).cuda(), torch.from_numpy(y).cuda())
    ref.append(y, y)
    equal_cache(cache, ref, "past the border")
    assert msa.device_error() == 0


def test_append_flags_bad_lengths_and_overflow():
    from top_document_sparse_b200 import msa
    mem, _ = memory(torch.bfloat16, 2, 64)
    B, cap = 5, 32
    cache = msa.Cache8(mem, B, cap, 16, "int8")
    ref = R.RefCache(B, 2, cap, 64, 16, "int8")
    kv = torch.randn(2, B, 20, 2, 64, device="cuda").bfloat16()
    cache.append(kv[0], kv[1])
    ref.append(f64(kv[0]), f64(kv[1]))
    msa.device_error()
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    start, n = [20, -1, 33, 32, 3], [20, 1, 1, 1, 21]
    cache.append(kv[0], kv[1], n_tokens=i32(n), start=i32(start))
    ref.append(f64(kv[0]), f64(kv[1]), n, start)
    assert msa.device_error() == msa.DEVERR_BAD_LENGTH | msa.DEVERR_CACHE_OVERFLOW
    equal_cache(cache, ref)
    # at cache_len, without start
    cache.append(kv[0], kv[1], n_tokens=i32([1, 2, 3, 4, 5]))
    ref.append(f64(kv[0]), f64(kv[1]), [1, 2, 3, 4, 5])
    assert msa.device_error() == msa.DEVERR_CACHE_OVERFLOW
    equal_cache(cache, ref)


# ---------------------------------------------------------------- attention
def run_attend(mem, content, cache, ref, ids, T, G, n, q_scale=1.0, decay=None, seed=11):
    from top_document_sparse_b200 import msa
    B, H, D = cache.batch, mem.n_kv_heads, mem.head_dim
    g = torch.Generator(device="cuda").manual_seed(seed)
    Q = (torch.randn(B, T, H * G, D, generator=g, device="cuda") * q_scale).to(mem.dtype)
    O = torch.full((B, T, H * G, D), 7.0, device="cuda").to(mem.dtype)
    lse = torch.full((B, T, H * G), 7.0, device="cuda")
    k = ids.shape[1] if ids is not None else 0
    ws = msa.workspace(cache.attend_workspace_size(T, k, H * G))
    ws.fill_(0xFF)
    nt = None if n is None else torch.tensor(n, dtype=torch.int32, device="cuda")
    w0 = None if decay is None else f64(cache.weights)
    cache.attend(content, ids, Q, O, ws, lse=lse, n_tokens=nt, weight_decay=decay)
    cnt = [T] * B if n is None else n
    rows = R.content_rows(mem, content, ids) if k else [(np.zeros((0, H, D)),) * 2] * B
    want, wl, W, pv, amp = R.attend(ref, rows, f64(Q), cnt)
    vmax = max([np.abs(ref.values(b, h, "v")).max(initial=0.0) for b in range(B) for h in range(H)]
               + [np.abs(r[1]).max(initial=0.0) for r in rows])
    nrow = cache.capacity + 4096
    ds = (D + 16) * U * amp
    tl = ds + (nrow + 8) * U + 4 * U * np.where(np.isfinite(wl), np.abs(wl), 0)
    w_round = 2.0 ** -11 if mem.dtype == torch.bfloat16 else 2.0 ** -22
    to = (2 * ds[..., None] + w_round + (nrow + 16) * U) * pv + nrow * 2.0 ** -28 * vmax
    if mem.dtype == torch.bfloat16:
        to = to + 2.0 ** -8 * (np.abs(want) + to)
    for b in range(B):
        c = cnt[b]
        assert torch.all(O[b, c:] == 7.0) and torch.all(lse[b, c:] == 7.0), "padding tokens written"
        err = np.abs(f64(O)[b, :c] - want[b, :c])
        assert np.all(err <= to[b, :c]), f"O of query {b}: {err.max():.3e}, bound there {to[b, :c].flat[err.argmax()]:.3e}"
        gl, w_ = f64(lse)[b, :c], wl[b, :c]
        assert np.array_equal(np.isneginf(gl), np.isneginf(w_))
        fin = np.isfinite(w_)
        assert np.all(np.abs(gl[fin] - w_[fin]) <= tl[b, :c][fin]), f"lse of query {b}"
    if decay is not None:
        got = f64(cache.weights)
        rel = (2 * ds.max() + tl.max() + 16 * U)
        for b in range(B):
            ln = int(ref.lens[b])
            old = decay * w0[b, :, :ln] if decay else 0.0
            w = W[b, :, :ln] + old
            tol = rel * W[b, :, :ln] + 4 * U * w + 2.0 ** -100
            assert np.all(np.abs(got[b, :, :ln] - w) <= tol), f"weights of query {b}"
            assert np.array_equal(got[b, :, ln:], w0[b, :, ln:], equal_nan=True)
    assert msa.device_error() == 0
    return O, lse


ATT = [
    # dt, fmt, D, H, G, T, cap, bl, lens, n, k
    ("bf16", "int8", 128, 2, 4, 1, 256, 64, [1, 15, 16, 17, 200, 256], None, 3),
    ("bf16", "int8", 128, 8, 4, 1, 1024, 64, [1000], None, 6),           # split context
    ("bf16", "e4m3", 128, 2, 4, 1, 512, 16, [0, 1, 511, 300], [0, 1, 1, 0], 0),
    ("bf16", "e4m3", 64, 3, 5, 3, 384, 128, [3, 2, 0, 384], [3, 3, 2, 1], 0),  # rows that see nothing
    ("bf16", "int8", 64, 1, 16, 1, 128, 32, [77, 128], None, 2),
    ("bf16", "int8", 64, 1, 16, 2, 128, 32, [2, 100], [1, 2], 2),
    ("bf16", "int8", 128, 1, 1, 13, 64, 16, [13, 64, 40], None, 1),
    ("bf16", "e4m3", 128, 2, 3, 41, 320, 64, [41, 320, 133], [41, 7, 0], 4),
    ("bf16", "int8", 128, 1, 8, 70, 192, 64, [192, 71], [70, 70], 5),
    ("bf16", "int8", 64, 2, 2, 150, 448, 64, [448, 150, 149], None, 2),
    # tensor cores (48 columns of a kv head and more, D = 128): several splits and ring rounds, odd
    # groups, one and two tiles, queries that see nothing, every block length
    ("bf16", "int8", 128, 2, 4, 33, 1024, 16, [1024, 700], [33, 20], 6),
    ("bf16", "e4m3", 128, 1, 16, 20, 2048, 128, [2048], None, 0),
    ("bf16", "int8", 128, 1, 3, 16, 192, 64, [5, 16, 0], [16, 9, 0], 0),
    ("bf16", "e4m3", 128, 1, 5, 29, 1088, 32, [1087, 29, 64], None, 3),
    ("bf16", "int8", 128, 1, 1, 48, 64, 32, [48, 64], [47, 48], 1),
    ("f32", "int8", 64, 2, 2, 1, 256, 64, [1, 31, 33, 256], None, 3),
    ("f32", "e4m3", 128, 1, 5, 9, 128, 16, [9, 128, 4, 0], [9, 3, 9, 0], 2),
    ("f32", "e4m3", 64, 1, 1, 3, 64, 32, [2, 0], [3, 0], 0),
    ("f32", "int8", 128, 2, 4, 1, 2048, 128, [2000], None, 6),
]


@pytest.mark.parametrize("case", ATT, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
def test_attend_matches_fp64(case):
    dt, fmt, D, H, G, T, cap, bl, lens, n, k = case
    mem, content = memory(torch.bfloat16 if dt == "bf16" else torch.float32, H, D)
    B = len(lens)
    cache, ref = filled(mem, B, cap, bl, fmt, lens, seed=D + T)
    rng = np.random.default_rng(1)
    ids = torch.from_numpy(np.stack([rng.choice(6, k, replace=False) for _ in range(B)]).astype(np.int32)).cuda() if k else None
    run_attend(mem, content, cache, ref, ids, T, G, n)


@pytest.mark.parametrize("dt,fmt,T,G,decay", [("bf16", "int8", 1, 4, 0.0), ("bf16", "e4m3", 7, 3, 1.0),
                                              ("f32", "int8", 2, 2, 0.5), ("bf16", "int8", 40, 2, 0.9),
                                              ("bf16", "e4m3", 30, 3, 0.25),
                                              ("bf16", "int8", 100, 4, 1.0), ("bf16", "e4m3", 50, 3, 0.5),
                                              ("bf16", "int8", 3, 4, 0.7), ("f32", "e4m3", 8, 2, 0.0),
                                              ("bf16", "int8", 51, 4, 0.5), ("bf16", "e4m3", 33, 3, 0.0)])
def test_attend_accumulates_weights(dt, fmt, T, G, decay):
    D = 128 if T in (30, 50, 100) else 64
    mem, content = memory(torch.bfloat16 if dt == "bf16" else torch.float32, 2, D)
    lens, n = [200, 1, 77, 150], [T, 1, T // 2, T]
    if T in (51, 100):  # several tiles of rows and of columns
        lens, n = [700, 1, 77, 257], [T, 1, 50, 0]
    cache, ref = filled(mem, 4, 704 if T in (51, 100) else 256, 32, fmt, lens, seed=9, track=True)
    ids = torch.tensor([[0, 3], [1, 2], [5, 4], [3, 0]], dtype=torch.int32, device="cuda")
    for i in range(3):
        run_attend(mem, content, cache, ref, ids, T, G, n, decay=decay, seed=20 + i)


@pytest.mark.parametrize("q_scale,spread", [(12.0, 0.0), (2.0 ** 60, 0.0), (2.0 ** -90, 3.0), (1.0, 8.0)])
def test_attend_magnitudes(q_scale, spread):
    """Sharp softmaxes, queries far outside fp16's range, blocks of very different scales."""
    mem, content = memory(torch.bfloat16, 1, 128)
    cache, ref = filled(mem, 2, 512, 16, "int8", [512, 333], seed=4, spread=spread)
    ids = torch.tensor([[0, 3], [1, 5]], dtype=torch.int32, device="cuda")
    run_attend(mem, content, cache, ref, ids, 1, 4, None, q_scale=q_scale)
    run_attend(mem, content, cache, ref, None, 6, 2, None, q_scale=q_scale)
    run_attend(mem, content, cache, ref, ids, 40, 2, None, q_scale=q_scale)


@pytest.mark.parametrize("T", [2, 20, 80])  # scores kept, recomputed on mma.sync, on tcgen05
@pytest.mark.parametrize("q_scale,spread", [(4.0, 0.0), (2.0 ** -90, 3.0), (1.0, 8.0)])
def test_weights_magnitudes(T, q_scale, spread):
    mem, content = memory(torch.bfloat16, 1, 128)
    cache, ref = filled(mem, 2, 512, 16, "int8", [512, 333], seed=4, spread=spread, track=True)
    ids = torch.tensor([[0, 3], [1, 5]], dtype=torch.int32, device="cuda")
    run_attend(mem, content, cache, ref, ids, T, 2, None, q_scale=q_scale, decay=0.0)


@pytest.mark.parametrize("T,G", [(4, 4), (20, 2), (60, 2)])  # the three paths again
def test_weights_where_tokens_see_nothing(T, G):
    mem, content = memory(torch.bfloat16, 1, 128)
    cache, ref = filled(mem, 3, 320, 32, "e4m3", [2, 300, 0], seed=8, track=True)
    for i in range(2):  # more new tokens than rows: the first ones see no row, and there is no memory
        run_attend(mem, content, cache, ref, None, T, G, None, decay=0.5, seed=30 + i)


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("T", [1, 40])
def test_attend_repeated_and_bad_ids(dt, T):
    """A document named twice counts twice; ids out of range bring no rows and are flagged."""
    from top_document_sparse_b200 import msa
    mem, content = memory(dt, 2, 128)
    cache, ref = filled(mem, 2, 128, 32, "int8", [128, 70], seed=8)
    twice = torch.tensor([[3, 3, 0], [1, 1, 1]], dtype=torch.int32, device="cuda")
    run_attend(mem, content, cache, ref, twice, T, 2, None)
    good = torch.tensor([[2], [5]], dtype=torch.int32, device="cuda")
    bad = torch.tensor([[-1, 2, 6], [5, 2 ** 31 - 1, -7]], dtype=torch.int32, device="cuda")
    want, _ = run_attend(mem, content, cache, ref, good, T, 2, None, seed=12)
    Q = (torch.randn(*want.shape, generator=torch.Generator(device="cuda").manual_seed(12), device="cuda")).to(dt)
    O = torch.empty_like(Q)
    cache.attend(content, bad, Q, O, msa.workspace(cache.attend_workspace_size(T, 3, 4)))
    assert msa.device_error() == BAD_DOC_ID
    # each is within the output's rounding, a weight's (2^-11 in bf16, 2^-22 in fp32) and the sums'
    # (half a weight's; 4,300 rows' in fp32) of the exact value, none larger than the largest V
    top = max(float(content[:, 1].abs().max()), float(cache.read(None, 128)[1].abs().max()))
    step = 2.0 ** -8 + 1.5 * 2.0 ** -11 if dt == torch.bfloat16 else 2.0 ** -24 + 1.5 * 2.0 ** -22 + 4300 * U
    assert float((O.double() - want.double()).abs().max()) <= 2 * step * top


@pytest.mark.parametrize("T", [1, 40])
@pytest.mark.parametrize("k_scale,v_scale", [(2.0 ** -30, 2.0 ** 40), (8.0, 2.0 ** -40), (0.0, 0.0)])
def test_attend_memory_magnitudes(T, k_scale, v_scale):
    """Memory rows far larger and far smaller than the cached ones, and all-zero ones."""
    mem, content = memory(torch.bfloat16, 1, 128)
    content[:, 0] *= k_scale
    content[:, 1] *= v_scale
    cache, ref = filled(mem, 2, 256, 64, "int8", [256, 50], seed=6)
    ids = torch.tensor([[0, 3, 5], [1, 5, 2]], dtype=torch.int32, device="cuda")
    run_attend(mem, content, cache, ref, ids, T, 2, None)


def test_attend_over_fetched_rows_equals_resident_rows():
    """The host tier's slot cache holds the same rows elsewhere: the same bits."""
    from top_document_sparse_b200 import msa
    mem, content = memory(torch.bfloat16, 2, 128)
    host = mem.new_content(device="cpu", pin_memory=True)
    host.copy_(content)
    fetcher = msa.Fetcher(mem, host, n_slots=9, max_batch=2, max_k=3)
    ids = torch.tensor([[0, 3, 5], [1, 5, 2]], dtype=torch.int32, device="cuda")
    for T, G in ((1, 4), (17, 3)):
        cache, ref = filled(mem, 2, 256, 64, "e4m3", [256, 50], seed=6)
        O, lse = run_attend(mem, content, cache, ref, ids, T, G, None)
        fetcher.fetch(ids)
        Q = torch.randn(2, T, 2 * G, 128, generator=torch.Generator(device="cuda").manual_seed(11),
                        device="cuda").bfloat16()
        O2, lse2 = torch.empty_like(O), torch.empty_like(lse)
        cache.attend(fetcher, ids, Q, O2, msa.workspace(cache.attend_workspace_size(T, 3, 2 * G)), lse=lse2)
        assert torch.equal(O, O2) and torch.equal(lse, lse2)
    other, _ = memory(torch.bfloat16, 2, 128)
    with pytest.raises(msa.MsaError):
        c = msa.Cache8(other, 2, 64)
        c.attend(fetcher, ids, Q, O2, msa.workspace(c.attend_workspace_size(T, 3, 2 * G)))


def test_attend_and_append_past_32_bit_offsets():
    """A cache of 2^31 elements and more: the last query's rows lie past every 32-bit offset.  Checked
    on one head against torch in fp64."""
    from top_document_sparse_b200 import msa
    B, H, cap, D = 2, 8, (1 << 20) + 128, 128
    mem, content = memory(torch.bfloat16, H, D)
    cache = msa.Cache8(mem, B, cap, 128, "int8", track_weights=True)
    g = torch.Generator(device="cuda").manual_seed(3)
    for t in (cache.k, cache.v):
        for b in range(B):
            t[b] = torch.randint(-100, 101, (H, cap, D), generator=g, device="cuda", dtype=torch.int8)
    cache.k_scale.fill_(2.0 ** -6)
    cache.v_scale.fill_(2.0 ** -6)
    start = torch.tensor([5, cap - 3], dtype=torch.int32, device="cuda")
    kv = torch.randn(2, B, 2, H, D, generator=g, device="cuda").bfloat16()
    cache.append(kv[0], kv[1], start=start)
    Kr, _ = cache.read(start, 2)
    assert torch.all((Kr.float() - kv[0].float()).abs() <= 2.0 ** -6)  # half a step of the largest scale
    # (8 x 12 columns run on tcgen05, which adds 16 rows an accumulation into at most n / 128 partial sums)
    for T, G, sums in ((1, 1, 0), (2, 24 // 2, 0), (8, 12, (cap - 1) / 128)):
        Q = torch.randn(B, T, H * G, D, generator=g, device="cuda").bfloat16()
        O, lse = torch.empty_like(Q), torch.empty(B, T, H * G, device="cuda")
        cache.attend(None, None, Q, O, msa.workspace(cache.attend_workspace_size(T, 0, H * G)), lse=lse,
                     weight_decay=0.0)
        b, h, n = 1, H - 1, cap - 1
        sk = cache.k_scale[b, h].double().repeat_interleave(128)[:n, None]
        sv = cache.v_scale[b, h].double().repeat_interleave(128)[:n, None]
        V = cache.v[b, h, :n].double() * sv
        z = (cache.k[b, h, :n].double() * sk) @ Q[b, -1, h * G].double() / D ** 0.5
        p = torch.softmax(z, 0)
        want, size = p @ V, p @ V.abs()
        # see the bounds above; the row sum's error grows with the square root of the rows here, but
        # is bounded by (rows / 512) u: a split's lane adds that many terms
        tol = (2.0 ** -11 + 2.0 ** -12 + (n / 512 + sums) * U) * size + n * 2.0 ** -28 * 2
        err = (O[b, -1, h * G].double() - want).abs()
        assert torch.all(err <= tol + 2.0 ** -8 * (want.abs() + tol))
        assert abs(float(lse[b, -1, h * G]) - float(torch.logsumexp(z, 0))) <= 1e-4
        assert abs(float(cache.weights[b, h, :n].sum()) - T * G) <= 1e-3 * T * G
    assert msa.device_error() == 0


def test_attend_calls_on_two_streams_and_two_graphs_of_one_workspace():
    from top_document_sparse_b200 import msa
    mem, content = memory(torch.bfloat16, 2, 128)
    ids = torch.tensor([[0, 3], [1, 5]], dtype=torch.int32, device="cuda")
    sets = []
    for seed, T in ((1, 1), (2, 3), (3, 40)):
        cache, _ = filled(mem, 2, 1024, 64, "int8", [1024, 777], seed=seed, track=True)
        Q = torch.randn(2, T, 6, 128, device="cuda").bfloat16()
        need = cache.attend_workspace_size(T, 2, 6)
        sets.append((cache, Q, torch.empty_like(Q), need))
    want = []
    for cache, Q, O, need in sets:
        cache.attend(content, ids, Q, O, msa.workspace(need), weight_decay=0.0)
        want.append((O.clone(), cache.weights.clone()))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    spaces = [msa.workspace(need) for *_, need in sets]
    torch.cuda.synchronize()
    for _ in range(5):  # at the same time, a workspace each
        for (cache, Q, O, _), st, ws in zip(sets, streams, spaces):
            cache.attend(content, ids, Q, O, ws, weight_decay=0.0, stream=st)
    torch.cuda.synchronize()
    for (cache, _, O, _), (o, w) in zip(sets, want):
        # (as bits: the weights behind the last row hold the poison, NaN)
        assert torch.equal(O, o) and torch.equal(cache.weights.view(torch.int32), w.view(torch.int32))
    shared = msa.workspace(max(need for *_, need in sets))
    graphs = []
    for cache, Q, O, _ in sets:
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            cache.attend(content, ids, Q, O, shared, weight_decay=0.0)
        graphs.append(gr)
    for order in ((0, 1, 2), (2, 0, 1), (1, 2, 0)):
        for i in order:
            sets[i][2].zero_()
            graphs[i].replay()
    torch.cuda.synchronize()
    for (cache, _, O, _), (o, w) in zip(sets, want):
        # (as bits: the weights behind the last row hold the poison, NaN)
        assert torch.equal(O, o) and torch.equal(cache.weights.view(torch.int32), w.view(torch.int32))
    assert msa.device_error() == 0


def test_attend_flags_bad_counts():
    from top_document_sparse_b200 import msa
    mem, content = memory(torch.bfloat16, 2, 64)
    cache, ref = filled(mem, 3, 64, 16, "int8", [10, 20, 30], seed=1)
    cache.cache_len[1] = 65
    Q = torch.randn(3, 2, 4, 64, device="cuda").bfloat16()
    O = torch.full_like(Q, 7.0)
    ws = msa.workspace(cache.attend_workspace_size(2, 1, 4))
    ids = torch.tensor([[0], [1], [6]], dtype=torch.int32, device="cuda")  # 6 is no document
    cache.attend(content, ids, Q, O, ws, n_tokens=torch.tensor([3, 1, 2], dtype=torch.int32, device="cuda"))
    assert msa.device_error() == msa.DEVERR_BAD_LENGTH | msa.DEVERR_BAD_DOC_ID
    assert torch.all(O[:2] == 7.0) and torch.isfinite(O).all() and not torch.any(O[2] == 7.0)


# ---------------------------------------------------------------- eviction
EVICT = [
    # fmt, D, H, bl, cap, lens, budget, recent
    ("int8", 128, 2, 64, 1024, [1024, 1000, 300, 0, 513], 512, 100),
    ("e4m3", 64, 3, 16, 2048, [2047, 17, 2048, 1031], 16, 0),
    ("int8", 64, 1, 32, 256, [255, 256, 129, 128, 97], 128, 128),
    ("e4m3", 128, 1, 128, 512, [512, 500, 129, 256], 129, 1),
    ("int8", 64, 1, 16, 16 * 10304, [16 * 10304 - 3], 16 * 9000 + 5, 100),  # keys in the workspace
]


@pytest.mark.parametrize("case", EVICT, ids=lambda c: "-".join(str(x).replace(" ", "") for x in c))
@pytest.mark.parametrize("in_place", [True, False])
def test_evict_matches_the_rule(case, in_place):
    from top_document_sparse_b200 import msa
    fmt, D, H, bl, cap, lens, budget, recent = case
    mem, _ = memory(torch.bfloat16, H, D)
    B = len(lens)
    cache, ref = filled(mem, B, cap, bl, fmt, lens, seed=8, track=True)
    g = torch.Generator(device="cuda").manual_seed(2)
    w = torch.rand(B, H, cap, generator=g, device="cuda") ** 8
    w[:, :, :cap // 2] = (w[:, :, :cap // 2] * 4).round()  # many ties
    w[0, 0, bl + 1] = float("nan")
    w[-1] = 0.0
    cache.weights.copy_(w)
    ref.load(cache)
    ws = msa.workspace(cache.evict_workspace_size())
    ws.fill_(0xFF)
    old_len = ref.lens.copy()
    if in_place:
        cache.evict(budget, recent, ws)
        got = cache
    else:
        got = msa.Cache8(mem, B, -(-min(budget, cap) // bl) * bl, bl, fmt, track_weights=True)
        poison(got)
        before = cache.k.view(torch.int8).clone(), cache.weights.clone()
        cache.evict(budget, recent, ws, out=got)
        assert torch.equal(before[0], cache.k.view(torch.int8))
        assert torch.equal(before[1].view(torch.int32), cache.weights.view(torch.int32))
    ref.evict(budget, recent)
    equal_cache(got, ref)
    for b in range(B):
        n, end = int(ref.lens[b]), min(int(old_len[b]), got.capacity)
        assert np.array_equal(f64(got.weights[b, :, :n]), ref.w[b, :, :n], equal_nan=True)
        assert torch.all(got.weights[b, :, n:end] == 0)
        if not in_place:  # bytes behind the last row stay
            assert torch.all(got.k.view(torch.int8)[b, :, n:] == 0x7F)
    assert msa.device_error() == 0


# ---------------------------------------------------------------- as they are used
def test_decode_loop_of_all_operators():
    """Rotate, append, attend with weights and evict when the cache runs full, step after step, then
    compare the last attention with the formula on what the cache holds; the same loop's step
    captured as a graph and replayed on another stream gives the same bits."""
    from top_document_sparse_b200 import msa
    B, H, G, D, cap, bl = 3, 2, 4, 128, 96, 16
    mem, content = memory(torch.bfloat16, H, D)
    ids = torch.tensor([[0, 3], [1, 5], [2, 4]], dtype=torch.int32, device="cuda")
    steps = 70
    g = torch.Generator(device="cuda").manual_seed(1)
    qkv = torch.randn(steps, B, 1, (H * G + 2 * H) * D, generator=g, device="cuda").bfloat16()
    rope = msa.Rope(D, scaling="linear", factor=2.0)

    def loop(graphed):
        cache = msa.Cache8(mem, B, cap, bl, "int8", track_weights=True)
        ws = msa.workspace(max(cache.attend_workspace_size(1, 2, H * G), cache.evict_workspace_size()))
        pos = torch.zeros(B, 1, dtype=torch.int64, device="cuda")
        x = torch.zeros_like(qkv[0])
        q, kv = x[..., :H * G * D].view(B, 1, H * G, D), x[..., H * G * D:]
        k, v = kv[..., :H * D].view(B, 1, H, D), kv[..., H * D:].view(B, 1, H, D)
        qo, ko = torch.empty(B, 1, H * G, D, device="cuda").bfloat16(), torch.empty(B, 1, H, D, device="cuda").bfloat16()
        O, lse = torch.empty_like(qo), torch.empty(B, 1, H * G, device="cuda")

        def step():
            rope.rotate(q, k, pos, q_out=qo, k_out=ko)
            cache.evict(cap - bl, 24, ws)
            cache.append(ko, v)
            cache.attend(content, ids, qo, O, ws, lse=lse, weight_decay=1.0)
            pos.add_(1)

        run = step
        if graphed:
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=s):
                step()
            run = gr.replay
        for i in range(steps):
            x.copy_(qkv[i])
            run()
        torch.cuda.synchronize()
        return cache, qo.clone(), O.clone(), lse.clone()

    cache, qo, O, lse = loop(False)
    assert int(cache.cache_len.max()) <= cap
    ref = R.RefCache(B, H, cap, D, bl, "int8").load(cache)
    want, wl, _, pv, amp = R.attend(ref, R.content_rows(mem, content, ids), f64(qo), [1] * B)
    ds = (D + 16) * U * amp
    tol = (2 * ds[..., None] + 2.0 ** -11 + 5000 * U) * pv
    assert np.all(np.abs(f64(O) - want) <= tol + 2.0 ** -8 * (np.abs(want) + tol))
    assert np.all(np.abs(f64(lse) - wl) <= ds + 5000 * U + 4 * U * np.abs(wl))
    # every query token has handed out one unit of weight a head; memory rows took part of it
    assert torch.all(cache.weights.sum(-1) <= steps * G)
    cache2, _, O2, lse2 = loop(True)
    assert torch.equal(O, O2) and torch.equal(lse, lse2)
    assert torch.equal(cache.k, cache2.k) and torch.equal(cache.weights, cache2.weights)
    assert msa.device_error() == 0


def test_refusals():
    from top_document_sparse_b200 import msa
    mem, content = memory(torch.bfloat16, 2, 64)
    for kw in (dict(capacity=100), dict(capacity=0), dict(block_len=48), dict(fmt="int4"), dict(batch=0)):
        with pytest.raises(ValueError):
            msa.Cache8(mem, **{**dict(batch=1, capacity=64), **kw})
    cache = msa.Cache8(mem, 2, 64, 16)
    tracked = msa.Cache8(mem, 2, 64, 16, track_weights=True)
    K = torch.randn(2, 3, 2, 64, device="cuda").bfloat16()
    Q = torch.randn(2, 3, 4, 64, device="cuda").bfloat16()
    O, ids = torch.empty_like(Q), torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    ws = msa.workspace(cache.attend_workspace_size(3, 1, 4))
    none = torch.empty(0, dtype=torch.uint8, device="cuda")
    n = torch.ones(2, dtype=torch.int32, device="cuda")
    ev = msa.workspace(tracked.evict_workspace_size())
    before = msa.launch_count()
    for bad in (
            lambda: cache.append(K.float(), K), lambda: cache.append(K[:, :, :1], K[:, :, :1]),
            lambda: cache.append(K.transpose(2, 3), K), lambda: cache.append(K.cpu(), K.cpu()),
            lambda: cache.append(K, K, n_tokens=n.long()), lambda: cache.append(K, K, start=n[:1]),
            lambda: cache.append(K[:, :0], K[:, :0]), lambda: cache.read(None, 0),
            lambda: cache.attend(content, ids, Q[:, :, :3].contiguous(), O[:, :, :3].contiguous(), ws),
            lambda: cache.attend(content, ids, Q, O.float(), ws),
            lambda: cache.attend(content[1:], ids, Q, O, ws),
            lambda: cache.attend(content, ids.long(), Q, O, ws),
            lambda: cache.attend(content, ids, Q, O, ws, weight_decay=0.0),
            lambda: tracked.attend(content, ids, Q, O, ws, weight_decay=-1.0),
            lambda: tracked.attend(content, ids, Q, O, ws, weight_decay=float("nan")),
            lambda: tracked.attend(content, ids, Q, O, none),
            lambda: cache.evict(32, 0, ev), lambda: tracked.evict(15, 0, ev),
            lambda: tracked.evict(32, 33, ev), lambda: tracked.evict(32, -1, ev),
            lambda: tracked.evict(32, 0, none), lambda: tracked.evict(32, 0, ev, out=cache),
            lambda: tracked.evict(64, 0, ev, out=msa.Cache8(mem, 2, 32, 16, track_weights=True)),
            lambda: tracked.evict(32, 0, ev, out=msa.Cache8(mem, 2, 64, 32, track_weights=True))):
        with pytest.raises((ValueError, TypeError, msa.MsaError)):
            bad()
    assert msa.launch_count() == before, "a refused call enqueued something"


def test_evict_flags_bad_lengths():
    from top_document_sparse_b200 import msa
    mem, _ = memory(torch.bfloat16, 1, 64)
    cache, _ = filled(mem, 3, 128, 16, "int8", [128, 100, 10], seed=1, track=True)
    cache.weights.zero_()
    cache.cache_len.copy_(torch.tensor([129, -1, 10]))
    cache.evict(64, 0, msa.workspace(cache.evict_workspace_size()))
    assert msa.device_error() == msa.DEVERR_BAD_LENGTH
    assert cache.cache_len.tolist() == [64, 0, 10]


def test_append_of_many_shapes_at_once_equals_block_by_block():
    """Units that share a CTA (small blocks), one of them with non-finite values, against the same
    rows appended to caches of one head."""
    from top_document_sparse_b200 import msa
    for D, bl, H in ((64, 16, 3), (128, 16, 5), (64, 32, 1)):
        mem, _ = memory(torch.bfloat16, H, D)
        one, _ = memory(torch.bfloat16, 1, D)
        kv = torch.randn(2, 2, 50, H, D, device="cuda").bfloat16()
        kv[0, 1, 20, H - 1, 3] = float("inf")
        kv[1, 0, 33, 0, 5] = float("nan")
        cache = msa.Cache8(mem, 2, 64, bl, "int8")
        cache.append(kv[0], kv[1])
        for h in range(H):
            single = msa.Cache8(one, 2, 64, bl, "int8")
            single.append(kv[0][:, :, h:h + 1].contiguous(), kv[1][:, :, h:h + 1].contiguous())
            assert torch.equal(cache.k[:, h:h + 1], single.k) and torch.equal(cache.v[:, h:h + 1], single.v)
            assert torch.equal(cache.k_scale[:, h:h + 1], single.k_scale)
            assert torch.equal(cache.v_scale[:, h:h + 1], single.v_scale)
