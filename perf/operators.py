"""What is measured of the 8-bit local cache and the rotary positions that feed it.

Four operators: rotary positions (forward and backward), appending tokens to the 8-bit cache and
reading rows back, attention over the retrieved memory rows and the 8-bit cache (with the attention
weight that each cached row received), and eviction by that weight.  Every case is one call as a
serving or training loop makes it.  Lengths are ragged by a fixed rule, values come from the seed.
"""
from __future__ import annotations

import math

import torch

own = False  # set by the caller: False, elementary torch operations; True, the library's calls

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ES = {"bf16": 2, "f32": 4}
LOG2E = 1.4426950408889634


# ---------------------------------------------------------------------------- cases
def listed():
    return [
        # one decode step's Q and K of 64 queries, as slices of one projection's output
        dict(name="rope decode", op="rope", dtype="bf16", batch=64, tokens=1, q_heads=32, kv_heads=8,
             head_dim=128, rotary_dim=128, layout="half", scaling="none", factor=1.0, original=4096,
             reach=4096, backward=False),
        # prefill of 64 queries of 256 tokens far into a stretched context
        dict(name="rope prefill yarn", op="rope", dtype="bf16", batch=64, tokens=256, q_heads=32,
             kv_heads=8, head_dim=128, rotary_dim=128, layout="half", scaling="yarn", factor=8.0,
             original=8192, reach=1 << 20, backward=False),
        # training: gradients of Q and K where half of each head is rotated, in neighbouring pairs
        dict(name="rope backward", op="rope", dtype="f32", batch=4, tokens=1021, q_heads=8, kv_heads=2,
             head_dim=64, rotary_dim=32, layout="interleaved", scaling="ntk", factor=4.0,
             original=4096, reach=32768, backward=True),
        # one decode step's rows of 64 queries at ragged lengths, and the touched blocks read back
        dict(name="append decode", op="append", dtype="bf16", fmt="int8", batch=64, tokens=1, kv_heads=8,
             head_dim=128, capacity=4096, block=64, ragged=True),
        # a prefilled query batch goes into the cache at once
        dict(name="append prefill", op="append", dtype="bf16", fmt="int8", batch=64, tokens=1000,
             kv_heads=8, head_dim=128, capacity=2048, block=64, ragged=True),
        # the same in 8-bit floating point from fp32 rows, small heads
        dict(name="append e4m3 f32", op="append", dtype="f32", fmt="e4m3", batch=3, tokens=77, kv_heads=2,
             head_dim=64, capacity=512, block=16, ragged=False),
        # the decode step of one query: latency counts
        dict(name="attend one query", op="attend", dtype="bf16", fmt="int8", batch=1, tokens=1, q_heads=32,
             kv_heads=8, head_dim=128, capacity=256, block=64, k=16, doc_len=512, n_docs=32,
             full=True, weights=False),
        # the decode step of 64 queries over long ragged caches, bandwidth counts
        dict(name="attend decode", op="attend", dtype="bf16", fmt="int8", batch=64, tokens=1, q_heads=32,
             kv_heads=8, head_dim=128, capacity=8192, block=64, k=16, doc_len=512, n_docs=256,
             full=False, weights=False),
        # four drafted tokens checked at once on two long queries, with the rows' attention weight
        dict(name="attend draft weights", op="attend", dtype="bf16", fmt="e4m3", batch=2, tokens=4, q_heads=32,
             kv_heads=8, head_dim=128, capacity=32768, block=32, k=8, doc_len=500, n_docs=64,
             full=True, weights=True),
        # a prompt's next 512 tokens over a cache of 8K rows: arithmetic counts
        dict(name="attend chunk", op="attend", dtype="bf16", fmt="int8", batch=1, tokens=512, q_heads=32,
             kv_heads=8, head_dim=128, capacity=8704, block=64, k=16, doc_len=512, n_docs=64,
             full=True, weights=False),
        # a decode batch's caches brought back to half, into the smaller cache that serves on
        dict(name="evict batch", op="evict", fmt="int8", batch=16, kv_heads=8, head_dim=128,
             capacity=8192, block=64, budget=4096, recent=256),
        # one short query
        dict(name="evict one", op="evict", fmt="e4m3", batch=1, kv_heads=2, head_dim=64,
             capacity=1024, block=16, budget=700, recent=50),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "evict"])
    while True:
        D = rng.choice([64, 128, 128])
        kv = rng.choice([1, 2, 4, 8, 8])
        block = rng.choice([16, 32, 64, 64, 128])
        fmt = rng.choice(["int8", "int8", "e4m3"])
        if op == "rope":
            c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), batch=_log(rng, 1, 64),
                     tokens=_log(rng, 1, 4096), q_heads=kv * rng.choice([1, 2, 4, 8]), kv_heads=kv,
                     head_dim=D, rotary_dim=rng.choice([D, D, D // 2, D // 4]),
                     layout=rng.choice(["half", "interleaved"]),
                     scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                     factor=float(rng.choice([2, 4, 8, 32])), original=rng.choice([2048, 4096, 8192]),
                     reach=_log(rng, 4096, 1 << 20), backward=rng.random() < 0.4)
        elif op == "append":
            cap = block * _log(rng, 1, 8192 // block)
            c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f32"]), fmt=fmt, batch=_log(rng, 1, 64),
                     tokens=_log(rng, 1, cap), kv_heads=kv, head_dim=D, capacity=cap, block=block,
                     ragged=rng.random() < 0.7)
        elif op == "attend":
            T = 1 if rng.random() < 0.5 else _log(rng, 2, 512)
            cap = block * _log(rng, max(1, -(-T // block)), 32768 // block)
            dt = rng.choice(["bf16", "bf16", "bf16", "f32"])
            c = dict(op=op, dtype=dt, fmt=fmt, batch=_log(rng, 1, 64), tokens=T,
                     q_heads=kv * rng.choice([1, 2, 4, 8] if dt == "bf16" else [1, 2]), kv_heads=kv,
                     head_dim=D, capacity=cap, block=block, k=rng.choice([0, 1, 4, 8, 16]),
                     doc_len=rng.choice([100, 500, 512]), n_docs=rng.choice([16, 64, 128]),
                     full=rng.random() < 0.3, weights=rng.random() < 0.3)
        else:
            cap = block * _log(rng, 2, 32768 // block)
            budget = max(block, int(cap * rng.uniform(0.2, 0.9)))
            c = dict(op=op, fmt=fmt, batch=_log(rng, 1, 32), kv_heads=kv, head_dim=D, capacity=cap,
                     block=block, budget=budget, recent=int(budget * rng.uniform(0, 0.5)))
        w = work(c)
        if w["bytes"] < 3e8 and w["flops"] < (7e10 if c.get("dtype") != "f32" else 4e9) \
                and _plain_bytes(c) < 8e9:
            return c


def _plain_bytes(c):
    """What the plain form holds at once: draw() leaves out what no card's memory takes three times."""
    if c["op"] == "attend":
        rows = c["capacity"] + c["k"] * -(-c["doc_len"] // 64)
        return 4.0 * c["batch"] * rows * (3 * c["q_heads"] * c["tokens"] + 5 * c["kv_heads"] * c["head_dim"])
    if c["op"] == "rope":
        return 0.0
    return 16.0 * c["batch"] * c["capacity"] * c["kv_heads"] * c["head_dim"]


def _spread(n, lo, hi, phase):
    """n whole numbers spread over lo..hi, the same for every seed."""
    return [lo + int((hi - lo) * ((0.6180339887 * i + phase) % 1.0)) for i in range(n)]


def _lengths(c):
    """Rows in the cache: before an append, after it for the attention, before an eviction."""
    B, cap = c["batch"], c["capacity"]
    if c["op"] == "append":
        return _spread(B, 0, cap - c["tokens"], 0.37) if c["ragged"] else [cap - c["tokens"]] * B
    if c["op"] == "attend":
        return [cap] * B if c["full"] else _spread(B, max(c["tokens"], cap // 4), cap, 0.53)
    return _spread(B, (cap + c["budget"]) // 2, cap, 0.71)


def _counts(c):
    """New tokens of each query (the rest of its `tokens` places are padding)."""
    B, T = c["batch"], c["tokens"]
    ragged = c["ragged"] if c["op"] == "append" else not c["full"]
    return _spread(B, (T + 1) // 2, T, 0.91) if ragged and T > 1 else [T] * B


def work(c):
    """Bytes read and written once, and the operations, of one pass."""
    op, B, H, D = c["op"], c["batch"], c["kv_heads"], c["head_dim"]
    if op == "rope":
        n = B * c["tokens"] * (c["q_heads"] + H)
        return dict(bytes=2 * n * D * ES[c["dtype"]] + 8 * B * c["tokens"], flops=3 * n * c["rotary_dim"])
    bl = c["block"]
    if op == "append":
        rows, back = 0, 0
        for s, n in zip(_lengths(c), _counts(c)):
            rows += n
            back += s % bl + n  # rows of the touched blocks that are read back
        e = ES[c["dtype"]]
        return dict(bytes=2 * H * D * (rows * (e + 1) + back * (1 + e)), flops=4 * rows * H * D)
    if op == "attend":
        T, Hq, e = c["tokens"], c["q_heads"], ES[c["dtype"]]
        mem = c["k"] * -(-c["doc_len"] // 64)
        by = fl = 0
        for ln, n in zip(_lengths(c), _counts(c)):
            by += ln * H * (2 * D + 8 / bl + (4 if c["weights"] else 0)) + mem * 2 * H * D * e
            by += 2 * n * Hq * D * e + n * Hq * 4
            fl += 4 * D * Hq * (n * mem + sum(ln - n + t + 1 for t in range(n)))
        return dict(bytes=by, flops=fl)
    by = 0
    for ln in _lengths(c):
        new = (c["budget"] - ln % bl) // bl * bl + ln % bl if ln > c["budget"] else ln
        by += H * (4 * ln + 2 * new * (2 * D + 4 + 8 / bl))
    return dict(bytes=by, flops=B * H * c["capacity"])


# ---------------------------------------------------------------------------- 8-bit values, plain
QMAX = {"int8": 127.0, "e4m3": 448.0}


def _block_scale(amax, fmt):
    """The smallest power of two s with amax <= qmax * s; 0 for a block of zeros."""
    m, e = torch.frexp(amax)
    mq, eq = math.frexp(QMAX[fmt])
    e = (e - eq + (m > mq).to(e.dtype)).clamp(min=-126)
    return torch.where(amax > 0, torch.ldexp(torch.ones_like(amax), e), torch.zeros_like(amax))


def _to8(x, s, fmt):
    """x / s rounded to the format (s broadcasts; an all-zero block has s = 0)."""
    y = x / torch.where(s > 0, s, torch.ones_like(s))
    return torch.round(y).to(torch.int8) if fmt == "int8" else y.to(torch.float8_e4m3fn)


def _fill8(B, H, cap, D, bl, fmt, gen):
    """A cache's content: normal rows with a magnitude of its own for each head, quantised."""
    q = torch.empty(B, H, cap, D, dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn, device="cuda")
    scale = torch.empty(B, H, cap // bl, device="cuda")
    mag = torch.exp(0.5 * torch.randn(B, H, 1, 1, 1, generator=gen, device="cuda"))
    step = max(1, (1 << 27) // (H * cap * D))
    for b in range(0, B, step):
        x = torch.randn(min(step, B - b), H, cap // bl, bl, D, generator=gen, device="cuda")
        x = (x * mag[b:b + step]).bfloat16().float()
        s = _block_scale(x.abs().amax((3, 4)), fmt)
        q[b:b + step] = _to8(x, s[..., None, None], fmt).reshape(-1, H, cap, D)
        scale[b:b + step] = s
    return q, scale


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _memory(c, n_docs, doc_len):
    """The library's memory handle (one is kept by every program that serves)."""
    from top_document_sparse_b200 import msa
    return msa.Memory([doc_len * i for i in range(n_docs + 1)], 64, c["kv_heads"], c["head_dim"], 8, 128,
                      DT[c.get("dtype", "bf16")], 1e6, 64)


def _cache(c, mem, capacity, k, ks, v, vs, lens, weights=None):
    from top_document_sparse_b200 import msa
    cache = msa.Cache8(mem, c["batch"], capacity, c["block"], c["fmt"], track_weights=weights is not None)
    if k is not None:
        for a, b in ((cache.k, k), (cache.v, v), (cache.k_scale, ks), (cache.v_scale, vs)):
            a.copy_(b)
        if weights is not None:
            cache.weights.copy_(weights)
    if lens is not None:
        cache.cache_len.copy_(lens)
    return cache


# ---------------------------------------------------------------------------- inputs
def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(c=c)
    B, H, D = c["batch"], c["kv_heads"], c["head_dim"]
    if c["op"] == "rope":
        T, Hq = c["tokens"], c["q_heads"]
        qkv = torch.randn(B, T, (Hq + 2 * H) * D, generator=gen, device="cuda").to(DT[c["dtype"]])
        st["q"] = qkv[..., :Hq * D].view(B, T, Hq, D)
        st["k"] = qkv[..., Hq * D:(Hq + H) * D].view(B, T, H, D)
        first = torch.randint(0, max(1, c["reach"] - T), (B, 1), generator=gen, device="cuda")
        st["pos"] = first + torch.arange(T, device="cuda")
        if own:
            from top_document_sparse_b200 import msa
            st["rope"] = msa.Rope(D, c["rotary_dim"], 1e6, c["layout"], c["scaling"], c["factor"], c["original"])
        return st
    cap, bl, fmt = c["capacity"], c["block"], c["fmt"]
    lens = _lengths(c)
    st["lens"] = _i32(lens)
    k, ks = _fill8(B, H, cap, D, bl, fmt, gen)
    v, vs = _fill8(B, H, cap, D, bl, fmt, gen)
    if c["op"] == "append":
        T = c["tokens"]
        dt = DT[c["dtype"]]
        # the new rows as the projection leaves them: K and V of a token side by side
        kv = torch.randn(B, T, 2 * H * D, generator=gen, device="cuda").mul_(1.3).to(dt)
        st["K"], st["V"] = kv[..., :H * D].view(B, T, H, D), kv[..., H * D:].view(B, T, H, D)
        st["n"] = _i32(_counts(c))
        st["begin"] = _i32([s // bl * bl for s in lens])
        st["rows"] = min(cap, ((T + bl - 2) // bl + 1) * bl)
        if own:
            st["cache"] = _cache(c, _memory(c, 2, 64), cap, k, ks, v, vs, st["lens"])
        else:
            st.update(k=k, ks=ks, v=v, vs=vs)
        return st
    if c["op"] == "attend":
        T, Hq, kk, dt = c["tokens"], c["q_heads"], c["k"], DT[c["dtype"]]
        cpd = -(-c["doc_len"] // 64)
        st["Q"] = torch.randn(B, T, Hq, D, generator=gen, device="cuda").to(dt)
        st["n"] = _i32(_counts(c))
        st["content"] = (torch.randn(c["n_docs"] * cpd, 2, H, D, generator=gen, device="cuda") * 0.4).to(dt)
        st["ids"] = torch.rand(B, c["n_docs"], generator=gen, device="cuda").argsort(1)[:, :kk].int().contiguous()
        st["O"] = torch.zeros(B, T, Hq, D, dtype=dt, device="cuda")
        st["lse"] = torch.zeros(B, T, Hq, device="cuda")
        st["w"] = torch.zeros(B, H, cap, device="cuda") if c["weights"] else None
        if own:
            from top_document_sparse_b200 import msa
            mem = _memory(c, c["n_docs"], c["doc_len"])
            st["cache"] = _cache(c, mem, cap, k, ks, v, vs, st["lens"], st["w"])
            st["ws"] = msa.workspace(st["cache"].attend_workspace_size(T, kk, Hq))
        else:
            st.update(k=k, ks=ks, v=v, vs=vs)
        return st
    # attention weight as it accumulates: a few heavy rows, a long tail
    w = torch.rand(B, H, cap, generator=gen, device="cuda").pow_(12).mul_(8)
    new_cap = -(-c["budget"] // bl) * bl
    if own:
        from top_document_sparse_b200 import msa
        mem = _memory(c, 2, 64)
        st["cache"] = _cache(c, mem, cap, k, ks, v, vs, st["lens"], w)
        st["into"] = _cache(c, mem, cap, None, None, None, None, None, w)
        for t in (st["into"].k.view(torch.int8), st["into"].v.view(torch.int8), st["into"].k_scale,
                  st["into"].v_scale, st["into"].weights):
            t.zero_()
        st["ws"] = msa.workspace(st["cache"].evict_workspace_size())
    else:
        st.update(k=k, ks=ks, v=v, vs=vs, w=w)
    st["new_cap"] = new_cap
    return st


# ---------------------------------------------------------------------------- one pass
def run(st):
    return {"rope": _rope, "append": _append, "attend": _attend, "evict": _evict}[st["c"]["op"]](st)


def _inv_freq(c):
    """Radians a position for each pair, and the magnitude, in 64 bits."""
    r, theta, f = c["rotary_dim"], 1e6, c["factor"]
    i = torch.arange(r // 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "ntk":
        theta = theta * f ** (r / (r - 2))
    inv = theta ** (-2.0 * i / r)
    if c["scaling"] == "linear":
        return inv / f, 1.0
    if c["scaling"] != "yarn":
        return inv, 1.0
    dim = lambda turns: r * math.log(c["original"] / (turns * 2 * math.pi)) / (2 * math.log(theta))
    low, high = max(math.floor(dim(32.0)), 0), min(math.ceil(dim(1.0)), r - 1)
    ramp = ((i - low) / max(high - low, 0.001)).clamp(0, 1)
    return inv / f * ramp + inv * (1 - ramp), 0.1 * math.log(f) + 1.0


def _rotate(x, cos, sin, c):
    r = c["rotary_dim"]
    y = x.float()
    if c["layout"] == "half":
        a, b = y[..., :r // 2], y[..., r // 2:r]
        rot = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = y[..., 0:r:2], y[..., 1:r:2]
        rot = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([rot, y[..., r:]], -1).to(x.dtype)


def _rope(st):
    c = st["c"]
    if own:
        call = st["rope"].backward if c["backward"] else st["rope"].rotate
        return call(st["q"], st["k"], st["pos"])
    inv, mag = _inv_freq(c)
    ang = st["pos"].double()[..., None] * inv * (-1.0 if c["backward"] else 1.0)
    cos, sin = (torch.cos(ang) * mag).float()[:, :, None], (torch.sin(ang) * mag).float()[:, :, None]
    return _rotate(st["q"], cos, sin, c), _rotate(st["k"], cos, sin, c)


def _append_plain(q, scale, x, start, n, begin, rows, c):
    """The touched blocks as values after the append: [B][rows][H][D], in the type of the rows."""
    B, H, cap, D = q.shape
    bl, T = c["block"], c["tokens"]
    at = begin[:, None].long() + torch.arange(rows, device="cuda")           # [B][rows]
    inside = (at < cap)
    row = at.clamp(max=cap - 1)
    old = torch.gather(q.view(torch.uint8), 2, row[:, None, :, None].expand(B, H, rows, D)).view(q.dtype).float()
    s_old = torch.gather(scale, 2, (row // bl)[:, None, :].expand(B, H, rows))
    is_old = at < start[:, None]
    t = at - start[:, None]
    is_new = (t >= 0) & (t < n[:, None]) & inside
    new = torch.gather(x, 1, t.clamp(0, T - 1)[:, :, None, None].expand(B, rows, H, D)).float().transpose(1, 2)
    s_old = torch.where(is_old[:, None], s_old, torch.zeros_like(s_old))
    val = torch.where(is_old[:, None, :, None], old * s_old[..., None], torch.where(is_new[:, None, :, None], new, 0.0))
    blocks = val.view(B, H, rows // bl, bl, D)
    need = _block_scale(torch.where(is_new[:, None, :, None], new, 0.0).view_as(blocks).abs().amax((3, 4)), c["fmt"])
    s = torch.maximum(need, s_old.view(B, H, rows // bl, bl).amax(3))[..., None, None]
    return (_to8(blocks, s, c["fmt"]).float() * s).view(B, H, rows, D).transpose(1, 2).to(x.dtype).contiguous()


def _append(st):
    c = st["c"]
    if own:
        cache = st["cache"]
        cache.append(st["K"], st["V"], n_tokens=st["n"], start=st["lens"])
        k, v = cache.read(st["begin"], st["rows"])
        return k, v, cache.cache_len
    a = (st["lens"], st["n"], st["begin"], st["rows"], c)
    return (_append_plain(st["k"], st["ks"], st["K"], *a), _append_plain(st["v"], st["vs"], st["V"], *a),
            st["lens"] + st["n"])


def _dequant(q, s, bl):
    B, H, cap, D = q.shape
    return (q.view(B, H, cap // bl, bl, D).float() * s[..., None, None]).view(B, H, cap, D)


def _attend(st):
    c = st["c"]
    if own:
        st["cache"].attend(st["content"], st["ids"], st["Q"], st["O"], st["ws"], lse=st["lse"], n_tokens=st["n"],
                           weight_decay=0.0 if c["weights"] else None)
        return (st["O"], st["lse"]) + ((st["cache"].weights,) if c["weights"] else ())
    B, T, Hq, D, H, cap = c["batch"], c["tokens"], c["q_heads"], c["head_dim"], c["kv_heads"], c["capacity"]
    G, cpd = Hq // H, -(-c["doc_len"] // 64)
    rows = (st["ids"].long()[:, :, None] * cpd + torch.arange(cpd, device="cuda")).view(B, -1)
    mem = st["content"][rows].float()                                        # [B][M][2][H][D]
    M = rows.shape[1]
    K = torch.cat([mem[:, :, 0].transpose(1, 2), _dequant(st["k"], st["ks"], c["block"])], 2)
    V = torch.cat([mem[:, :, 1].transpose(1, 2), _dequant(st["v"], st["vs"], c["block"])], 2)
    Q = st["Q"].float().view(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    S = torch.matmul(Q, K.transpose(2, 3)).view(B, H, T, G, M + cap) * (D ** -0.5)
    last = st["lens"][:, None] - st["n"][:, None] + torch.arange(T, device="cuda")  # the row of token t
    x = torch.arange(M + cap, device="cuda") - M
    seen = x <= last[..., None]                                              # [B][T][M + cap]
    S = S.masked_fill(~seen[:, None, :, None], float("-inf"))
    m = S.amax(-1, keepdim=True)
    P = torch.exp(S - torch.where(torch.isfinite(m), m, torch.zeros_like(m)))
    L = P.sum(-1, keepdim=True)
    real = (torch.arange(T, device="cuda") < st["n"][:, None])[:, None, :, None, None]
    lse = torch.where(real, m + torch.log(L), torch.zeros_like(m))
    P = torch.where(real & (L > 0), P / L, torch.zeros_like(P))
    O = torch.matmul(P.view(B, H, T * G, M + cap), V).view(B, H, T, G, D)
    O = O.permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(st["Q"].dtype)
    lse = lse[..., 0].permute(0, 2, 1, 3).reshape(B, T, Hq)
    if not c["weights"]:
        return O, lse
    return O, lse, P[..., M:].sum((2, 3))


def _evict(st):
    c = st["c"]
    if own:
        st["cache"].evict(c["budget"], c["recent"], st["ws"], out=st["into"])
        o, n = st["into"], st["new_cap"]
        nb = n // c["block"]
        return (o.k.view(torch.int8), o.v.view(torch.int8), o.k_scale, o.v_scale, o.weights, o.cache_len)
    B, H, D, cap, bl = c["batch"], c["kv_heads"], c["head_dim"], c["capacity"], c["block"]
    nb, dev = cap // bl, "cuda"
    lens = st["lens"].long()
    full, tail = lens // bl, lens % bl
    keep = torch.where(lens > c["budget"], (c["budget"] - tail) // bl, full)
    recent = torch.minimum(torch.full_like(keep, -(-c["recent"] // bl)), keep)
    # block weight: summed in 64 bits, compared in 32; the last ones count as infinite
    j = torch.arange(nb, device=dev)
    score = st["w"].view(B, H, nb, bl).double().sum(3).float()
    score = torch.where((j >= (full - recent)[:, None])[:, None], float("inf"), score)
    score = torch.where((j < full[:, None])[:, None], score, float("-inf"))
    order = torch.sort(score, dim=2, descending=True, stable=True).indices
    rank = torch.empty_like(order).scatter_(2, order, j.expand(B, H, nb).contiguous())
    kept = rank < keep[:, None, None]
    part = (j == full[:, None])[:, None] & (tail > 0)[:, None, None]         # the partial last block
    kept = kept | part
    # kept blocks in order, then nothing
    src = torch.sort((~kept).to(torch.uint8), dim=2, stable=True).indices    # [B][H][nb]
    new_len = keep * bl + tail
    live = (j * bl < new_len[:, None])[:, None]                              # [B][1][nb]
    rows = (torch.arange(cap, device=dev) < new_len[:, None])[:, None]       # [B][1][cap]

    def move(q):
        x = q.view(torch.int8).view(B, H, nb, bl * D)
        y = torch.gather(x, 2, src[..., None].expand(-1, -1, -1, bl * D)).view(B, H, cap, D)
        return torch.where(rows[..., None], y, torch.zeros_like(y))

    def pick(s):
        return torch.where(live, torch.gather(s, 2, src), torch.zeros_like(s))

    w = torch.gather(st["w"].view(B, H, nb, bl), 2, src[..., None].expand(-1, -1, -1, bl)).view(B, H, cap)
    return (move(st["k"]), move(st["v"]), pick(st["ks"]), pick(st["vs"]), torch.where(rows, w, torch.zeros_like(w)),
            new_len.int())


# ---------------------------------------------------------------------------- the definitions, 64 bits
def exact(c, seed):
    global own
    was, own = own, False
    try:
        st = prepare(c, seed)
    finally:
        own = was
    B, H, D = c["batch"], c["kv_heads"], c["head_dim"]
    if c["op"] == "rope":
        inv, mag = _inv_freq(c)
        z = torch.polar(torch.full_like(st["pos"].double()[..., None] * inv, mag),
                        st["pos"].double()[..., None] * inv)[:, :, None]
        z = z.conj() if c["backward"] else z
        r = c["rotary_dim"]

        def turn(x):
            y = x.double().clone()
            if c["layout"] == "half":
                u = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * z
                y[..., :r // 2], y[..., r // 2:r] = u.real, u.imag
            else:
                u = torch.complex(y[..., 0:r:2].contiguous(), y[..., 1:r:2].contiguous()) * z
                y[..., 0:r:2], y[..., 1:r:2] = u.real, u.imag
            return y
        return turn(st["q"]), turn(st["k"])
    bl = c["block"]
    if c["op"] == "append":
        qmax = QMAX[c["fmt"]]

        def grid(y):
            if c["fmt"] == "int8":
                return torch.round(y)
            step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
            return torch.round(y / step) * step

        def one(q, scale, x):
            out = torch.zeros(B, H, st["rows"], D, dtype=torch.float64, device="cuda")
            for b in range(B):
                s0, n, b0 = int(st["lens"][b]), int(st["n"][b]), int(st["begin"][b])
                end = -(-(s0 + n) // bl) * bl
                val = torch.zeros(H, end - b0, D, dtype=torch.float64, device="cuda")
                val[:, s0 - b0:s0 - b0 + n] = x[b, :n].double().transpose(0, 1)
                amax = val.view(H, -1, bl * D).abs().amax(2)
                s = torch.where(amax > 0, torch.exp2(torch.ceil(torch.log2(amax / qmax))), torch.zeros_like(amax))
                if s0 > b0:
                    first = scale[b, :, b0 // bl].double()
                    val[:, :s0 - b0] = q[b, :, b0:s0].double() * first[:, None, None]
                    s[:, 0] = torch.maximum(s[:, 0], first)
                s = s.repeat_interleave(bl, 1)[..., None]
                out[b, :, :end - b0] = grid(val / s.clamp(min=2.0 ** -140)) * s
            return out.transpose(1, 2).contiguous()
        return one(st["k"], st["ks"], st["K"]), one(st["v"], st["vs"], st["V"]), None
    if c["op"] == "evict":
        return None
    T, Hq, G, cpd = c["tokens"], c["q_heads"], c["q_heads"] // H, -(-c["doc_len"] // 64)
    O = torch.zeros(B, T, Hq, D, dtype=torch.float64, device="cuda")
    lse = torch.zeros(B, T, Hq, dtype=torch.float64, device="cuda")
    W = torch.zeros(B, H, c["capacity"], dtype=torch.float64, device="cuda")
    for b in range(B):
        ln, n = int(st["lens"][b]), int(st["n"][b])
        rows = [int(d) * cpd + i for d in st["ids"][b] for i in range(cpd)]
        M = len(rows)
        mem = st["content"][torch.tensor(rows, dtype=torch.long, device="cuda")].double()
        hide = torch.arange(ln, device="cuda")[None] > torch.arange(ln - n, ln, device="cuda")[:, None]
        hide = torch.cat([torch.zeros(n, M, dtype=torch.bool, device="cuda"), hide], 1)
        for g in range(H):
            sk = st["ks"][b, g].double().repeat_interleave(bl)[:ln, None]
            sv = st["vs"][b, g].double().repeat_interleave(bl)[:ln, None]
            K = torch.cat([mem[:, 0, g], st["k"][b, g, :ln].double() * sk])
            V = torch.cat([mem[:, 1, g], st["v"][b, g, :ln].double() * sv])
            q = st["Q"][b, :n, g * G:(g + 1) * G].double()
            z = torch.einsum("tgd,xd->tgx", q, K) / math.sqrt(D)
            z = z.masked_fill(hide[:, None], float("-inf"))
            p = torch.softmax(z, -1)
            O[b, :n, g * G:(g + 1) * G] = torch.einsum("tgx,xd->tgd", p, V)
            lse[b, :n, g * G:(g + 1) * G] = torch.logsumexp(z, -1)
            W[b, g, :ln] = p[..., M:].sum((0, 1))
    return (O, lse, W) if c["weights"] else (O, lse)
