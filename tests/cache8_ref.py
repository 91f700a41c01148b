"""Plain 64-bit restatement of the 8-bit cache operators, for the tests: values are numpy float64,
one query and one head at a time, no sharing with the library."""
from __future__ import annotations

import math

import numpy as np
import torch

QMAX = {"int8": 127.0, "e4m3": 448.0}


def scale_of(amax: float, fmt: str) -> float:
    """Smallest power of two s with amax <= qmax * s (0 for amax 0)."""
    if amax == 0.0:
        return 0.0
    e = math.floor(math.log2(amax / QMAX[fmt])) - 1
    while QMAX[fmt] * 2.0 ** e < amax:
        e += 1
    return 2.0 ** max(e, -126)


def grid(y: np.ndarray, fmt: str) -> np.ndarray:
    """Round to the format, ties to even; |y| <= qmax."""
    if fmt == "int8":
        return np.round(y)
    a = np.maximum(np.abs(y), 2.0 ** -6)
    step = 2.0 ** (np.floor(np.log2(a)) - 3)
    return np.round(y / step) * step


def stored(x: np.ndarray, s: float, fmt: str) -> np.ndarray:
    """What a block of scale s holds of x, as values / s."""
    y = np.where(np.isnan(x), 0.0, x) / (s if s > 0 else 1.0)
    y = np.where(np.isinf(x), np.copysign(QMAX[fmt], x), y)
    y = np.where(s > 0, y, np.where(np.isinf(x), y, 0.0))
    return grid(np.clip(y, -QMAX[fmt], QMAX[fmt]), fmt)


class RefCache:
    """q [B][H][cap][D] (values / scale), s [B][H][cap / bl], lens [B], weights."""

    def __init__(self, B, H, cap, D, bl, fmt):
        self.B, self.H, self.cap, self.D, self.bl, self.fmt = B, H, cap, D, bl, fmt
        self.k = np.zeros((B, H, cap, D))
        self.v = np.zeros((B, H, cap, D))
        self.ks = np.zeros((B, H, cap // bl))
        self.vs = np.zeros((B, H, cap // bl))
        self.lens = np.zeros(B, dtype=np.int64)
        self.w = np.zeros((B, H, cap))

    def append(self, K, V, n=None, start=None):
        for b in range(self.B):
            s0 = int(self.lens[b] if start is None else start[b])
            cnt = K.shape[1] if n is None else int(n[b])
            if not (0 <= s0 <= self.cap and 0 <= cnt <= K.shape[1]):
                continue
            end = min(self.cap, s0 + cnt)
            for h in range(self.H):
                for q, sc, X in ((self.k, self.ks, K), (self.v, self.vs, V)):
                    for blk in range(s0 // self.bl, -(-end // self.bl)):
                        x0 = blk * self.bl
                        lo, hi = max(x0, s0), min(x0 + self.bl, end)
                        if lo >= hi:
                            continue
                        x = X[b, lo - s0:hi - s0, h].astype(np.float64)
                        fin = x[np.isfinite(x)]
                        s_old = sc[b, h, blk] if lo > x0 else 0.0
                        s = max(scale_of(float(np.abs(fin).max()) if fin.size else 0.0, self.fmt), s_old)
                        if s > s_old and lo > x0:
                            q[b, h, x0:lo] = stored(q[b, h, x0:lo] * s_old, s, self.fmt)
                        sc[b, h, blk] = s
                        q[b, h, lo:hi] = stored(x, s, self.fmt)
                self.w[b, h, s0:end] = 0.0
            self.lens[b] = end

    def values(self, b, h, which):
        q, s = (self.k, self.ks) if which == "k" else (self.v, self.vs)
        return q[b, h, :self.lens[b]] * np.repeat(s[b, h], self.bl)[:self.lens[b], None]

    def load(self, cache):
        """Take over a library cache's content (rows below cache_len)."""
        self.lens = cache.cache_len.cpu().numpy().astype(np.int64)
        for mine, its in ((self.k, cache.k), (self.v, cache.v)):
            x = its.float().cpu().numpy().astype(np.float64)
            for b in range(self.B):
                mine[b] = 0.0
                mine[b, :, :self.lens[b]] = x[b, :, :self.lens[b]]
        self.ks, self.vs = (t.cpu().numpy().astype(np.float64) for t in (cache.k_scale, cache.v_scale))
        if cache.weights is not None:
            self.w = cache.weights.cpu().numpy().astype(np.float64)
        return self

    def evict(self, budget, recent):
        bl, B = self.bl, self.B
        kept_of = {}
        for b in range(B):
            ln = int(self.lens[b])
            if ln <= budget:
                continue
            full, tail = ln // bl, ln % bl
            keep = (budget - tail) // bl
            rec = min(-(-recent // bl), keep)
            new = keep * bl + tail
            for h in range(self.H):
                w = self.w[b, h, :full * bl].reshape(full, bl)
                key = [float(np.float32(np.sum(w[j]))) for j in range(full - rec)]
                key = [-math.inf if x != x else x for x in key]
                order = sorted(range(full - rec), key=lambda j: (-key[j], j))[:keep - rec]
                src = sorted(order) + list(range(full - rec, full)) + ([full] if tail else [])
                kept_of[b, h] = src
                rows = np.concatenate([np.arange(j * bl, (j + 1) * bl) for j in src]).astype(int)[:new]
                for q, s in ((self.k, self.ks), (self.v, self.vs)):
                    q[b, h, :new] = q[b, h, rows].copy()
                    s[b, h, :len(src)] = s[b, h, src].copy()
                wr = self.w[b, h, rows].copy()
                self.w[b, h, :new] = wr
                self.w[b, h, new:ln] = 0.0
            self.lens[b] = new
        return kept_of


def attend(ref: RefCache, mem_rows, Q, n, scale=None):
    """mem_rows[b]: (K, V) [M][H][D] of the retrieved rows.  Returns O, lse, weight [B][H][cap] and
    the scales of the error bounds: sum p |v|, the largest sum |q k| / sqrt(D) of a token."""
    B, T, Hq, D = Q.shape
    G = Hq // ref.H
    O, lse = np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    W, pv, amp = np.zeros((B, ref.H, ref.cap)), np.zeros((B, T, Hq, D)), np.zeros((B, T, Hq))
    for b in range(B):
        ln = int(ref.lens[b])
        for g in range(ref.H):
            Km = np.concatenate([mem_rows[b][0][:, g], ref.values(b, g, "k")])
            Vm = np.concatenate([mem_rows[b][1][:, g], ref.values(b, g, "v")])
            M = mem_rows[b][0].shape[0]
            for t in range(int(n[b])):
                seen = M + max(0, ln - int(n[b]) + t + 1)
                for h in range(g * G, (g + 1) * G):
                    if seen == 0:
                        lse[b, t, h] = -np.inf
                        continue
                    z = Km[:seen] @ Q[b, t, h] / math.sqrt(D)
                    m = z.max()
                    p = np.exp(z - m)
                    L = p.sum()
                    lse[b, t, h] = m + math.log(L)
                    p /= L
                    O[b, t, h] = p @ Vm[:seen]
                    pv[b, t, h] = p @ np.abs(Vm[:seen])
                    amp[b, t, h] = (np.abs(Km[:seen]) @ np.abs(Q[b, t, h])).max() / math.sqrt(D)
                    W[b, g, :seen - M] += p[M:]
    return O, lse, W, pv, amp


def content_rows(mem, content, ids):
    """The retrieved chunk rows of every query, as float64."""
    c = content.float().cpu().numpy().astype(np.float64)
    off = mem.doc_chunk_offsets
    out = []
    for row in (ids.cpu().numpy() if ids is not None else []):
        r = [x for d in row for x in range(off[d], off[d + 1])]
        out.append((c[r, 0], c[r, 1]))
    return out


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().double().cpu().numpy()
