"""Rotary positions (msa_rope_apply) against the formula in fp64.

Bound: the angle is exact modulo a turn up to its rounding to 24 bits (pi * 2^-25 rad), sincospi
adds two units in the last place, the magnitude one rounding and each of the two products and the
sum one: together below 2^-21 of |magnitude| (|a| + |b|).  A bf16 output adds half a step."""
import math

import numpy as np
import pytest
import torch

from cache8_ref import f64

pytestmark = pytest.mark.gpu


def freqs(r, theta, scaling, factor, original):
    i = np.arange(r // 2, dtype=np.float64)
    if scaling == "ntk":
        theta = theta * factor ** (r / (r - 2))
    inv = theta ** (-2 * i / r)
    if scaling == "linear":
        inv = inv / factor
    mag = 1.0
    if scaling == "yarn":
        idx = lambda turns: r * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(theta))
        low, high = max(math.floor(idx(32)), 0), min(math.ceil(idx(1)), r - 1)
        ramp = np.clip((i - low) / max(high - low, 0.001), 0, 1)
        inv = inv / factor * ramp + inv * (1 - ramp)
        mag = 0.1 * math.log(factor) + 1
    return inv, mag


def reference(x, pos, r, layout, inv, mag, sign):
    ang = pos[..., None].astype(np.float64) * inv * sign
    c, s = (np.cos(ang) * mag)[..., None, :], (np.sin(ang) * mag)[..., None, :]
    y, size = x.copy(), np.zeros_like(x)
    ia, ib = (slice(0, r // 2), slice(r // 2, r)) if layout == "half" else (slice(0, r, 2), slice(1, r, 2))
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, b * c + a * s
    size[..., ia] = size[..., ib] = abs(mag) * (np.abs(a) + np.abs(b))
    return y, size


def check(got, want, size):
    want, tol = want, 2.0 ** -21 * size
    if got.dtype == torch.bfloat16:
        tol = tol + 2.0 ** -8 * (np.abs(want) + tol)
    err = np.abs(f64(got) - want)
    assert np.all(err <= tol), f"worst {np.max(err - tol):.3e} over at error {err.max():.3e}"


CASES = [
    # dtype, lead, Hq, Hk, D, r, layout, scaling, factor, original
    ("bf16", (1,), 1, 1, 128, 128, "half", "none", 1, 0),
    ("bf16", (3, 17), 32, 8, 128, 128, "half", "yarn", 8, 4096),
    ("f32", (2, 5), 8, 2, 64, 64, "interleaved", "linear", 4, 0),
    ("f32", (37,), 3, 5, 64, 32, "half", "ntk", 4, 0),
    ("bf16", (2, 9), 5, 0, 64, 48, "interleaved", "none", 1, 0),
    ("bf16", (4, 3), 2, 2, 10, 6, "half", "none", 1, 0),       # no 16-byte rows
    ("f32", (4, 3), 2, 1, 14, 10, "interleaved", "yarn", 2, 64),
    ("f32", (2,), 1, 1, 512, 512, "half", "none", 1, 0),
    ("bf16", (1, 300), 1, 1, 64, 2, "half", "linear", 3, 0),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("backward", [False, True])
def test_rope_matches_the_formula(case, backward):
    from top_document_sparse_b200 import msa
    dt, lead, Hq, Hk, D, r, layout, scaling, factor, original = case
    dtype = torch.bfloat16 if dt == "bf16" else torch.float32
    g = torch.Generator(device="cuda").manual_seed(sum(lead) + D)
    q = torch.randn(*lead, Hq, D, generator=g, device="cuda").to(dtype)
    k = torch.randn(*lead, Hk, D, generator=g, device="cuda").to(dtype) if Hk else None
    pos = torch.randint(0, 3_000_000_000, lead, generator=g, device="cuda")
    pos.view(-1)[0] = 0
    rope = msa.Rope(D, r, 1e6, layout, scaling, factor, original)
    fn = rope.backward if backward else rope.rotate
    qo, ko = fn(q, k, pos)
    inv, mag = freqs(r, 1e6, scaling, factor, original)
    sign = -1.0 if backward else 1.0
    for x, y in ((q, qo), (k, ko)):
        if x is None:
            assert y is None
            continue
        want, size = reference(f64(x), pos.cpu().numpy(), r, layout, inv, mag, sign)
        # fp64 angles of positions up to 3e9 are themselves off by up to 3e9 * 2^-53 * 2 rad
        check(y, want, size * (1 + 3e9 * 2.0 ** -52 * 2.0 ** 21))
        assert torch.equal(y[..., r:], x[..., r:])


def test_rope_in_place_slices_negative_positions_and_no_tokens():
    from top_document_sparse_b200 import msa
    B, T, Hq, Hk, D = 3, 7, 4, 2, 64
    qkv = torch.randn(B, T, (Hq + 2 * Hk) * D, device="cuda").bfloat16()
    keep = qkv.clone()
    q, k = qkv[..., :Hq * D].view(B, T, Hq, D), qkv[..., Hq * D:(Hq + Hk) * D].view(B, T, Hk, D)
    pos = torch.arange(B * T, device="cuda").view(B, T) - 9
    rope = msa.Rope(D)
    qo, ko = rope.rotate(q, k, pos)
    rope.rotate(q, k, pos, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(qkv[..., (Hq + Hk) * D:], keep[..., (Hq + Hk) * D:])  # V untouched
    inv, mag = freqs(D, 1e6, "none", 1, 0)
    want, size = reference(f64(keep[..., :Hq * D].reshape(B, T, Hq, D)), pos.cpu().numpy(), D, "half",
                           inv, mag, 1.0)
    check(qo, want, size)
    # an odd start: rows that are not 16-byte aligned take the scalar path
    flat = torch.randn(1 + B * T * Hq * D, device="cuda")
    odd = flat[1:].view(B, T, Hq, D)
    want, size = reference(f64(odd), pos.cpu().numpy(), D, "half", inv, mag, 1.0)
    check(rope.rotate(odd, None, pos)[0], want, size)
    none, _ = rope.rotate(q[:, :0], None, pos[:, :0])
    assert none.shape == (B, 0, Hq, D)


def test_rope_gradient_against_differences():
    """d/dx of sum(w * rotate(x)): the map is linear, so a difference of step 1 is its gradient up to
    rounding: three fp32 roundings of sums of |w| (|a| + |b|)-sized terms a side."""
    from top_document_sparse_b200 import msa
    rope = msa.Rope(16, 8, 1e4, "interleaved", "yarn", 4.0, 128)
    x = torch.randn(5, 2, 16, device="cuda")
    w = torch.randn(5, 2, 16, device="cuda")
    pos = torch.tensor([0, 1, 77, 1000, 123456], device="cuda")
    grad, _ = rope.backward(w, None, pos)
    base = f64(rope.rotate(x, None, pos)[0])
    for i in range(16):
        step = x.clone()
        step[..., i] += 1.0
        diff = (f64(rope.rotate(step, None, pos)[0]) - base) * f64(w)
        bound = 2.0 ** -20 * (np.abs(f64(x)).max() + 2) * np.abs(f64(w)).sum(-1) * 1.2
        assert np.all(np.abs(diff.sum(-1) - f64(grad)[..., i]) <= bound)


def test_rope_refuses():
    from top_document_sparse_b200 import msa
    rope = msa.Rope(64)
    q = torch.randn(2, 3, 4, 64, device="cuda")
    pos = torch.zeros(2, 3, dtype=torch.int64, device="cuda")
    for bad in (lambda: rope.rotate(q, None, pos.int()), lambda: rope.rotate(q[..., :32], None, pos),
                lambda: rope.rotate(q, q.bfloat16(), pos), lambda: rope.rotate(q, None, pos[:, :2]),
                lambda: rope.rotate(q.transpose(1, 2).contiguous().transpose(1, 2), None, pos),
                lambda: rope.rotate(q, None, pos.cpu()), lambda: rope.rotate(q.half(), None, pos)):
        with pytest.raises((ValueError, TypeError)):
            bad()


def test_rope_on_another_stream_leaves_freed_blocks_alone():
    """A block that the current stream freed while work there still reads it must not become the
    output of a call on another stream."""
    from top_document_sparse_b200 import msa
    rope = msa.Rope(64)
    n = 5000
    q = torch.randn(n, 8, 64, device="cuda")
    pos = torch.arange(n, device="cuda")
    other = torch.cuda.Stream()
    keep = torch.empty_like(q)
    torch.cuda.synchronize()
    want, _ = rope.rotate(q, None, pos)
    torch.cuda.synchronize()
    freed = torch.full_like(q, 7.0)
    torch.cuda._sleep(20_000_000)
    keep.copy_(freed)
    del freed  # its block is free for the current stream's next allocation
    got, _ = rope.rotate(q, None, pos, stream=other)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and torch.all(keep == 7.0)


@pytest.mark.parametrize("original", [1, 4, 6, 7])
def test_rope_yarn_of_short_original_lengths(original):
    """Where no pair turns once within original_length (2 pi positions) every frequency is divided by
    the factor, as in linear scaling; above it pair 0 keeps its own."""
    from top_document_sparse_b200 import msa
    x = torch.randn(9, 2, 64, device="cuda")
    pos = torch.arange(9, device="cuda") * 1001
    yarn, _ = msa.Rope(64, scaling="yarn", factor=4.0, original_length=original, magnitude=1.0).rotate(x, None, pos)
    linear, _ = msa.Rope(64, scaling="linear", factor=4.0, magnitude=1.0).rotate(x, None, pos)
    plain, _ = msa.Rope(64, magnitude=1.0).rotate(x, None, pos)
    if original < 2 * math.pi:
        assert torch.equal(yarn, linear)
    else:
        assert torch.equal(yarn[..., ::32], plain[..., ::32]) and torch.equal(yarn[..., 1::32], linear[..., 1::32])
