"""64-bit definitions of the 8-bit cache and of its operators, for their tests (numpy only)."""
from __future__ import annotations

import numpy as np

from tests import _serving as S

#: what the 256 codes of e4m3 stand for
E4M3 = np.array([(-1.0 if c & 128 else 1.0) * (np.nan if c & 127 == 127 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10) if c & 120
                                               else (c & 7) * 2.0 ** -9) for c in range(256)])


def values(codes, exps):
    """What codes [..., hd] and exponent bytes [...] stand for."""
    e = np.asarray(exps, np.int64)[..., None]
    return np.where(e > 0, E4M3[np.asarray(codes)] * np.exp2(e - 127.0), E4M3[np.asarray(codes)] * 0.0)


def exponent(x):
    """The exponent byte of a row x of finite values."""
    top = np.abs(x).max()
    if top == 0:
        return 0
    b = 1
    while top > 448.0 * 2.0 ** (b - 127):
        b += 1
    return b


def nearest(x, b):
    """The values nearest to x among the codes under 2^(b - 127): four significant bits, ties to even."""
    if b == 0:
        return np.zeros_like(x)
    y = x * 2.0 ** (127 - b)
    return np.rint(y / step(y)) * step(y) * 2.0 ** (b - 127)


def step(y):
    """The distance of the codes at y."""
    return np.exp2(np.maximum(np.floor(np.log2(np.where(y == 0, 1.0, np.abs(y)))), -6.0) - 3.0)


def rotate(x, pos, layout, dims=0, theta=10000.0, factor=1.0, original=0.0, low=1.0, high=4.0, magnitude=1.0):
    """x [..., head_dim] at position pos."""
    x = np.asarray(x, np.float64)
    if layout is None:
        return x.copy()
    dims = dims or x.shape[-1]
    i = np.arange(dims // 2)
    f = np.float64(theta) ** (-2.0 * i / dims)
    kept = np.clip((original * f / (2 * np.pi) - low) / (high - low), 0, 1) if original > 0 else 0.0 * f
    a = pos * f * (kept + (1 - kept) / factor)
    e0, e1 = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + dims // 2)
    out = x.copy()
    out[..., e0] = magnitude * (x[..., e0] * np.cos(a) - x[..., e1] * np.sin(a))
    out[..., e1] = magnitude * (x[..., e0] * np.sin(a) + x[..., e1] * np.cos(a))
    return out


def rotation_slack(x, layout, dims=0, magnitude=1.0, **_):
    """How far a rotation in 32 bits may be from rotate(): the sine and cosine are off by 2^-26 of a turn (9.4e-8) and their
    rounding, with the magnitude (2 x 6e-8), the two products and the sum by 2^-24 each: below 2^-21 of |a| + |b|."""
    x = np.abs(np.asarray(x, np.float64))
    out = np.zeros_like(x)
    if layout is None:
        return out
    dims = dims or x.shape[-1]
    i = np.arange(dims // 2)
    e0, e1 = (2 * i, 2 * i + 1) if layout == "interleaved" else (i, i + dims // 2)
    out[..., e0] = out[..., e1] = 2.0 ** -21 * magnitude * (x[..., e0] + x[..., e1])
    return out


def check_row(codes, b, x, slack):
    """Is the row that codes and exponent hold x (known to `slack`) in the cache's form?"""
    b, want = int(b), exponent(x)
    if b != want:  # only where the largest value is next to a border
        top = np.abs(x).max()
        i = np.abs(x).argmax()
        border = 448.0 * 2.0 ** (min(b, want) - 127)
        assert abs(b - want) == 1 and abs(top - border) <= slack[i] + 1e-300, (b, want, top)
    got = values(codes, b)
    far = 0.5 * step((np.abs(x) + slack) * 2.0 ** (127 - b)) * 2.0 ** (b - 127) if b else 0.0
    assert (np.abs(got - x) <= far + slack).all(), np.abs(got - x).max()


def lost_weights(q, k, v_codes, v_exps, scale):
    """What the weights' fp16 leaves out below its smallest step: the kernel weighs code values with w_j 2^(e_j), brought to
    2^11 or more where largest; fp16's steps end at 2^-24, so a rounding is off by 2^-25 at least there, 2^-36 of the largest
    w_j 2^(e_j), for each position and times its code."""
    if not len(k):
        return 0.0
    s = (k @ q) * scale
    w = np.exp(s - s.max())
    size = np.exp2(np.asarray(v_exps, np.float64) - 127.0)
    return 2.0 ** -36 * (w * size).max() / w.sum() * np.abs(E4M3[v_codes]).sum(0) * 1.01


def attention_tolerance(ref, weighted, score_size, n, hd, bf16, lost=0.0):
    """How far the attention over the 8-bit cache may be from `ref` (over the codes' values); lost: lost_weights().

    fp32: as the plain cache's; besides, a query's two fp16 parts leave out 2^-22 of it, which adds 4 to the score's hd + 2
    roundings of 2^-24, and the weights' parts the same of each weight (another 4 of the 2 n + 64).
    bf16: a bf16 query is exact in fp16; each weight is rounded once to fp16 (2^-11), the output once to bf16 (2^-8)."""
    rel = 2.0 ** -24 * (2 * (hd + 2 + 4) * score_size + 2 * n + 64 + 4)
    tol = rel * 2 * weighted + lost + 1e-30
    if bf16:
        tol = tol + 2.0 ** -11 * weighted * 1.01 + 2.0 ** -8 * np.abs(ref) * 1.01
    return tol


def shared_tolerance(ref, weighted, score_size, n, hd, bf16, quant, lost=0.0):
    """Behind a shared prefix: the prefix's weights are rounded to bf16 where the queries are (2^-8), what follows it as by
    the one-token attention, and the join of the parts weighs each once more (its two exponentials, 2^-22 each, are within
    the 64 roundings)."""
    if bf16 or not quant:
        return S.attention_tolerance(ref, weighted, score_size, n, hd, bf16) + lost
    return attention_tolerance(ref, weighted, score_size, n, hd, bf16, lost)
