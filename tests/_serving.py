"""64-bit definitions of the serving operators, for their tests (numpy only)."""
from __future__ import annotations

import numpy as np


def sample_row(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """The token of one row (include/mfs.h, mfs_sample_rows), in float64."""
    x = np.asarray(logits, np.float64)
    cols = np.nonzero(~np.isnan(x))[0]
    if cols.size == 0:
        return 0
    order = cols[np.argsort(-x[cols], kind="stable")]
    top = x[order[0]]
    if not temperature > 0 or top == -np.inf:
        return int(order[0])

    def weight(v):
        with np.errstate(invalid="ignore", over="ignore"):
            return np.where(v == top, 1.0, np.exp((v - top) / np.float64(temperature)))

    w = weight(x[order])
    m = len(order)
    if min_p > 0:
        m = int((w >= min(np.float64(min_p), 1.0)).sum())
    if top_k > 0:
        m = min(m, int(top_k))
    if top_p < 1:
        c = np.cumsum(w[:m])
        m = min(m, 1 + int(np.searchsorted(c, max(0.0, np.float64(top_p)) * c[-1], side="left")))
    kept = np.sort(order[:m])
    c = np.cumsum(weight(x[kept]))
    at = int(np.searchsorted(c, max(0.0, np.float64(u)) * c[-1], side="right"))
    return int(kept[min(at, np.nonzero(weight(x[kept]))[0][-1])])


def rotate(x, pos, rope, theta):
    """x [..., head_dim] at position pos, float64."""
    x = np.asarray(x, np.float64)
    if rope is None:
        return x.copy()
    hd = x.shape[-1]
    i = np.arange(hd // 2)
    a = pos * np.float64(theta) ** (-2.0 * i / hd)
    e0, e1 = (2 * i, 2 * i + 1) if rope == "interleaved" else (i, i + hd // 2)
    out = np.empty_like(x)
    out[..., e0] = x[..., e0] * np.cos(a) - x[..., e1] * np.sin(a)
    out[..., e1] = x[..., e0] * np.sin(a) + x[..., e1] * np.cos(a)
    return out


def attend(q, k, v, scale):
    """One query row over keys k, values v [n, head_dim], float64: the output, sum_j p_j |v_j| (what errors of
    the weights act on), and the largest scale * sum_e |q_e k_je| (what errors of the scores act on)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    if k.shape[0] == 0:
        return np.zeros(q.shape[-1]), np.zeros(q.shape[-1]), 0.0
    s = (k @ q) * scale
    p = np.exp(s - s.max())
    p /= p.sum()
    return p @ v, p @ np.abs(v), float((np.abs(k) @ np.abs(q)).max() * scale)


def attention_tolerance(ref, weighted, score_size, n, hd, bf16):
    """How far an output may be from `ref`.

    fp32: a score's products and sums are each off by 2^-24 of at most score_size (hd + 2 of them), which moves a
    weight by twice that, relatively; the exponential is within 2^-22; the sums over n keys add n 2^-24, the
    rescaling of the running sums as much again.
    bf16: besides, each weight is rounded once (2^-8) and the output once (2^-8)."""
    rel = 2.0 ** -24 * (2 * (hd + 2) * score_size + 2 * n + 64)
    tol = rel * 2 * weighted + 1e-30
    if bf16:
        tol = tol + 2.0 ** -8 * weighted * 1.01 + 2.0 ** -8 * np.abs(ref) * 1.01
    return tol


def kv_rows(cache_k, table_row, page_size, lo, hi):
    """Rows lo .. hi - 1 of one sequence from a pool [pages, heads, page_size, hd]: [hi - lo, heads, hd]."""
    return np.stack([cache_k[table_row[p // page_size], :, p % page_size] for p in range(lo, hi)]) if hi > lo else \
        np.zeros((0,) + cache_k.shape[1:2] + cache_k.shape[3:])
