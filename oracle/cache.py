"""Paged key/value cache oracle -- TEST INFRASTRUCTURE (see ``oracle/__init__``).

fp64 numpy definitions of the 4-bit form, of where a stream's tokens lie and of the
attention of one token per response over them.  Pinned by ``tests/test_cache_oracle.py``.
"""
from __future__ import annotations

import numpy as np

GROUP = 32


def steps(x):
    """Steps of x's groups of 32 (last dimension): a seventh of the largest magnitude, in fp32, rounded up to five
    significant bits; NaN for a group that is not finite."""
    top = np.abs(np.asarray(x, dtype=np.float32)).reshape(*x.shape[:-1], -1, GROUP).max(-1)
    t = (top / np.float32(7.0)).astype(np.float64)
    with np.errstate(invalid="ignore"):
        _, e = np.frexp(np.where(np.isfinite(t), t, 1.0))
        unit = np.ldexp(1.0, e - 5)
        return np.where(np.isfinite(t), np.ceil(t / unit) * unit, np.nan)


def codes(x, step):
    """Codes 1 .. 15 of x: nearest multiple of the group's step, from half way to the larger magnitude, plus 8."""
    x = np.asarray(x, dtype=np.float64)
    s = np.repeat(step, GROUP, -1)
    with np.errstate(invalid="ignore", divide="ignore"):
        n = np.where(s > 0, np.floor(np.abs(x) / s + 0.5), 0.0)
    return (np.sign(x) * n + 8).astype(np.int64)


def values(code, step):
    return (np.asarray(code) - 8.0) * np.repeat(np.asarray(step, dtype=np.float64), GROUP, -1)


def unpack_codes(b):
    """[..., D / 2] bytes as [..., D] codes, the even value in the low half."""
    b = np.asarray(b)
    return np.stack((b & 15, b >> 4), -1).reshape(*b.shape[:-1], -1).astype(np.int64)


def rows(pool, table_row, lo, hi):
    """Tokens [lo, hi) of a stream from a pool [pages, heads, page size, ...] as [tokens, heads, ...]."""
    ps = pool.shape[2]
    i = np.arange(lo, hi)
    page = np.asarray(table_row, dtype=np.int64)[i // ps]
    return pool[page, :, i % ps]


def attend(q, k, v, scale, position, first, window):
    """q [Hq, D] at `position` over keys [n, Hkv, D] at positions first ..: (out [Hq, D], lse [Hq],
    sum of p |v| [Hq, D], largest sum |q| |k| scale [Hq])."""
    q, k, v = (np.asarray(x, dtype=np.float64) for x in (q, k, v))
    Hq, D = q.shape
    pos = np.concatenate([np.asarray(f) for f in first])
    seen = (pos <= position) & ((position - pos < window) if window > 0 else True)
    k, v = k[seen], v[seen]
    if not k.shape[0]:
        return np.zeros((Hq, D)), np.full(Hq, -np.inf), np.zeros((Hq, D)), np.zeros(Hq)
    Hkv = k.shape[1]
    qg = q.reshape(Hkv, Hq // Hkv, D)
    x = scale * np.einsum("hgd,thd->hgt", qg, k)
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m)
    total = e.sum(-1, keepdims=True)
    p = e / total
    mag = scale * np.einsum("hgd,thd->hgt", np.abs(qg), np.abs(k)).max(-1)
    return (np.einsum("hgt,thd->hgd", p, v).reshape(Hq, D), (m + np.log(total)).reshape(Hq),
            np.einsum("hgt,thd->hgd", p, np.abs(v)).reshape(Hq, D), mag.reshape(Hq))
