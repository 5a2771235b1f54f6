"""Per-head norm and position rotation oracle -- TEST INFRASTRUCTURE (see ``oracle/__init__``).

fp64 numpy definitions of the step between the projections and attention on
packed rows.  The rotation is written as a complex product and its adjoint as
the product with the conjugate; positions come from ``oracle.index``.  Pinned by
``tests/test_rope_oracle.py`` (central differences, a hand-worked rotation,
norm preservation, relative positions).
"""
from __future__ import annotations

import numpy as np

from .index import build_index


def positions(P, off):
    return np.asarray(build_index(P, list(off))[1], dtype=np.float64)


def _split(x, rope_dim, interleaved):
    h = rope_dim // 2
    return (x[..., 0:rope_dim:2], x[..., 1:rope_dim:2]) if interleaved else (x[..., :h], x[..., h:rope_dim])


def turn(x, pos, inv_freq, interleaved, sign=1.0):
    """x [T, H, D] with every pair turned by sign * position * frequency."""
    x = np.asarray(x, dtype=np.float64)
    f = np.asarray(inv_freq, dtype=np.float64)
    y = x.copy()
    if f.size:
        a, b = _split(x, 2 * f.size, interleaved)
        z = (a + 1j * b) * np.exp(1j * sign * np.outer(pos, f))[:, None, :]
        ya, yb = _split(y, 2 * f.size, interleaved)
        ya[...] = z.real
        yb[...] = z.imag
    return y


def forward(x, w, w0, eps, pos, inv_freq, interleaved):
    """x [T, H, D] -> y [T, H, D]; w None: no norm."""
    x = np.asarray(x, dtype=np.float64)
    if w is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps) * (np.asarray(w, dtype=np.float64) + w0)
    return turn(x, pos, inv_freq, interleaved)


def backward(x, dy, w, w0, eps, pos, inv_freq, interleaved):
    """Gradients (dx, dw) for the upstream gradient dy; dw None without weights."""
    x = np.asarray(x, dtype=np.float64)
    dn = turn(dy, pos, inv_freq, interleaved, -1.0)
    if w is None:
        return dn, None
    r = 1.0 / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + eps)
    u = dn * (np.asarray(w, dtype=np.float64) + w0)
    dx = r * u - x * r ** 3 * np.mean(u * x, axis=-1, keepdims=True)
    return dx, (dn * x * r).sum(axis=(0, 1))
