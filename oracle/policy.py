"""Token log-probability and policy loss oracle -- TEST INFRASTRUCTURE (see ``oracle/__init__``).

fp64 numpy definitions over packed response tokens, one token at a time and
row by row.  Pinned by ``tests/test_policy_oracle.py`` (torch float64 autograd
on the replicated sequences, central differences, hand-worked values).
"""
from __future__ import annotations

import math

import numpy as np


def predictor(P, off):
    """Local logits row of each response token (rows P - 1 .. T - 1, all rows if P = 0); -1 for none."""
    rows = []
    for a, b in zip(off, off[1:]):
        for i in range(a, b):
            rows.append((0 if P > 0 else -1) if i == a else (i if P > 0 else i - 1))
    return np.asarray(rows, dtype=np.int64)


def rows_of(P, off):
    return off[-1] + (1 if P > 0 else 0)


def logprobs(logits, tokens, scale, P, off):
    """(logp [n], entropy [n], lse [M]); zeros where nothing is predicted."""
    z = np.asarray(logits, dtype=np.float64) * scale
    n = off[-1]
    logp, ent, lse = np.zeros(n), np.zeros(n), np.zeros(rows_of(P, off))
    for i, m in enumerate(predictor(P, off)):
        if m < 0 or tokens[i] < 0:
            continue
        top = z[m].max()
        if top == -np.inf:
            lse[m] = logp[i] = -np.inf
            continue
        lp = z[m] - top
        lp = lp - np.log(np.exp(lp).sum())  # holds for rows of any offset, which top + log(sum) need not
        lse[m] = top - lp[z[m].argmax()]
        logp[i] = lp[tokens[i]]
        on = lp > -np.inf
        ent[i] = -(np.exp(lp[on]) * lp[on]).sum()
    return logp, ent, lse


def logprobs_backward(logits, tokens, scale, P, off, lse, entropy, dlogp, dentropy):
    """dlogits [M, V] for the given lse and entropies; dentropy None: no entropy gradient."""
    z = np.asarray(logits, dtype=np.float64) * scale
    d = np.zeros_like(z)
    for i, m in enumerate(predictor(P, off)):
        if m < 0 or tokens[i] < 0 or lse[m] == -np.inf:
            continue
        p = np.exp(z[m] - lse[m])
        d[m] -= scale * dlogp[i] * p
        d[m, tokens[i]] += scale * dlogp[i]
        if dentropy is not None:
            on = p > 0
            d[m][on] -= scale * dentropy[i] * p[on] * (z[m][on] - lse[m] + entropy[i])
    return d


def weights(mask, off, reduction):
    live = np.array([mask[a:b].sum() for a, b in zip(off, off[1:])], dtype=np.float64)
    N, total = len(live), live.sum()
    w = {"token_mean": lambda k: 1.0 / total, "seq_mean": lambda k: 1.0 / (N * k), "seq_sum": lambda k: 1.0 / N}[reduction]
    return np.array([w(k) if k else 0.0 for k in live])


def token_terms(logp, old, ref, A, lo, hi, dual):
    """One token: (policy, its derivative by logp, beyond a bound, kl, its derivative by logp)."""
    ratio = math.exp(logp - old)
    bound, beyond = ratio, False
    if A > 0 and ratio > 1 + hi:
        bound, beyond = 1 + hi, True
    elif A < 0 and ratio < 1 - lo:
        bound, beyond = 1 - lo, True
    elif A < 0 and dual and ratio > dual:
        bound, beyond = dual, True
    kl = dkl = 0.0
    if ref is not None:
        x = ref - logp
        kl = math.expm1(x) - x if abs(x) > 1e-3 else x * x * (0.5 + x / 6 + x * x / 24 + x ** 3 / 120)
        dkl = -math.expm1(x)
    return -A * bound, 0.0 if beyond else -A * ratio, beyond, kl, dkl


def loss(logp, old, ref, ent, adv, mask, off, lo, hi, dual, b, e, reduction, dloss=1.0, w=None):
    """adv per token.  Returns dict: loss, stats [4], weights, dlogp, dentropy, and what tolerances need."""
    n = off[-1]
    mask = np.ones(n, dtype=bool) if mask is None else np.asarray(mask, dtype=bool)
    w = weights(mask, off, reduction) if w is None else w
    policy = kl = H = mag = klmag = 0.0
    beyond = 0
    dlogp, dent, tol = np.zeros(n), np.zeros(n), np.zeros(n)
    for s, (a, z) in enumerate(zip(off, off[1:])):
        for i in range(a, z):
            if not mask[i]:
                continue
            r = None if ref is None else float(ref[i])
            p, dp, far, k, dk = token_terms(float(logp[i]), float(old[i]), r, float(adv[i]), lo, hi, dual)
            policy += w[s] * p
            mag += w[s] * abs(p)
            kl += w[s] * k
            x = 0.0 if r is None else r - float(logp[i])
            klmag += w[s] * (k + (math.exp(x) + 1) * abs(x))
            beyond += far
            if ent is not None:
                H += w[s] * float(ent[i])
            dlogp[i] = dloss * w[s] * (dp + b * dk)
            dent[i] = -dloss * w[s] * e
            tol[i] = abs(dloss) * w[s] * (abs(dp) + abs(b) * (abs(dk) + math.exp(x) * abs(x)))
    live = mask.sum()
    return dict(loss=policy + b * kl - e * H, stats=np.array([policy, kl, H, beyond / live if live else 0.0]), weights=w,
                dlogp=dlogp, dentropy=dent, mag=mag, klmag=klmag, entmag=0.0 if ent is None else float(
                    sum(w[s] * abs(float(ent[i])) for s, (a, z) in enumerate(zip(off, off[1:])) for i in range(a, z)
                        if mask[i])), tol=tol)
