"""The per-token operators on seeded random layouts, sizes and options, against the fp64 oracle with the
tolerances that tests/test_gpu_rope.py, tests/test_gpu_logprobs.py and tests/test_gpu_policy.py derive."""
import random

import numpy as np
import pytest
import torch

import test_gpu_logprobs as tl
import test_gpu_policy as tp
import test_gpu_rope as tr
from oracle import policy as opl
from oracle import rope as orp
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _layout(rng, most):
    """P and offsets of a few responses, some of them empty, with at least one row."""
    R = [rng.choice([0, 1, rng.randrange(1, most)]) for _ in range(rng.randrange(1, 7))]
    P = rng.choice([0, 1, rng.randrange(1, most)])
    if P + sum(R) == 0:
        R[0] = 1
    return P, [0] + np.cumsum(R).tolist()


@pytest.mark.parametrize("seed", range(12))
def test_norm_and_rotation(seed):
    rng = random.Random(100 + seed)
    P, off = _layout(rng, 90)
    N, T = len(off) - 1, P + off[-1]
    D = rng.choice([64, 128, 512])
    Hkv = rng.randrange(1, 5)
    Hq = Hkv * rng.randrange(1, 6)
    rope_dim = 16 * rng.randrange(0, D // 16 + 1)
    inter, w0 = rng.random() < 0.5, rng.choice([0.0, 1.0])
    q, k, qw, kw, f, dq_out, dk_out = tr._inputs(P, off, Hq, Hkv, D, rope_dim, rng.choice([None, BF, F32]),
                                                 rng.random() < 0.5, seed, base=rng.choice([10.0, 1e4]))
    f = f if rope_dim else None
    y = dk.qk_norm_rope(q, k, P, off, f, qw, kw, tr.EPS, w0, inter)
    g = dk.qk_norm_rope_backward(q, k, dq_out, dk_out, P, off, f, qw, kw, tr.EPS, w0, inter)
    pos, fn = orp.positions(P, off), [] if f is None else tr._np(f)
    for i, (x, w, dy) in enumerate(((q, qw, dq_out), (k, kw, dk_out))):
        wn = None if w is None else tr._np(w)
        tr._check_forward(tr._np(y[i]), tr._np(x), wn, w0, pos, fn, inter)
        dw = None if w is None else tr._np(g[2 + i])
        tr._check_backward(tr._np(g[i]), dw, tr._np(x), tr._np(dy), wn, w0, pos, fn, inter)


@pytest.mark.parametrize("seed", range(12))
def test_token_log_probabilities(seed):
    rng = random.Random(200 + seed)
    P, off = _layout(rng, 40)
    V = rng.choice([rng.randrange(1, 40), rng.randrange(1000, 9000), rng.randrange(30000, 90000)])
    dtype, scale = rng.choice([BF, F32]), rng.choice([1.0, 0.5, 2.0])
    logits, tok, dlogp, dent = tl._inputs(P, off, V, dtype, rng.randrange(0, 9), seed, ignored=rng.choice([0.0, 0.3, 1.0]))
    if V > 4 and rng.random() < 0.5:
        logits[:, V // 3: V // 2] = -float("inf")
    entropy = rng.random() < 0.5
    if opl.rows_of(P, off) == 0:
        return
    got = dk.token_logprobs(logits, tok, P, off, scale=scale, entropy=entropy)
    tl._check_forward(got, logits, tok, scale, P, off)
    kw = dict(entropy=got[1], dentropy=dent) if entropy else {}
    d = dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off, scale=scale, **kw)
    tl._check_backward(d, logits, tok, scale, P, off, got[2], got[1], dlogp, dent if entropy else None)
    dk.dualkv_check_status()


@pytest.mark.parametrize("seed", range(16))
def test_policy_loss(seed):
    rng = random.Random(300 + seed)
    _, off = _layout(rng, rng.choice([20, 3000]))
    if off[-1] == 0:
        off[-1] = 5
    per_token = rng.random() < 0.5
    # up to differences of several units, where the ratio comes from the exponential itself
    x = tp._inputs(off, seed, per_token, rng.choice([None, 0.2, 0.95]), sigma=rng.choice([0.02, 0.3, 3.0]))
    b, e = rng.choice([0.0, 0.05]), rng.choice([0.0, 0.01, -0.1])
    if b == 0.0 and rng.random() < 0.5:
        x["ref"] = None
    if e == 0.0 and rng.random() < 0.5:
        x["ent"] = None
    tp._run_and_check(x, off, rng.choice([0.0, 0.2, 0.9]), rng.choice([0.0, 0.28, 5.0]), rng.choice([0.0, 1.5, 10.0]), b, e,
                      rng.choice(list(dk.LOSS_REDUCTIONS)), per_token)
