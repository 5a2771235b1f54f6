"""Pins of the log-probability and policy loss oracle (``oracle.policy``) -- CPU only."""
import math

import numpy as np
import pytest
import torch

from oracle import policy as opl


def test_predictor_worked_by_hand():
    # prompt p0 p1, segments a0 a1 | (empty) | c0: local row 0 is p1, rows 1.. are a0 a1 c0
    assert opl.predictor(2, [0, 2, 2, 3]).tolist() == [0, 1, 0]
    # without a prompt the openers are not predicted; a1 is predicted by row a0
    assert opl.predictor(0, [0, 2, 2, 3]).tolist() == [-1, 0, -1]


@pytest.mark.parametrize("P", [0, 3])
def test_against_autograd_on_replicated_sequences(P):
    """Each segment scored as a sequence of its own, its first token from a copy of the prompt's last row."""
    rng = np.random.default_rng(P)
    off, V, scale = [0, 3, 3, 4, 8], 7, 0.7
    M, n = opl.rows_of(P, off), off[-1]
    z, tok = rng.standard_normal((M, V)), rng.integers(0, V, n)
    tok[5] = -1
    g, h = rng.standard_normal(n), rng.standard_normal(n)
    x = torch.from_numpy(z).requires_grad_()
    total, logp, ent = 0.0, np.zeros(n), np.zeros(n)
    for a, b in zip(off, off[1:]):
        rows = x[([0] if P else []) + list(range(a + (1 if P else 0), b + (1 if P else 0)))] * scale
        lp = torch.log_softmax(rows, -1)
        H = -(lp.exp() * lp).sum(-1)
        for r in range(0 if P else 1, b - a):
            i, k = a + r, r if P else r - 1
            if tok[i] >= 0:
                total = total + g[i] * lp[k, tok[i]] + h[i] * H[k]
                logp[i], ent[i] = lp[k, tok[i]].item(), H[k].item()
    total.backward()
    got = opl.logprobs(z, tok, scale, P, off)
    np.testing.assert_allclose(got[0], logp, atol=1e-13)
    np.testing.assert_allclose(got[1], ent, atol=1e-13)
    d = opl.logprobs_backward(z, tok, scale, P, off, got[2], got[1], g, h)
    np.testing.assert_allclose(d, x.grad.numpy(), atol=1e-13)


def test_masked_rows():
    z = np.array([[0.0, -np.inf, 0.0], [-np.inf] * 3])
    logp, ent, lse = opl.logprobs(z, [2, 0], 1.0, 1, [0, 2])
    assert math.isclose(logp[0], -math.log(2)) and math.isclose(ent[0], math.log(2))
    assert lse[1] == logp[1] == -np.inf and ent[1] == 0.0
    d = opl.logprobs_backward(z, [2, 0], 1.0, 1, [0, 2], lse, ent, np.ones(2), np.ones(2))
    np.testing.assert_allclose(d, [[-0.5, 0.0, 0.5], [0.0] * 3], atol=1e-15)


def test_loss_worked_by_hand():
    # ratios 2, 0.5, 2, 4: bounds 0.75, 1.25, dual clip 3
    old = np.zeros(4)
    logp = np.log([2.0, 0.5, 2.0, 4.0])
    r = opl.loss(logp, old, None, None, [1.0, -1.0, -1.0, -1.0], None, [0, 2, 4], 0.25, 0.25, 3.0, 0.0, 0.0, "token_mean")
    # -1.25, +0.75, +2, +3
    assert math.isclose(r["loss"], (-1.25 + 0.75 + 2.0 + 3.0) / 4)
    np.testing.assert_allclose(r["dlogp"], [0.0, 0.0, 0.5, 0.0])
    assert r["stats"][3] == 0.75


@pytest.mark.parametrize("reduction", ["token_mean", "seq_mean", "seq_sum"])
def test_loss_gradients_against_central_differences(reduction):
    rng = np.random.default_rng(1)
    off = [0, 3, 3, 8, 9]
    n = off[-1]
    logp, ent, adv = rng.standard_normal(n), rng.standard_normal(n), rng.standard_normal(n)
    old, ref = logp + 0.3 * rng.standard_normal(n), logp + rng.standard_normal(n)
    mask = np.ones(n, dtype=bool)
    mask[[1, 8]] = False

    def f(lp, en):
        return opl.loss(lp, old, ref, en, adv, mask, off, 0.2, 0.3, 1.5, 0.1, 0.05, reduction)

    r = f(logp, ent)
    for i in range(n):
        e = np.zeros(n)
        e[i] = 1e-6
        assert abs((f(logp + e, ent)["loss"] - f(logp - e, ent)["loss"]) / 2e-6 - r["dlogp"][i]) < 1e-8
        assert abs((f(logp, ent + e)["loss"] - f(logp, ent - e)["loss"]) / 2e-6 - r["dentropy"][i]) < 1e-8
    assert math.isclose(r["loss"], r["stats"][0] + 0.1 * r["stats"][1] - 0.05 * r["stats"][2])


def test_reductions_with_an_empty_segment():
    mask = np.array([1, 1, 0, 0, 1], dtype=bool)
    off = [0, 2, 4, 5]
    assert opl.weights(mask, off, "token_mean").tolist() == [1 / 3, 0, 1 / 3]
    assert opl.weights(mask, off, "seq_mean").tolist() == [1 / 6, 0, 1 / 3]
    assert opl.weights(mask, off, "seq_sum").tolist() == [1 / 3, 0, 1 / 3]
    assert opl.weights(mask & False, off, "token_mean").tolist() == [0, 0, 0]
