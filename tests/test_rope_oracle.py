"""Pins of the norm-and-rotation oracle (``oracle.rope``) -- CPU only."""
import numpy as np
import pytest

from oracle import rope as orp


def test_worked_rotation():
    # one pair turned by a quarter: (1, 0) -> (0, 1); the rest of the head is kept
    x = np.array([[[1.0, 7.0, 0.0, 8.0, 9.0]]])
    y = orp.turn(x, np.array([1.0]), [np.pi / 2, 0.0], False)
    np.testing.assert_allclose(y[0, 0], [0.0, 7.0, 1.0, 8.0, 9.0], atol=1e-15)
    x = np.array([[[1.0, 0.0, 7.0, 8.0, 9.0]]])
    y = orp.turn(x, np.array([1.0]), [np.pi / 2, 0.0], True)
    np.testing.assert_allclose(y[0, 0], [0.0, 1.0, 7.0, 8.0, 9.0], atol=1e-15)


def test_positions_restart_behind_the_prompt():
    assert orp.positions(3, [0, 2, 2, 5]).tolist() == [0, 1, 2, 3, 4, 3, 4, 5]


@pytest.mark.parametrize("inter", [False, True])
def test_scores_depend_on_relative_positions(inter):
    rng = np.random.default_rng(0)
    q, k = rng.standard_normal((1, 1, 32)), rng.standard_normal((1, 1, 32))
    f = 100.0 ** (-np.arange(8) / 8.0)
    s = [float((orp.turn(q, [p + 5.0], f, inter) * orp.turn(k, [float(p)], f, inter)).sum()) for p in (0, 3, 40)]
    assert max(s) - min(s) < 1e-12
    assert np.isclose((orp.turn(q, [9.0], f, inter) ** 2).sum(), (q ** 2).sum(), rtol=1e-14)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("weights", [False, True])
def test_gradients_against_central_differences(inter, weights):
    rng = np.random.default_rng(3)
    T, H, D = 4, 2, 16
    x, dy = rng.standard_normal((T, H, D)), rng.standard_normal((T, H, D))
    w = rng.standard_normal(D) if weights else None
    pos, f = orp.positions(2, [0, 1, 2]), [1.0, 0.3, 0.1]
    dx, dw = orp.backward(x, dy, w, 1.0, 1e-3, pos, f, inter)
    loss = lambda x, w: float((orp.forward(x, w, 1.0, 1e-3, pos, f, inter) * dy).sum())  # noqa: E731
    h = 1e-5
    for idx in np.ndindex(T, H, D):
        e = np.zeros_like(x)
        e[idx] = h
        assert abs((loss(x + e, w) - loss(x - e, w)) / (2 * h) - dx[idx]) < 1e-8
    for d in range(D if weights else 0):
        e = np.zeros(D)
        e[d] = h
        assert abs((loss(x, w + e) - loss(x, w - e)) / (2 * h) - dw[d]) < 1e-8
