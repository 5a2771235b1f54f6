"""Pins of the paged-cache oracle (``oracle.cache``) -- CPU only."""
import numpy as np

import oracle
from oracle import cache as oc


def test_worked_group():
    # largest magnitude 10.5: a seventh is 1.5, which has two significant bits
    x = np.zeros((1, 32), dtype=np.float32)
    x[0, :6] = [10.5, -10.5, 0.75, -0.75, 0.74, 2.25]
    step = oc.steps(x)
    assert step.tolist() == [[1.5]]
    c = oc.codes(x, step)
    assert c[0, :7].tolist() == [15, 1, 9, 7, 8, 10, 8]
    assert oc.values(c, step)[0, :6].tolist() == [10.5, -10.5, 1.5, -1.5, 0.0, 3.0]


def test_steps_round_up_to_five_bits():
    x = np.zeros((4, 32), dtype=np.float32)
    x[:, 3] = [7.0, 7.0 * (1 + 2.0 ** -10), 7.0 * 1.96875, 0.0]  # 1, just above 1, 63/32 (six bits), nothing
    assert oc.steps(x)[:, 0].tolist() == [1.0, 1.0625, 2.0, 0.0]
    assert (oc.codes(x, oc.steps(x))[3] == 8).all()
    x[0, 5] = np.inf
    assert np.isnan(oc.steps(x)[0, 0])


def test_values_are_within_half_a_step_and_exact_in_bf16():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((50, 4, 64)) * np.exp(rng.uniform(-20, 20, (50, 4, 1)))).astype(np.float32)
    step = oc.steps(x)
    y = oc.values(oc.codes(x, step), step)
    assert np.all(np.abs(y - x) <= np.repeat(step, 32, -1) / 2 * (1 + 2.0 ** -22))
    m, _ = np.frexp(y)
    assert np.all(m * 256 == np.round(m * 256))  # eight significant bits
    again = oc.steps(y.astype(np.float32))
    assert np.all(again <= step)


def test_packed_bytes_and_rows():
    assert oc.unpack_codes(np.array([[0x21, 0xF0]], dtype=np.uint8)).tolist() == [[1, 2, 0, 15]]
    pool = np.arange(3 * 2 * 4).reshape(3, 2, 4)
    assert oc.rows(pool, [2, 0, -1], 3, 6).tolist() == [[19, 23], [0, 4], [1, 5]]


def test_attend_is_the_packed_oracles_last_row():
    # a response's last token attends to the prompt and to its own tokens: the packed layout's rule
    P, R, Hq, Hkv, D = 9, [4, 6], 4, 2, 64
    off = np.concatenate(([0], np.cumsum(R))).tolist()
    rng = np.random.default_rng(1)
    q, k, v = (rng.standard_normal((P + off[-1], h, D)).astype(np.float32) for h in (Hq, Hkv, Hkv))
    for window in (0, 5):
        ref = oracle.dualkv(P, 2, off, Hq, Hkv, D, 0.3, window, q, k, v, np.zeros_like(q))
        for n in range(2):
            own = slice(P + off[n], P + off[n + 1])
            kk, vv = (np.concatenate((x[:P], x[own])) for x in (k, v))
            out, lse, _, _ = oc.attend(q[own][-1], kk, vv, 0.3, P + R[n] - 1, (np.arange(P), P + np.arange(R[n])), window)
            np.testing.assert_allclose(out, ref["out"][P + off[n + 1] - 1], atol=1e-12)
            np.testing.assert_allclose(lse, ref["lse"][:, P + off[n + 1] - 1], atol=1e-12)
