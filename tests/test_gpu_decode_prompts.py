"""The prompts' kernel where windows cut its tiles, and where pages do not exist."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk
from test_gpu_decode import U, Case, _np, _ragged

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


# tokens that the groups see times rows and kv-heads: above 3.4 M in each
WINDOWS = [
    ("the end of one prompt", dict(groups=[0, 64], prompts=[9_001], lens=_ragged(64, 0, 700, 1), Hq=16, Hkv=4, D=128, ps=16,
                                   window=5_000)),
    ("inside a tile", dict(groups=[0, 64], prompts=[8_192], lens=list(range(64)), Hq=16, Hkv=4, D=128, ps=64, window=4_133)),
    ("blocks of rows that see different parts", dict(groups=[0, 130], prompts=[7_000], lens=[8 * i for i in range(130)], Hq=16, Hkv=2,
                                                     D=128, ps=32, window=3_333)),
    ("two prompts, ended ones", dict(groups=[0, 40, 100], prompts=[6_500, 3_001], lens=_ragged(100, -1, 1_500, 2), Hq=32, Hkv=4, D=128,
                                     ps=48, window=4_096)),
    ("narrow heads", dict(groups=[0, 64], prompts=[9_001], lens=_ragged(64, 0, 700, 3), Hq=16, Hkv=4, D=64, ps=16, window=5_000)),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("case", WINDOWS, ids=[c[0] for c in WINDOWS])
def test_windows(case, bits):
    c = Case(**case[1], bits=bits, seed=33)
    heads = c.Hq // c.Hkv
    seen = [c.prompts[g] - min(min(c.first_seen(b), c.prompts[g]) for b in range(c.groups[g], c.groups[g + 1]) if c.lens[b] >= 0)
            for g in range(c.G)]
    assert sum(n * (c.groups[g + 1] - c.groups[g]) * heads * c.Hkv for g, n in enumerate(seen)) > 3_400_000
    out, lse = c.run()
    dk.dualkv_check_status()
    c.check(out, lse, only=range(0, c.B, max(1, c.B // 30)))


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D,ps", [(128, 16), (128, 64), (64, 16), (64, 48)])
def test_pages_that_do_not_exist(D, ps, bits):
    # reported; their keys do not count, the first and the last ones, a whole tile and single pages among them
    P, N, Hq, Hkv = 5_003, 64, 16, 4
    c = Case([0, N, N + 40], [P, 4_000], _ragged(N + 40, 0, 60, 4), Hq, Hkv, D, ps, bits, seed=34)
    want, want_lse = c.run()
    dk.dualkv_check_status()
    r = np.random.default_rng(5)
    pages = -(-P // ps)
    bad = sorted({0, pages - 1, *range(pages // 2, pages // 2 + 256 // ps + 1), *r.integers(0, pages, 9).tolist()})
    for i, page in enumerate(bad):
        c.d_tables[0][0, page] = [-1, c.cache.pages, 1 << 30, -(1 << 31)][i % 4]
    out, lse = c.run()
    with pytest.raises(dk.DualKVError) as e:
        dk.dualkv_check_status()
    assert e.value.code == dk.DUALKV_ERR_DEVICE
    # the other group keeps its bits
    assert torch.equal(out[N:], want[N:]) and torch.equal(lse[:, N:], want_lse[:, N:])
    i = np.arange(P)
    i = i[~np.isin(i // ps, bad)]
    q = _np(c.q)
    for b in range(0, N, 5):
        n = c.lens[b]
        own = np.arange(n)
        k, v = (np.concatenate([x[c.tables[0][0][i // ps], :, i % ps], x[c.tables[1][b][own // ps], :, own % ps]]) for x in c.pools)
        ref, ref_lse, A, X = oc.attend(q[b], k, v, c.scale, P + n - 1, (i, P + own), 0)
        d = (4 * D + 32) * U * X
        assert np.all(np.abs(_np(out)[b] - ref) <= 2.0 ** -8 * (np.abs(ref) + A) + (2 * d[:, None] + 2.0 ** -20) * A)
        assert np.all(np.abs(_np(lse)[:, b] - ref_lse) <= d + 2.0 ** -20 + 4 * U * np.abs(ref_lse))


@pytest.mark.parametrize("bits", [16, 4])
def test_no_page_exists(bits):
    c = Case([0, 64], [6_000], [5] * 63 + [0], 16, 4, 128, 64, bits, seed=35)
    c.d_tables[0].fill_(-1)
    out, lse = c.run()
    with pytest.raises(dk.DualKVError):
        dk.dualkv_check_status()
    c.prompts = [0]
    c.check(out, lse, only=range(0, 64, 7))
    assert not bool(out[63].any()) and bool(torch.isneginf(lse[:, 63]).all())
