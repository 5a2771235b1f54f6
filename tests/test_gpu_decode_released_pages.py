"""Pages behind a sliding window may be given away: table entries of pages that no response sees any more name no page,
or one outside the pool, and the call reports nothing and returns the same bits as before."""
import numpy as np
import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk
from test_gpu_decode import Case, _ragged

pytestmark = pytest.mark.gpu

CASES = [
    ("own pages", dict(groups=[0, 1], prompts=[0], lens=[777], Hq=4, Hkv=1, D=64, ps=16, window=100)),
    ("every offset in a tile", dict(groups=list(range(34)), prompts=[0] * 33, lens=list(range(200, 233)), Hq=2, Hkv=1, D=64, ps=16,
                                    window=40)),
    ("prompt and own", dict(groups=[0, 3, 5], prompts=[400, 331], lens=[5, 30, 0, 250, 260], Hq=8, Hkv=2, D=128, ps=16, window=90)),
    ("some ended", dict(groups=[0, 4], prompts=[300], lens=[-1, 7, 20, -1], Hq=32, Hkv=2, D=128, ps=32, window=61)),
    ("wide", dict(groups=[0, 3], prompts=[200], lens=[1, 60, 170], Hq=8, Hkv=2, D=512, ps=16, window=33)),
    ("large group", dict(groups=[0, 60], prompts=[3_000], lens=_ragged(60, 0, 300, 4), Hq=8, Hkv=2, D=64, ps=16, window=500)),
    ("block kernel", dict(groups=[0, 64], prompts=[9_000], lens=_ragged(64, 0, 300, 5), Hq=32, Hkv=8, D=128, ps=16, window=5_003)),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_pages_in_front_of_the_window(case, bits):
    pbuild.build()
    c = Case(**case[1], bits=bits, seed=60)
    want = c.run()
    dk.dualkv_check_status()
    c.check(*want)
    gone = 0
    for table, b_of, tokens in ((c.tables[0], lambda g: range(c.groups[g], c.groups[g + 1]), "prompt"),
                                (c.tables[1], lambda b: (b,), "own")):
        for i in range(len(table)):
            live = [b for b in b_of(i) if c.lens[b] >= 0]
            n = c.prompts[i] if tokens == "prompt" else max(c.lens[i], 0)
            first = min([min(c.first_seen(b), n) if tokens == "prompt" else max(0, c.lens[b] - c.window) for b in live], default=n)
            table[i, :first // c.ps] = [-1, 1 << 30][i % 2]
            gone += first // c.ps
    assert gone > 2
    for d, t in zip(c.d_tables, c.tables):
        d.copy_(torch.from_numpy(t))
    got = c.run()
    dk.dualkv_check_status()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    # a page that is seen: reported
    b = int(np.argmax(c.lens))
    c.d_tables[1][b, (c.lens[b] - 1) // c.ps] = -1
    c.run()
    with pytest.raises(dk.DualKVError):
        dk.dualkv_check_status()
