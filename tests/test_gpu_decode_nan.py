"""A NaN in a key that a query sees (a 4-bit group that was not finite has the scale NaN) is in its out and in its lse; lse -inf stays
the mark of a query that sees nothing."""
import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk
from test_gpu_decode import Case

pytestmark = pytest.mark.gpu

CASES = [
    ("walk", dict(groups=[0, 2, 4], prompts=[70, 30], lens=[40, 9, 3, 0], Hq=8, Hkv=2, D=128, ps=16)),
    ("wide", dict(groups=[0, 2, 4], prompts=[70, 30], lens=[40, 9, 3, 0], Hq=8, Hkv=2, D=512, ps=16)),
    ("block kernel", dict(groups=[0, 64, 128], prompts=[3_000, 2_000], lens=[5] * 128, Hq=16, Hkv=2, D=64, ps=16)),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_nan_is_seen(case, bits):
    pbuild.build()
    c = Case(**case[1], bits=bits, seed=8)
    out, lse = c.run()
    rows, heads = c.groups[1], c.Hq // c.Hkv
    # a key of the first prompt's second kv-head, then one of the last response but one's
    keys = c.cache.k if bits == 16 else c.cache.k_scale
    for table, token, first, last in ((c.tables[0][0], 21, 0, rows), (c.tables[1][c.B - 2], 2, c.B - 2, c.B - 1)):
        at = (int(table[token // c.ps]), 1, token % c.ps, 1)
        kept = keys[at].clone()
        keys[at] = float("nan")
        got, got_lse = c.run()
        dk.dualkv_check_status()
        hit = torch.zeros(c.B, c.Hq, dtype=torch.bool, device="cuda")
        hit[first:last, heads:] = True
        assert bool(torch.isnan(got[hit]).all()) and bool(torch.isnan(got_lse.t()[hit]).all())
        assert torch.equal(got[~hit], out[~hit]) and torch.equal(got_lse.t()[~hit], lse.t()[~hit])
        keys[at] = kept
