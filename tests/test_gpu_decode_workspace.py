"""Nothing is written behind a decode's workspace, in any form of its kernels, with as many partial results as can be."""
import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk
from test_gpu_decode import Case, _ragged

pytestmark = pytest.mark.gpu

CASES = [
    ("one response", dict(groups=[0, 1], prompts=[0], lens=[40_000], Hq=4, Hkv=1, ps=64)),
    ("eight rows", dict(groups=[0, 3], prompts=[9_000], lens=[9_000, 2_000, 7], Hq=16, Hkv=2, ps=16)),
    ("sixteen rows", dict(groups=[0, 3], prompts=[9_000], lens=[9_000, 2_000, 7], Hq=32, Hkv=2, ps=16)),
    ("large group", dict(groups=[0, 64], prompts=[6_000], lens=_ragged(64, 0, 400, 6), Hq=16, Hkv=2, ps=32)),
    ("large group, sixteen rows", dict(groups=[0, 9, 12], prompts=[7_000, 3_000], lens=_ragged(12, 0, 900, 7), Hq=32, Hkv=2, ps=32)),
]


@pytest.mark.parametrize("window", [0, 2_500])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("D", [64, 128, 512])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_its_end_is_kept(case, D, bits, window):
    pbuild.build()
    c = Case(**case[1], D=D, bits=bits, window=window, seed=12)
    need = dk.dualkv_decode_workspace_bytes(c.G, c.groups, c.Hq, c.Hkv, D)
    ws = torch.full((need + (1 << 20),), 0xA5, dtype=torch.uint8, device="cuda")
    out, lse = c.run(workspace=ws[:need])
    dk.dualkv_check_status()
    assert bool((ws[need:] == 0xA5).all())
    c.check(out, lse, only=range(0, c.B, max(1, c.B // 6)))
