"""A decode's workspace holds what the kernels of its form can leave, no more: a slot is a maximum, a sum, a count and
a place (16 bytes) and D floats."""
import pytest

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


@pytest.mark.parametrize("B,Hq,Hkv,D,behind", [
    (4, 8, 2, 512, 152 * 8 * 8),               # 8 warps of 8 rows to a block, no prompts' kernel at this width
    (500, 8, 2, 512, 152 * 8 * 8),
    (1, 32, 8, 128, 152 * 16 * 8),             # 16 warps of 8 rows, too few rows for the prompts' kernel
    (7, 4, 1, 64, 152 * 16 * 8),
    (8, 4, 1, 64, 152 * (16 * 8 + 128)),       # 32 rows
    (32, 32, 8, 128, 152 * (16 * 8 + 128)),
    (1, 16, 1, 128, 152 * 12 * 16),            # 12 warps of 16 rows
    (2, 16, 1, 128, 152 * (12 * 16 + 128)),
])
def test_bytes(B, Hq, Hkv, D, behind):
    slots = 2 * B * Hq + behind
    assert dk.dualkv_decode_workspace_bytes(1, [0, B], Hq, Hkv, D) == -(-16 * slots // 256) * 256 + 4 * D * slots
