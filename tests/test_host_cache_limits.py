"""The longest tables of a decode: tokens are counted in 32 bits, tiles ahead included, so tables that end within 255 tokens
of 2^31 are refused (before any device work: no pointer is dereferenced)."""
import pytest

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk
from test_host_cache import _decode


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return dk.load()


@pytest.mark.parametrize("ps", [16, 48, 128])
def test_tables_up_to_2_31_tokens(lib, ps):
    most = ((1 << 31) - 256) // ps
    one = dict(ps=ps, G=1, off=[0, 1], q=0)  # a null q: refused next, where the tables pass
    assert _decode(lib, mp=most, **one) == dk.DUALKV_ERR_INVALID
    assert _decode(lib, mp=most + 1, **one) == dk.DUALKV_ERR_UNSUPPORTED
    assert _decode(lib, mp=((1 << 31) - 1) // ps, **one) == dk.DUALKV_ERR_UNSUPPORTED
    assert _decode(lib, mpp=most, **one) == dk.DUALKV_ERR_INVALID
    assert _decode(lib, mpp=most + 1, **one) == dk.DUALKV_ERR_UNSUPPORTED
    assert _decode(lib, mp=((1 << 31) // ps) + 1, **one) == dk.DUALKV_ERR_INVALID
