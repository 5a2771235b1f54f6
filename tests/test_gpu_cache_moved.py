"""A cache whose tensors were replaced, grown, set to other memory or freed is refused: calls would go on with memory that may
have been given to others."""
import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
NAMES = {16: ("k", "v"), 4: ("k", "v", "k_scale", "v_scale")}
MOVES = {
    "set to other memory": lambda t: t.set_(torch.zeros_like(t)),
    "other data": lambda t: setattr(t, "data", torch.zeros_like(t)),
    "grown": lambda t: t.resize_(t.shape[0] + 100, *t.shape[1:]),
    "freed": lambda t: t.untyped_storage().resize_(0),
}


def _calls(cache):
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.ones(1, cache.Hkv, cache.D, dtype=torch.bfloat16, device="cuda")
    table, lens = i32(0)[None], i32(1)
    return [lambda: dk.cache_append(x, x, x, cache, table, lens, i32(0), [0, 1]), lambda: dk.cache_read(cache, table, lens, [0, 1]),
            lambda: dk.decode(x, cache, None, None, table, lens, [0, 1])]


@pytest.mark.parametrize("move", MOVES)
@pytest.mark.parametrize("bits,name", [(b, n) for b in NAMES for n in NAMES[b]])
def test_a_moved_pool_is_refused(bits, name, move):
    pbuild.build()
    cache = dk.KVCache.empty(16, 2, 16, 64, bits)
    for call in _calls(cache):
        call()
    MOVES[move](getattr(cache, name))
    for call in _calls(cache):
        with pytest.raises(ValueError):
            call()
    dk.dualkv_check_status()


def test_attributes_stay():
    cache = dk.KVCache.empty(3, 2, 16, 64, 4)
    assert (cache.pages, cache.Hkv, cache.page_size, cache.D, cache.bits, cache.device) == (3, 2, 16, 64, 4, 0)
    for name in ("k", "v", "k_scale", "v_scale", "pages", "Hkv", "page_size", "D", "bits", "device"):
        with pytest.raises(AttributeError):
            setattr(cache, name, getattr(cache, name))
    assert cache.k.shape == (3, 2, 16, 32) and cache.v_scale.shape == (3, 2, 16, 2)
    assert dk.KVCache.empty(3, 2, 16, 64).k_scale is None
