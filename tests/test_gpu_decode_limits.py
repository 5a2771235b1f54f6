"""Decodes at the ends of 32 bits.  A stream of up to 2^31 - 256 tokens repeats one page, so its attention is that over the
page's tokens, each as often as it occurs.

Tolerances: as in test_gpu_decode, and for long sums: of n tokens a warp (912 of them at least) takes n / 912, and a lane
or a matrix instruction adds up 16 of those at once, so that sums, which may be cut off at each of the `adds` = n / (16 * 912)
additions, are off by `adds` 2^-23 of them.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16
MOST = 2 ** 31 - 256


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _cache(ps, Hkv, D, bits, pages=1, seed=5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    if bits == 16:
        return dk.KVCache(*(rn(pages, Hkv, ps, D).to(BF) for _ in range(2)))
    scale = [((0.1 + 0.2 * torch.rand(pages, Hkv, ps, D // 32, generator=g, device="cuda")).to(BF).view(torch.int16) & ~7).view(BF)
             for _ in range(2)]
    return dk.KVCache(*(torch.randint(0, 256, (pages, Hkv, ps, D // 2), generator=g, device="cuda", dtype=torch.uint8)
                        for _ in range(2)), *scale)


def _values(cache, page=0):
    """Keys and values of a page in 64 bits, [Hkv, ps, D]."""
    k, v = (t[page].cpu() for t in (cache.k, cache.v))
    if cache.bits == 16:
        return k.double().numpy(), v.double().numpy()
    return tuple(oc.values(oc.unpack_codes(x.numpy()), s[page].cpu().double().numpy())
                 for x, s in ((k, cache.k_scale), (v, cache.v_scale)))


def _counts(lo, hi, ps):
    """How often tokens [lo, hi) of a stream that repeats a page hit each slot."""
    full = lambda n: n // ps + (np.arange(ps) < n % ps)  # noqa: E731
    return (full(hi) - full(lo)).astype(np.float64)


def _check(out, lse, q, parts, scale, adds):
    """out [Hq, D], lse [Hq] against attention over parts (keys, values, counts)."""
    k, v = (np.concatenate([p[i] for p in parts], 1) for i in (0, 1))
    n = np.concatenate([p[2] for p in parts])
    Hkv, D = k.shape[0], k.shape[2]
    qg = q.reshape(Hkv, -1, D)
    x = scale * np.einsum("hgd,htd->hgt", qg, k)
    x = np.where(n > 0, x, -np.inf)
    m = x.max(-1, keepdims=True)
    e = np.exp(x - m) * n
    total = e.sum(-1, keepdims=True)
    p = e / total
    want, A = (np.einsum("hgt,htd->hgd", p, y).reshape(-1, D) for y in (v, np.abs(v)))
    X = scale * np.einsum("hgd,htd->hgt", np.abs(qg), np.abs(k))[..., n > 0].max(-1).reshape(-1)
    want_lse = (m + np.log(total)).reshape(-1)
    d, long = (4 * D + 32) * U * X, 2 * U * adds
    assert np.all(np.abs(out - want) <= 2.0 ** -8 * (np.abs(want) + A) + (2 * d[:, None] + 2.0 ** -20 + 2 * long) * A)
    assert np.all(np.abs(lse - want_lse) <= d + 2.0 ** -20 + 4 * U * np.abs(want_lse) + 2 * long)


def _np(t):
    return t.detach().double().cpu().numpy()


def _i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _own(n, window, D, bits, Hq, Hkv, ps, table_tokens=MOST):
    """One response of n tokens, all of them in one page."""
    cache = _cache(ps, Hkv, D, bits)
    pages = torch.zeros(1, table_tokens // ps, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(9)
    q = torch.randn(1, Hq, D, generator=g, device="cuda").to(BF)
    out, lse = dk.decode(q, cache, None, None, pages, _i32(n), [0, 1], window)
    dk.dualkv_check_status()
    lo = max(0, n - window) if window else 0
    adds = -(-(n - lo) // (16 * 912)) + 8
    _check(_np(out)[0], _np(lse)[:, 0], _np(q)[0], [(*_values(cache), _counts(lo, n, ps))], D ** -0.5, adds)


@pytest.mark.parametrize("D,bits,ps", [(64, 4, 256), (64, 16, 16), (128, 16, 32), (128, 4, 64), (512, 16, 128), (512, 4, 256)])
@pytest.mark.parametrize("n", [MOST, MOST - 1, MOST - 63, MOST - 64])
def test_a_window_at_the_end_of_the_longest_table(D, bits, ps, n):
    _own(n, 500, D, bits, 4, 1, ps)


def test_every_token_of_the_longest_table():
    _own(MOST, 0, 64, 4, 1, 1, 256)


@pytest.mark.parametrize("bits,D,times", [(16, 64, 1), (4, 128, 1), (16, 512, 1), (16, 128, 2), (4, 64, 2)])
@pytest.mark.parametrize("P,lens,window", [
    (2 ** 31 - 65536, [200_000, 150_000, 70_000, 66_000], 1000),  # every response past 2^31: the prompt is out of sight
    (2 ** 31 - 65536, [65_000, 65_536 + 600, 300, 70_000], 1000),  # some see its end
    (2 ** 31 - 65536, [0, 64, 1, 2 ** 31 - 65536], 128),
    (2 ** 31 - 65536, [100, 50_000, 7, 0], 150_000),  # 32 queries for 150,000 of its tokens: the prompts' kernel
])
def test_positions_past_2_31(bits, D, times, P, lens, window):
    # prompt and responses repeat a page each; positions run up to 2^32
    ps, Hkv = 65536, 1
    lens = lens * times
    B, Hq = len(lens), 4
    cache = _cache(ps, Hkv, D, bits, pages=2)
    prompt_pages = torch.zeros(1, P // ps, dtype=torch.int32, device="cuda")
    pages = torch.ones(B, max(lens) // ps + 1 if max(lens) < P else P // ps, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(10)
    q = torch.randn(B, Hq, D, generator=g, device="cuda").to(BF)
    out, lse = dk.decode(q, cache, prompt_pages, _i32(P), pages, _i32(*lens), [0, B], window)
    dk.dualkv_check_status()
    held = [_values(cache, page) for page in (0, 1)]
    for b, n in enumerate(lens):
        lo = max(0, P + n - window)
        parts = [(*held[0], _counts(min(lo, P), P, ps)), (*held[1], _counts(max(lo - P, 0), n, ps))]
        _check(_np(out)[b], _np(lse)[:, b], _np(q)[b], parts, D ** -0.5, 150_000 // (16 * 152) + 8)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("tiles", [2 ** 20, 2 ** 21 - 1, 2 ** 21, 2 ** 21 + 1, 2 ** 21 + 2431, 2 ** 24 - 1, 2 ** 24 + 3])
def test_deals_around_2_21_tiles(tiles, bits):
    # the deal's quotients come from fp32 below 2^21 and from integers above; tiles of 64 keys (D = 64)
    ps, D = 256, 64
    _own(64 * tiles - 5, 0, D, bits, 1, 1, ps, table_tokens=64 * 2 ** 24 + 1024)


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("lens", [[64 * 911, 1, 64 * 7001 + 3, 0], [3, 64 * 2 ** 19, 64 * 2 ** 19 + 1, 64 * 2 ** 19 - 1]])
def test_deals_of_several_sources(lens, bits):
    # some 2^21 tiles of four responses and two kv-heads (the second one's tiles behind the first one's), a page each
    ps, D, Hkv, Hq = 64, 64, 2, 4
    cache = _cache(ps, Hkv, D, bits, pages=4)
    pages = torch.arange(4, dtype=torch.int32, device="cuda")[:, None].repeat(1, max(lens) // ps + 1)
    g = torch.Generator(device="cuda").manual_seed(11)
    q = torch.randn(4, Hq, D, generator=g, device="cuda").to(BF)
    out, lse = dk.decode(q, cache, None, None, pages, _i32(*lens), [0, 1, 2, 3, 4])
    dk.dualkv_check_status()
    for b, n in enumerate(lens):
        if n:
            _check(_np(out)[b], _np(lse)[:, b], _np(q)[b], [(*_values(cache, b), _counts(0, n, ps))], D ** -0.5,
                   sum(lens) // (16 * 912) + 8)
        else:
            assert not bool(out[b].any()) and bool(torch.isneginf(lse[:, b]).all())


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("tiles", [2 ** 20 // 151, 2 ** 20 + 1, 2 ** 21 + 5])
def test_long_prompts_of_a_large_group(tiles, bits):
    # the prompts' kernel: 32 queries, tiles of 128 keys
    ps, D = 128, 64
    P = 128 * tiles - 77
    cache = _cache(ps, 1, D, bits, pages=2)
    prompt_pages = torch.zeros(1, tiles, dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(12)
    q = torch.randn(8, 4, D, generator=g, device="cuda").to(BF)
    lens = [3, 0, 100, 1, 7, 64, 65, 20]
    out, lse = dk.decode(q, cache, prompt_pages, _i32(P), torch.ones(8, 1, dtype=torch.int32, device="cuda"), _i32(*lens), [0, 8])
    dk.dualkv_check_status()
    for b, n in enumerate(lens):
        parts = [(*_values(cache, 0), _counts(0, P, ps)), (*_values(cache, 1), _counts(0, n, ps))]
        _check(_np(out)[b], _np(lse)[:, b], _np(q)[b], parts, D ** -0.5, P // (16 * 152) + 8)
