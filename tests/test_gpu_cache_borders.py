"""4-bit keys next to a border.  Codes and scales are step functions of a key, so the arithmetic that a key comes from is part
of the definition: fp32, each operation rounded once, in this order (x a value, y its partner in the rotation):

  r = rsqrt(mean(x^2) + eps), the mean rounded from its exact value;  a = (x r) (w + w0), b = (y r) (w' + w0)
  key = (a c) - (b s) or (b c) + (a s), c and s rounded from the cosine and sine of the angle in 64 bits
  step = ceil5(max |key| / 7),  n = floor(|key| / step + 1/2)

The reference below is that, in elementary operations; codes and scales have to be equal, all of them.  The angle in 64 bits is
good to 2^-52 of itself here and in the kernel, so a cosine may be rounded otherwise where it lies that near to half way
between two floats: with angles up to 11,000 radians one in 20,000 of them, which moves a key by 2^-24 of its pair, and
so one in 10^11 over a border.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _held(k, inv_freq, weight, w0, start, interleaved):
    """Codes and scales [T, Hkv, ..] of the keys of one stream of T tokens at positions start ..."""
    T, Hkv, D = k.shape
    cache = dk.KVCache.empty(-(-T // 64), Hkv, 64, D, 4)
    pages = torch.arange(cache.pages, dtype=torch.int32, device="cuda")[None]
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    dk.cache_append(k, k, k, cache, pages, i32(T), i32(start), [0, T], inv_freq, weight, weight, EPS, w0, interleaved)
    dk.dualkv_check_status()
    flat = lambda t: t.transpose(1, 2).flatten(0, 1)[:T].cpu()  # noqa: E731
    return oc.unpack_codes(flat(cache.k).numpy()), flat(cache.k_scale).float().numpy()


def _keys(k, f, w, w0, pos, interleaved):
    x = k.float()
    if w is not None:
        mean = x.double().square().mean(-1, keepdim=True).float()
        x = x * torch.rsqrt(mean + EPS) * (w.float() + w0)
    if f is None:
        return x
    angle = pos.double()[:, None] * f.double()
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]
    y, n = x.clone(), 2 * f.numel()
    cut = ((slice(0, n, 2), slice(1, n, 2)) if interleaved else (slice(0, n // 2), slice(n // 2, n)))
    a, b = x[..., cut[0]], x[..., cut[1]]
    y[..., cut[0]], y[..., cut[1]] = a * c - b * s, b * c + a * s
    return y


def _check(codes, scales, keys):
    """Returns how many values lie within 1e-6 of a step of half way."""
    keys = keys.cpu().numpy()
    top = np.abs(keys).reshape(*keys.shape[:-1], -1, oc.GROUP).max(-1)
    step = ((top / np.float32(7)).view(np.int32) + 0x7FFFF & ~0x7FFFF).view(np.float32)
    assert np.array_equal(scales, step)
    step = np.repeat(step, oc.GROUP, -1)
    n = np.abs(keys) / np.where(step > 0, step, np.float32(1))
    assert n.dtype == np.float32
    want = np.sign(keys) * np.floor(n + np.float32(0.5)) + 8
    wrong = codes != want
    assert not wrong.any(), f"{wrong.sum()} of {wrong.size} codes"
    n = n.astype(np.float64)
    return int((np.abs(n - np.floor(n) - 0.5) < 1e-6).sum())


FORMS = [
    ("wide, offset weights, interleaved", dict(T=4000, Hkv=2, D=512, rope_dim=128, inter=True, w0=1.0, start=0, wdtype=BF)),
    ("full rotation", dict(T=8000, Hkv=4, D=128, rope_dim=128, inter=False, w0=0.0, start=3000, wdtype=torch.float32)),
    ("narrow heads, half turned", dict(T=9001, Hkv=3, D=64, rope_dim=32, inter=False, w0=0.0, start=1, wdtype=BF)),
    ("norm alone", dict(T=8000, Hkv=4, D=128, rope_dim=0, inter=False, w0=1.0, start=0, wdtype=torch.float32)),
    ("rotation alone", dict(T=6000, Hkv=5, D=128, rope_dim=64, inter=True, w0=0.0, start=0, wdtype=None)),
    ("large channels", dict(T=4000, Hkv=4, D=128, rope_dim=128, inter=False, w0=0.0, start=0, wdtype=BF, large=20.0)),
    ("small values", dict(T=4000, Hkv=4, D=128, rope_dim=128, inter=False, w0=0.0, start=0, wdtype=None, size=1e-18)),
    ("the first positions", dict(T=3, Hkv=30, D=128, rope_dim=128, inter=False, w0=0.0, start=0, wdtype=None, base=1e6)),
]


@pytest.mark.parametrize("seed", range(3))
@pytest.mark.parametrize("form", FORMS, ids=[f[0] for f in FORMS])
def test_codes_are_those_of_the_fp32_keys(form, seed):
    c = form[1]
    g = torch.Generator(device="cuda").manual_seed(17 + seed)
    k = (c.get("size", 1.0) * torch.randn(c["T"], c["Hkv"], c["D"], generator=g, device="cuda")).to(BF)
    j = torch.arange(c["rope_dim"] // 2, dtype=torch.float64)
    f = (c.get("base", 1e4) ** (-2.0 * j / max(c["rope_dim"], 1))).float().cuda() if c["rope_dim"] else None
    w = None
    if c["wdtype"] is not None:
        w = 1.0 - c["w0"] + 0.2 * torch.randn(c["D"], generator=g, device="cuda")
        w[5::37] *= c.get("large", 1.0)
        w = w.to(c["wdtype"])
    codes, scales = _held(k, f, w, c["w0"], c["start"], c["inter"])
    pos = torch.arange(c["T"], device="cuda") + c["start"]
    _check(codes, scales, _keys(k, f, w, c["w0"], pos, c["inter"]))


def _pairs(rows, rope_dim, base):
    j = torch.arange(rope_dim // 2, dtype=torch.float64)
    f = (base ** (-2.0 * j / rope_dim)).float().cuda()
    a = torch.arange(0x3f80, 0x4080, dtype=torch.int32, device="cuda").to(torch.int16).view(BF).double()  # [1, 4)
    return f, a, torch.arange(1, rows + 1, dtype=torch.float64, device="cuda")


def test_keys_a_hair_from_half_way():
    # rows whose turned values are picked so that they lie as near to half way between two codes as bf16 pairs come: of some
    # 16,000 of them hundreds within fp32's rounding.  Values 16 .. 31 of the group are not turned; one of them, 6.90625, sets the
    # step to 1 (6.90625 / 7 is far from five bits)
    D, rope_dim, rows = 64, 16, 2000
    f, a, pos = _pairs(rows, rope_dim, 1e4)
    k = torch.zeros(rows, 1, D, dtype=BF, device="cuda")
    for i in range(rope_dim // 2):
        for r0 in range(0, rows, 250):
            angle = pos[r0:r0 + 250] * f[i].double()
            x = a[:, None] * angle.cos()[:, None, None] - a * angle.sin()[:, None, None]  # [rows, a, b]
            n = x.abs()
            off = (n - n.floor() - 0.5).abs() + (n > 6.5) * 9.0
            best = off.flatten(1).argmin(1)
            k[r0:r0 + 250, 0, i] = a[best // len(a)].to(BF)
            k[r0:r0 + 250, 0, i + rope_dim // 2] = a[best % len(a)].to(BF)
    k[:, 0, 16] = 6.90625
    codes, scales = _held(k, f, None, 0.0, 1, False)
    assert np.all(scales[:, 0, 0] == 1.0)
    assert _check(codes, scales, _keys(k, f, None, 0.0, pos, False)) > 1000


def test_steps_a_hair_from_five_bits():
    # the same for the scale: pairs whose larger turned value is as near as can be to seven times a number of five bits
    D, rope_dim, rows = 64, 16, 500
    f, a, pos = _pairs(rows, rope_dim, 1e4)
    k = torch.zeros(rows, 8, D, dtype=BF, device="cuda")
    for i in range(rope_dim // 2):  # a head for each pair
        for r0 in range(0, rows, 250):
            angle = pos[r0:r0 + 250] * f[i].double()
            c, s = angle.cos()[:, None, None], angle.sin()[:, None, None]
            t = torch.maximum((a[:, None] * c - a * s).abs(), (a * c + a[:, None] * s).abs()) / 7
            m = torch.frexp(t)[0] * 32
            best = (m - m.round()).abs().flatten(1).argmin(1)
            k[r0:r0 + 250, i, i] = a[best // len(a)].to(BF)
            k[r0:r0 + 250, i, i + rope_dim // 2] = a[best % len(a)].to(BF)
    k[..., 32] = 1.0
    codes, scales = _held(k, f, None, 0.0, 1, False)
    keys = _keys(k, f, None, 0.0, pos, False)
    t = keys[..., :32].abs().amax(-1).double() / 7
    m = torch.frexp(t)[0] * 32
    assert int(((m - m.round()).abs() < 1e-6).sum()) > 100
    _check(codes, scales, keys)
