"""4-bit keys next to a border: the code and the scale of a key are those of the exact key (here: formed in 64
bits), also where fp32 arithmetic would put it on the other side.

A key is x r (w + w0), turned by p f; step = ceil5(max |key| / 7), code = 8 + nearest(key / step).  The reference's error: an
angle p f to 2^-52 of it; the kernel's: the same, and 2^-42 of the pair's size.  With angles up to 11,000 radians,
pairs up to 100 and steps from 0.1 on a quotient is good to (2 * 11,000 * 2^-52 + 2^-42) * 1,000 = 5.2e-9; 1e-8 is left
undecided.  Where angles stay below 2,000, pairs below 6 and the step is 1, (2 * 2,000 * 2^-52 + 2^-42) * 6 = 6.8e-12; 1e-11 is.
What is half way, or a step of five bits, in 64 bits (bf16 values that are not turned) is decided.
"""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import rope as orp
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _held(k, v, inv_freq, weight, w0, start, interleaved):
    """Codes and scales [T, Hkv, ..] of the keys of one stream of T tokens at positions start ..."""
    T, Hkv, D = k.shape
    cache = dk.KVCache.empty(-(-T // 64), Hkv, 64, D, 4)
    pages = torch.arange(cache.pages, dtype=torch.int32, device="cuda")[None]
    i32 = lambda x: torch.tensor([x], dtype=torch.int32, device="cuda")  # noqa: E731
    dk.cache_append(k, k, v, cache, pages, i32(T), i32(start), [0, T], inv_freq, weight, weight, EPS, w0, interleaved)
    dk.dualkv_check_status()
    flat = lambda t: t.transpose(1, 2).flatten(0, 1)[:T].cpu()  # noqa: E731
    return oc.unpack_codes(flat(cache.k).numpy()), flat(cache.k_scale).double().numpy()


def _check(codes, scales, keys, sure):
    """Against exact keys in 64 bits; returns how many values lie within 1e-6 of a step of half way."""
    t = np.abs(keys).reshape(*keys.shape[:-1], -1, oc.GROUP).max(-1) / 7
    _, e = np.frexp(t)
    unit = np.ldexp(1.0, e - 5)
    step = np.ceil(t / unit) * unit
    off = np.abs(t / unit - np.round(t / unit))  # units are a 16th to a 31st of t
    decided = (off > 32 * sure) | (off == 0)
    assert decided.mean() > 0.99 and np.array_equal(scales[decided], step[decided])
    decided, step = (np.repeat(x, oc.GROUP, -1) for x in (decided, step))
    n = np.abs(keys) / np.where(step > 0, step, 1.0)  # a group of zeros: scale 0, code 8
    off = np.abs(n - np.floor(n) - 0.5)
    want = np.sign(keys) * np.floor(n + 0.5) + 8
    right = (codes == want) | ~decided | ((off <= sure) & (off > 0))
    assert right.all(), f"{(~right).sum()} of {right.size} codes, the farthest {off[~right].max():.2g} of a step from half way"
    return int((off < 1e-6).sum())


FORMS = [
    ("wide, offset weights, interleaved", dict(T=4000, Hkv=2, D=512, rope_dim=128, inter=True, w0=1.0, start=0, wdtype=BF)),
    ("full rotation", dict(T=8000, Hkv=4, D=128, rope_dim=128, inter=False, w0=0.0, start=3000, wdtype=torch.float32)),
    ("narrow heads, half turned", dict(T=9001, Hkv=3, D=64, rope_dim=32, inter=False, w0=0.0, start=1, wdtype=BF)),
    ("norm alone", dict(T=8000, Hkv=4, D=128, rope_dim=0, inter=False, w0=1.0, start=0, wdtype=torch.float32)),
    ("rotation alone", dict(T=6000, Hkv=5, D=128, rope_dim=64, inter=True, w0=0.0, start=0, wdtype=None)),
    ("large channels", dict(T=4000, Hkv=4, D=128, rope_dim=128, inter=False, w0=0.0, start=0, wdtype=BF, large=20.0)),
]


@pytest.mark.parametrize("form", FORMS, ids=[f[0] for f in FORMS])
def test_codes_are_those_of_the_exact_keys(form):
    c = form[1]
    g = torch.Generator(device="cuda").manual_seed(17)
    k, v = (torch.randn(c["T"], c["Hkv"], c["D"], generator=g, device="cuda").to(BF) for _ in range(2))
    j = torch.arange(c["rope_dim"] // 2, dtype=torch.float64)
    f = (1e4 ** (-2.0 * j / max(c["rope_dim"], 1))).float().cuda() if c["rope_dim"] else None
    w = None
    if c["wdtype"] is not None:
        w = 1.0 - c["w0"] + 0.2 * torch.randn(c["D"], generator=g, device="cuda")
        w[5::37] *= c.get("large", 1.0)
        w = w.to(c["wdtype"])
    codes, scales = _held(k, v, f, w, c["w0"], c["start"], c["inter"])
    pos = np.arange(c["T"], dtype=np.float64) + c["start"]
    eps = float(np.float32(EPS))
    keys = orp.forward(_np(k), None if w is None else _np(w), c["w0"], eps, pos, [] if f is None else _np(f), c["inter"])
    assert _check(codes, scales, keys, 1e-8) > 0


def test_keys_a_hair_from_half_way():
    # rows whose turned values are picked so that they lie as near to half way between two codes as bf16 pairs come: of some
    # 16,000 of them hundreds within fp32's rounding.  Values 16 .. 31 of the group are not turned; one of them, 6.90625, sets the
    # step to 1 (6.90625 / 7 is far from five bits)
    D, rope_dim, rows = 64, 16, 2000
    j = torch.arange(rope_dim // 2, dtype=torch.float64)
    f = (1e4 ** (-2.0 * j / rope_dim)).float().cuda()
    a = torch.arange(0x3f80, 0x4080, dtype=torch.int32, device="cuda").to(torch.int16).view(BF).double()  # [1, 4)
    pos = torch.arange(1, rows + 1, dtype=torch.float64, device="cuda")
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
    codes, scales = _held(k, k, f, None, 0.0, 1, False)
    keys = orp.forward(_np(k), None, 0.0, EPS, _np(pos), _np(f), False)
    assert np.all(scales[:, 0, 0] == 1.0)
    assert _check(codes, scales, keys, 1e-11) > 1000


def test_steps_a_hair_from_five_bits():
    # the same for the scale: pairs whose larger turned value is as near as can be to seven times a number of five bits
    D, rope_dim, rows = 64, 16, 500
    j = torch.arange(rope_dim // 2, dtype=torch.float64)
    f = (1e4 ** (-2.0 * j / rope_dim)).float().cuda()
    a = torch.arange(0x3f80, 0x4080, dtype=torch.int32, device="cuda").to(torch.int16).view(BF).double()
    pos = torch.arange(1, rows + 1, dtype=torch.float64, device="cuda")
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
    codes, scales = _held(k, k, f, None, 0.0, 1, False)
    keys = orp.forward(_np(k), None, 0.0, EPS, _np(pos), _np(f), False)
    t = np.abs(keys[..., :32]).max(-1) / 7
    _, e = np.frexp(t)
    unit = np.ldexp(1.0, e - 5)
    off = np.abs(t / unit - np.round(t / unit))
    sure = off > 1e-11
    assert (sure & (off < 1e-6)).sum() > 100 and np.array_equal(scales[..., 0][sure], (np.ceil(t / unit) * unit)[sure])
