"""GPU parity of dualkv_cache_append and dualkv_cache_read against ``oracle.rope`` and ``oracle.cache`` (fp64).

Tolerances, with u = 2^-24 (half an fp32 step):
  q, bf16 k   as dualkv_qk_norm_rope's: 2^-8 |y| for the rounding to bf16 plus 32 u (|n_a| + |n_b|) for the fp32
              arithmetic on the value's pair (error e below).
  bf16 v, what is read back   exact.
  4-bit v     codes and scales exact: a bf16 value over a step of five bits is never within an fp32 rounding of
              half way without being half way.
  4-bit k     the exact k is off by at most e from the fp32 one, whose group's scale is a seventh of its largest
              magnitude (one rounding) rounded up by less than one part in 16; the value that a code
              stands for is within half a step of it (and 2 u of the quotient's 8).
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import cache as oc
from oracle import rope as orp
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
EPS = 1e-5
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _tables(counts, ps, extra, seed):
    """Page table of streams with these tokens from a shuffled pool of `extra` more pages than they need."""
    need = [-(-n // ps) for n in counts]
    pool = sum(need) + extra
    order = np.random.default_rng(seed).permutation(pool)
    t = np.full((len(counts), max(need + [1])), -1, dtype=np.int32)
    at = 0
    for i, k in enumerate(need):
        t[i, :k] = order[at:at + k]
        at += k
    return pool, t


def _fill(cache, value):
    """A pattern that shows which places a call writes."""
    for t in (cache.k, cache.v, cache.k_scale, cache.v_scale):
        if t is not None:
            t.fill_(value)


class Case:
    def __init__(self, rows, held, starts, Hq, Hkv, D, ps, bits, rope_dim=None, inter=False, wdtype=BF, w0=0.0, fused=True,
                 seed=0, base=1e4):
        rope_dim = D if rope_dim is None else rope_dim
        self.rows, self.lens, self.starts = rows, [a + b for a, b in zip(rows, held)], starts
        self.off = [0] + np.cumsum(rows).tolist()
        self.T, self.S, self.Hq, self.Hkv, self.D, self.ps, self.bits = self.off[-1], len(rows), Hq, Hkv, D, ps, bits
        self.inter, self.w0, self.rope_dim = inter, w0, rope_dim
        self.pool, self.table = _tables(self.lens, ps, 2, seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
        if fused:
            row = rn(self.T, (Hq + 2 * Hkv) * D + 8)
            cut = (0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D)
            self.q, self.k, self.v = (row[:, a:b].view(self.T, (b - a) // D, D) for a, b in zip(cut, cut[1:]))
        else:
            self.q, self.k, self.v = rn(self.T, Hq, D), rn(self.T, Hkv, D), rn(self.T, Hkv, D)
        self.w = [None, None]
        if wdtype is not None:
            self.w = [(0.3 * torch.randn(D, generator=g, device="cuda") + 1).to(wdtype) for _ in range(2)]
        self.f = (base ** (-2.0 * torch.arange(rope_dim // 2, dtype=torch.float64) / max(rope_dim, 1))).float().cuda()
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.d_table, self.d_lens, self.d_starts = torch.from_numpy(self.table).cuda(), i32(self.lens), i32(starts)
        self.cache = dk.KVCache.empty(self.pool, Hkv, ps, D, bits)
        _fill(self.cache, 7)
        self.index = np.concatenate([np.arange(n - r, n) for n, r in zip(self.lens, rows)]).astype(np.int64)
        self.stream = np.repeat(np.arange(self.S), rows)
        self.pos = (self.index + np.asarray(starts)[self.stream]).astype(np.float64)

    def append(self, q_out, stream=None):
        dk.dualkv_cache_append(self.q, self.k, self.v, *self.w, self.w0, EPS, self.f, self.rope_dim, self.inter, self.cache,
                               self.d_table, self.d_lens, self.d_starts, self.S, self.off, self.Hq, self.Hkv, self.D, q_out,
                               stream)

    def places(self):
        return self.table[self.stream, self.index // self.ps], self.index % self.ps


CASES = [
    ("one-token", Case, dict(rows=[1], held=[0], starts=[0], Hq=1, Hkv=1, D=64, ps=16)),
    ("a step", Case, dict(rows=[1] * 9, held=[0, 15, 16, 17, 31, 40, 3, 100, 63], starts=[64] * 9, Hq=2, Hkv=2, D=64, ps=16,
                          fused=False, wdtype=torch.float32, seed=1)),
    ("some streams idle", Case, dict(rows=[0, 3, 0, 0, 1, 0], held=[5, 14, 0, 0, 0, 9], starts=[0, 7, 0, 0, 1, 2], Hq=4,
                                     Hkv=2, D=128, ps=16, seed=2)),
    ("prompt and responses", Case, dict(rows=[70, 33, 5, 120], held=[0, 0, 0, 0], starts=[0, 70, 70, 70], Hq=8, Hkv=2,
                                        D=128, ps=32, seed=3)),
    ("odd heads", Case, dict(rows=[20, 3], held=[0, 30], starts=[0, 20], Hq=15, Hkv=5, D=64, ps=48, w0=1.0, seed=4)),
    ("interleaved", Case, dict(rows=[40, 2], held=[1, 50], starts=[5, 6], Hq=6, Hkv=3, D=64, ps=16, rope_dim=32, inter=True,
                               seed=5)),
    ("wide", Case, dict(rows=[25, 11], held=[0, 5], starts=[0, 25], Hq=4, Hkv=2, D=512, ps=16, rope_dim=128,
                        wdtype=torch.float32, w0=1.0, seed=6)),
    ("wide interleaved", Case, dict(rows=[25, 11], held=[0, 5], starts=[0, 25], Hq=3, Hkv=1, D=512, ps=64, inter=True,
                                    seed=7)),
    ("wide narrow rotation", Case, dict(rows=[9], held=[0], starts=[3], Hq=2, Hkv=1, D=512, ps=16, rope_dim=16, seed=8)),
    ("norm only", Case, dict(rows=[9, 4], held=[0, 1], starts=[0, 0], Hq=4, Hkv=2, D=128, ps=16, rope_dim=0, seed=9)),
    ("rotation only", Case, dict(rows=[9, 4], held=[0, 1], starts=[0, 9], Hq=4, Hkv=2, D=128, ps=16, wdtype=None, seed=10)),
    ("far positions", Case, dict(rows=[5, 1], held=[0, 17], starts=[149_900, 2_000_000_000], Hq=2, Hkv=1, D=64, ps=16,
                                 wdtype=None, seed=11)),
    ("many streams", Case, dict(rows=[i % 3 for i in range(300)], held=[i % 37 for i in range(300)], starts=[9] * 300, Hq=2,
                                Hkv=2, D=64, ps=16, seed=12)),
    ("many rows", Case, dict(rows=[3001, 4000, 2999], held=[0, 0, 5], starts=[0, 0, 0], Hq=3, Hkv=1, D=64, ps=128, seed=13)),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_append_and_read_match_the_oracle(case, bits):
    c = case[1](**case[2], bits=bits)
    q_out = torch.full((c.T, c.Hq, c.D), float("nan"), dtype=BF, device="cuda")
    c.append(q_out)
    k_out, v_out = (torch.full((c.T, c.Hkv, c.D), float("nan"), dtype=BF, device="cuda") for _ in range(2))
    dk.dualkv_cache_read(c.cache, c.d_table, c.d_lens, c.S, c.off, c.Hkv, c.D, k_out, v_out)
    dk.dualkv_check_status()
    w = [None if x is None else _np(x) for x in c.w]
    err = []
    for x, wt in ((c.q, w[0]), (c.k, w[1])):
        n = np.abs(orp.forward(_np(x), wt, c.w0, EPS, c.pos, [], c.inter))
        if c.rope_dim:
            a, b = orp._split(n.copy(), c.rope_dim, c.inter)
            ma, mb = orp._split(n, c.rope_dim, c.inter)
            ma[...] = mb[...] = a + b
        err.append(32 * U * n)
    want_q, want_k = (orp.forward(_np(x), wt, c.w0, EPS, c.pos, _np(c.f), c.inter) for x, wt in ((c.q, w[0]), (c.k, w[1])))
    assert np.all(np.abs(_np(q_out) - want_q) <= 2.0 ** -8 * np.abs(want_q) + err[0])
    page, slot = c.places()
    touched = np.zeros((c.pool, c.ps), dtype=bool)
    touched[page, slot] = True
    if bits == 16:
        assert np.all(np.abs(_np(k_out) - want_k) <= 2.0 ** -8 * np.abs(want_k) + err[1])
        assert torch.equal(v_out, c.v)
        for pool, got in ((c.cache.k, k_out), (c.cache.v, v_out)):
            assert np.array_equal(_np(pool)[page, :, slot], _np(got))
    else:
        v = c.v.float().cpu().numpy()
        step = oc.steps(v)
        assert np.array_equal(_np(c.cache.v_scale)[page, :, slot], step)
        assert np.array_equal(oc.unpack_codes(c.cache.v.cpu().numpy())[page, :, slot], oc.codes(v, step))
        assert np.array_equal(_np(v_out), oc.values(oc.codes(v, step), step))
        codes, ks = oc.unpack_codes(c.cache.k.cpu().numpy())[page, :, slot], _np(c.cache.k_scale)[page, :, slot]
        assert np.array_equal(_np(k_out), oc.values(codes, ks)) and codes.min() >= 1
        group = lambda x: x.reshape(*x.shape[:-1], -1, 32).max(-1)  # noqa: E731
        top, e = group(np.abs(want_k)) / 7, group(err[1]) / 7
        assert np.all(ks >= (top - e) * (1 - U)) and np.all(ks <= (top + e) * (1 + U) * (1 + 1 / 16))
        half = np.repeat(ks, 32, -1) * (0.5 + 16 * U)
        assert np.all(np.abs(_np(k_out) - want_k) <= half + err[1])
        for s in (c.cache.k_scale, c.cache.v_scale):
            assert bool((s.cpu().movedim(1, 2)[torch.from_numpy(~touched)] == 7).all())
    for pool in (c.cache.k, c.cache.v):
        assert bool((pool.cpu().movedim(1, 2)[torch.from_numpy(~touched)] == 7).all())


def test_groups_at_the_ends_of_the_range():
    # zeros, one value, ties at half a step, tiny and large magnitudes, infinities and NaN
    D, T = 64, 8
    v = torch.zeros(T, 1, D)
    v[1, 0, 5] = -3.0
    v[2, 0, :8] = torch.tensor([7.0, 0.5, -0.5, 1.5, -1.5, 6.5, -6.5, 0.4980])
    v[3, 0, :3] = torch.tensor([1e-37, -3e-38, 2e-38])
    v[4, 0, :3] = torch.tensor([9e37, -4e37, 1e37])
    v[5, 0, 3], v[6, 0, 40], v[7, 0, 2] = float("inf"), float("nan"), float("-inf")
    v[5, 0, 32:] = 1.0
    v = v.to(BF).cuda()
    cache = dk.KVCache.empty(1, 1, 16, D, 4)
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    lens, zero = torch.tensor([T], dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    dk.cache_append(v, v, v, cache, table, lens, zero, [0, T])
    k_out, v_out = dk.cache_read(cache, table, lens, [0, T])
    step = oc.steps(v.float().cpu().numpy())
    bad = np.isnan(np.repeat(step, 32, -1))
    want = oc.values(oc.codes(v.float().cpu().numpy(), np.nan_to_num(step)), step)
    for got in (k_out, v_out):
        assert np.array_equal(np.isnan(_np(got)), bad) and np.array_equal(_np(got)[~bad], want[~bad])
    assert bad.sum() == 3 * 32


@pytest.mark.parametrize("bits", [16, 4])
def test_repeats_on_another_stream_and_in_graphs(bits):
    c = Case([40, 0, 3, 200], [0, 4, 30, 0], [0, 40, 40, 40], 8, 2, 128, 32, bits, seed=21)
    q_out = torch.empty(c.T, c.Hq, c.D, dtype=BF, device="cuda")
    outs = [torch.empty(c.T, c.Hkv, c.D, dtype=BF, device="cuda") for _ in range(2)]
    off = dk.offsets(c.off)

    def step():
        c.append(q_out)
        dk.dualkv_cache_read(c.cache, c.d_table, c.d_lens, c.S, off, c.Hkv, c.D, *outs)

    step()
    want = [t.clone() for t in (q_out, *outs)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _fill(c.cache, 7)
        step()
    side.synchronize()
    for a, b in zip(want, (q_out, *outs)):
        assert torch.equal(a, b)
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for g in graphs + graphs:
        _fill(c.cache, 7)
        q_out.zero_()
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, (q_out, *outs)):
            assert torch.equal(a, b)


def test_pages_that_do_not_exist_are_reported_and_left():
    c = Case([3, 2, 4, 1], [14, 0, 16, 0], [0] * 4, 2, 1, 64, 16, 16, seed=22)
    c.d_table[0, 1] = c.pool  # tokens 16 of stream 0
    c.d_table[1, 0] = -1
    c.d_lens[2] = 3           # fewer than the call's rows
    q_out = torch.empty(c.T, c.Hq, c.D, dtype=BF, device="cuda")
    c.append(q_out)
    with pytest.raises(dk.DualKVError):
        dk.dualkv_check_status()
    k_out, v_out = dk.cache_read(c.cache, c.d_table, c.d_lens, c.off)
    with pytest.raises(dk.DualKVError):
        dk.dualkv_check_status()
    # row 2 is token 16 of stream 0, rows 3 and 4 are stream 1's; stream 2 is said to hold fewer than its four rows
    assert torch.equal(v_out[:2], c.v[:2]) and torch.equal(v_out[9], c.v[9])
    assert bool((v_out[2:9] == 0).all())
    c.d_lens[2] = 1000        # beyond the table
    c.append(q_out)
    with pytest.raises(dk.DualKVError):
        dk.dualkv_check_status()


def test_pools_past_32_bit_offsets():
    # 2.2 G values a pool: the last pages lie beyond 2^31 values and 2^32 bytes
    ps, Hkv, D, pool = 64, 8, 128, 33_000
    cache = dk.KVCache.empty(pool, Hkv, ps, D)
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(100, 3 * Hkv, D, generator=g, device="cuda").to(BF)
    q, k, v = x[:, :Hkv], x[:, Hkv:2 * Hkv], x[:, 2 * Hkv:]
    table = torch.tensor([[pool - 1, 5, pool - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([130], dtype=torch.int32, device="cuda")
    cache.k[pool - 1], cache.k[pool - 2], cache.k[5] = 7, 7, 7
    q_out = dk.cache_append(q, k, v, cache, table, lens, torch.zeros_like(lens), [0, 100])
    assert torch.equal(q_out, q)
    kk, vv = dk.cache_read(cache, table, lens, [0, 100])
    assert torch.equal(kk, k) and torch.equal(vv, v)
    assert torch.equal(cache.k[pool - 1, :, 30:].transpose(0, 1), k[:34]) and bool((cache.k[pool - 1, :, :30] == 7).all())
    assert bool((cache.k[pool - 2, :, 2:] == 7).all())
    dk.dualkv_check_status()


def test_binding_refuses_what_does_not_fit():
    c = Case([3, 2], [0, 0], [0, 0], 2, 1, 64, 16, 16, seed=23)
    q_out = torch.empty(c.T, c.Hq, c.D, dtype=BF, device="cuda")

    def call(**kw):
        a = dict(q=c.q, k=c.k, v=c.v, qw=c.w[0], kw=c.w[1], f=c.f, rd=c.rope_dim, cache=c.cache, table=c.d_table, lens=c.d_lens,
                 starts=c.d_starts, S=c.S, off=c.off, Hkv=c.Hkv, q_out=q_out)
        a.update(kw)
        dk.dualkv_cache_append(a["q"], a["k"], a["v"], a["qw"], a["kw"], 0.0, EPS, a["f"], a["rd"], False, a["cache"],
                               a["table"], a["lens"], a["starts"], a["S"], a["off"], c.Hq, a["Hkv"], c.D, a["q_out"])

    call()
    other = dk.KVCache.empty(2, 2, 16, 64)
    for bad in (dict(q=c.q[:-1]), dict(q=c.q.float()), dict(v=c.v.cpu()), dict(kw=None), dict(f=c.f[:-1]), dict(cache=other),
                dict(cache=None), dict(table=c.d_table.long()), dict(table=c.d_table[:1]), dict(table=c.d_table[0]),
                dict(lens=c.d_lens.long()), dict(starts=c.d_starts[:1]), dict(S=3), dict(off=[0, 3, 1 << 33]),
                dict(q_out=q_out.float()), dict(table=c.d_table.cpu())):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q_out=c.q if c.q.is_contiguous() else c.cache.k.view(-1)[:q_out.numel()].view(q_out.shape)),
                dict(off=[0, 3, 2], q=c.q[:2], k=c.k[:2], v=c.v[:2], q_out=q_out[:2])):
        with pytest.raises(dk.DualKVError):
            call(**bad)
    k, v = c.cache.k, c.cache.v
    codes, sc = torch.zeros(2, 1, 16, 32, dtype=torch.uint8, device="cuda"), torch.zeros(2, 1, 16, 2, dtype=BF, device="cuda")
    for bad in ((k, v, sc, sc), (k, v[:1]), (k, v.float()), (codes, codes), (codes, codes, sc), (codes, codes, sc, sc.float()),
                (codes, codes, sc, sc[..., :1]), (k.transpose(1, 2), v.transpose(1, 2)) if c.Hkv > 1 else (k[..., ::2], v[..., ::2])):
        with pytest.raises(ValueError):
            dk.KVCache(*bad)
    assert dk.KVCache(codes, codes, sc, sc).bits == 4 and isinstance(c.cache._c, ctypes.Structure)
    dk.dualkv_check_status()
