"""GPU parity of dualkv_decode against ``oracle.cache.attend`` (fp64) on the values that the cache holds.

Tolerances, with u = 2^-24 and for one output value: A = sum p |v|, X = largest scale sum |q| |k| of its head:
  d = (4 D + 32) u X   error of a log-weight: D products summed in fp32, twice half a step per addition (the matrix
                       instructions may cut off instead of rounding), the scaling and the subtraction of the maximum
  out  2^-8 |out| for its rounding, 2^-8 A for the weights' rounding to bf16, (2 d + 2^-20) A for the weights
       before it and their sum (base-2 exponentials are good to 2^-22, sums of positive terms to 2^-21 here)
  lse  d + 2^-20 + 4 u |lse|
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


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _np(t):
    return t.detach().double().cpu().numpy()


class Case:
    """Random prompts and responses in one pool; what no query sees holds NaN."""

    def __init__(self, groups, prompts, lens, Hq, Hkv, D, ps, bits, window=0, seed=0, spread=1.0, strided=False, table_extra=0):
        self.groups, self.prompts, self.lens = groups, prompts, lens
        self.Hq, self.Hkv, self.D, self.ps, self.bits, self.window = Hq, Hkv, D, ps, bits, window
        self.G, self.B, self.scale = len(prompts), len(lens), D ** -0.5
        need = [[-(-max(n, 0) // ps) for n in ns] for ns in (prompts, lens)]
        pool = sum(map(sum, need)) + 3
        order = np.random.default_rng(seed).permutation(pool)
        self.tables, at = [], 0
        for counts in need:
            t = np.full((len(counts), max(counts + [1]) + table_extra), -1, dtype=np.int32)
            for i, k in enumerate(counts):
                t[i, :k] = order[at:at + k]
                at += k
            self.tables.append(t)
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        x = [spread * rn(pool, Hkv, ps, D) for _ in range(2)]
        if bits == 16:
            self.cache = dk.KVCache(*(t.to(BF) for t in x))
        else:
            scale = [(0.01 + 0.4 * torch.rand(pool, Hkv, ps, D // 32, generator=g, device="cuda")).to(BF) for _ in range(2)]
            for s in scale:  # five significant bits, as append writes them
                s.copy_((s.view(torch.int16) & ~7).view(BF))
            # codes 0 to 15: all that a code can hold
            codes = [torch.randint(0, 256, (pool, Hkv, ps, D // 2), generator=g, device="cuda", dtype=torch.uint8)
                     for _ in range(2)]
            self.cache = dk.KVCache(*codes, *scale)
        self._spoil()
        q = rn(self.B, Hq * D + (64 if strided else 0)).to(BF)
        self.q = q[:, :Hq * D].view(self.B, Hq, D) if strided else q.view(self.B, Hq, D)
        for b, n in enumerate(lens):  # nothing of a response that has ended is used
            if n < 0:
                self.q[b] = float("nan")
        i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
        self.d_tables = [torch.from_numpy(t).cuda() for t in self.tables]
        self.d_prompts, self.d_lens = i32(prompts), i32(lens)
        self.pools = [_np(self.cache.k), _np(self.cache.v)] if bits == 16 else [
            oc.values(oc.unpack_codes(c.cpu().numpy()), _np(s)) for c, s in ((self.cache.k, self.cache.k_scale),
                                                                             (self.cache.v, self.cache.v_scale))]

    def first_seen(self, b):
        """First position that response b sees."""
        P = self.prompts[self.group(b)]
        return max(0, P + self.lens[b] - self.window) if self.window > 0 else 0

    def group(self, b):
        return int(np.searchsorted(self.groups, b, side="right")) - 1

    def _spoil(self):
        """NaN wherever no query of the call looks (in 4 bits: in the scales)."""
        seen = np.zeros((self.cache.pages, self.ps), dtype=bool)
        for b in range(self.B):
            g, n = self.group(b), self.lens[b]
            if n < 0:
                continue
            lo, P = self.first_seen(b), self.prompts[g]
            for table, i in ((self.tables[0][g], np.arange(lo, P)), (self.tables[1][b], np.arange(max(0, lo - P), n))):
                seen[table[i // self.ps], i % self.ps] = True
        mask = torch.from_numpy(~seen).cuda()[:, None, :, None]
        for t in ((self.cache.k, self.cache.v) if self.bits == 16 else (self.cache.k_scale, self.cache.v_scale)):
            t.masked_fill_(mask, float("nan"))

    def run(self, out=None, lse=None, **kw):
        return dk.decode(self.q, self.cache, self.d_tables[0], self.d_prompts, self.d_tables[1], self.d_lens, self.groups,
                         self.window, **kw)

    def check(self, out, lse, only=None):
        out, lse, q = _np(out), _np(lse), _np(self.q)
        for b in range(self.B) if only is None else only:
            g, n = self.group(b), self.lens[b]
            if n < 0:
                assert not out[b].any() and np.all(lse[:, b] == -np.inf)
                continue
            lo, P = self.first_seen(b), self.prompts[g]
            i = (np.arange(lo, P), np.arange(max(0, lo - P), n))
            k, v = (np.concatenate([x[t[j // self.ps], :, j % self.ps] for t, j in zip((self.tables[0][g], self.tables[1][b]), i)])
                    for x in self.pools)
            want, want_lse, A, X = oc.attend(q[b], k, v, self.scale, P + n - 1, (i[0], P + i[1]), self.window)
            d = (4 * self.D + 32) * U * X
            tol = 2.0 ** -8 * (np.abs(want) + A) + (2 * d[:, None] + 2.0 ** -20) * A
            assert np.all(np.abs(out[b] - want) <= tol), (b, float(np.max(np.abs(out[b] - want) - tol)))
            empty = np.isneginf(want_lse)
            assert np.array_equal(np.isneginf(lse[:, b]), empty)
            e = np.abs(lse[~empty, b] - want_lse[~empty])
            assert np.all(e <= (d + 2.0 ** -20 + 4 * U * np.abs(np.where(empty, 0, want_lse)))[~empty]), (b, e.max())


def _ragged(n, lo, hi, seed):
    return np.random.default_rng(seed).integers(lo, hi + 1, n).tolist()


CASES = [
    ("one token", dict(groups=[0, 1], prompts=[0], lens=[1], Hq=1, Hkv=1, D=64, ps=16)),
    ("prompt alone", dict(groups=[0, 2], prompts=[5], lens=[0, 0], Hq=2, Hkv=1, D=64, ps=16)),
    ("nothing seen", dict(groups=[0, 3, 3, 4], prompts=[0, 9, 1], lens=[0, -1, 2, -1], Hq=4, Hkv=2, D=128, ps=16)),
    ("edges of pages", dict(groups=[0, 8], prompts=[33], lens=[1, 15, 16, 17, 31, 32, 33, 64], Hq=4, Hkv=2, D=128, ps=16,
                            seed=1)),
    ("groups", dict(groups=[0, 3, 3, 8, 9], prompts=[130, 40, 1, 300], lens=[7, 200, -1, 64, 0, 1, 90, 33, 129], Hq=8, Hkv=2,
                    D=128, ps=32, seed=2)),
    ("seven to one", dict(groups=[0, 11, 22], prompts=[99, 260], lens=_ragged(22, 0, 150, 3), Hq=21, Hkv=3, D=64, ps=16, seed=3)),
    ("five to one, odd pages", dict(groups=[0, 2, 5], prompts=[97, 20], lens=[7, 95, 96, 97, 30], Hq=5, Hkv=1, D=128, ps=48,
                                    seed=4, strided=True)),
    ("sixteen to one", dict(groups=[0, 4], prompts=[70], lens=[5, 1, 33, 80], Hq=32, Hkv=2, D=128, ps=16, seed=5)),
    ("forty to one", dict(groups=[0, 3], prompts=[50], lens=[5, 1, 33], Hq=40, Hkv=1, D=64, ps=16, seed=6)),
    ("wide", dict(groups=[0, 3, 5], prompts=[70, 3], lens=[40, 1, 17, 100, 0], Hq=8, Hkv=2, D=512, ps=16, seed=7)),
    ("wide sixteen to one", dict(groups=[0, 3], prompts=[40], lens=[20, 1, 17], Hq=16, Hkv=1, D=512, ps=32, seed=8)),
    ("one head each", dict(groups=[0, 5], prompts=[200], lens=[100, 20, 3, 64, 65], Hq=3, Hkv=3, D=64, ps=128, seed=9)),
    ("large group", dict(groups=[0, 70], prompts=[333], lens=_ragged(70, 0, 60, 10), Hq=8, Hkv=2, D=128, ps=64, seed=10)),
    ("two large groups", dict(groups=[0, 40, 75], prompts=[513, 128], lens=_ragged(75, 0, 200, 11), Hq=16, Hkv=2, D=64, ps=32,
                              seed=11)),
    ("large group, wide", dict(groups=[0, 20], prompts=[200], lens=_ragged(20, 0, 40, 12), Hq=16, Hkv=2, D=512, ps=16, seed=12)),
    ("large values", dict(groups=[0, 4], prompts=[100], lens=[50, 3, 20, 90], Hq=4, Hkv=1, D=128, ps=16, seed=13, spread=6.0)),
    ("longer tables", dict(groups=[0, 4], prompts=[100], lens=[50, 3, 20, 90], Hq=4, Hkv=1, D=128, ps=16, seed=14,
                           table_extra=5)),
]


@pytest.mark.parametrize("window", [0, 1, 37, 100])
@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_matches_the_oracle(case, bits, window):
    c = Case(**case[1], bits=bits, window=window)
    out, lse = c.run()
    dk.dualkv_check_status()
    c.check(out, lse)


LONG = [
    ("one long response", dict(groups=[0, 1], prompts=[0], lens=[20_011], Hq=8, Hkv=2, D=128, ps=64)),
    ("long prompt, short responses", dict(groups=[0, 9], prompts=[9_001], lens=[1, 0, 3, -1, 50, 7, 7, 7, 12], Hq=16, Hkv=4,
                                          D=64, ps=32)),
    ("window over a long prompt", dict(groups=[0, 40], prompts=[5_000], lens=_ragged(40, 0, 1500, 5), Hq=4, Hkv=1, D=128,
                                       ps=16, window=1024)),
    ("large group over a long prompt", dict(groups=[0, 64], prompts=[6_000], lens=_ragged(64, 0, 100, 6), Hq=8, Hkv=2, D=128,
                                            ps=128)),
    ("many short responses", dict(groups=list(range(0, 1201, 2)), prompts=_ragged(600, 0, 30, 7), lens=_ragged(1200, -1, 40, 8),
                                  Hq=2, Hkv=1, D=64, ps=16)),
    ("prompt by the block kernel", dict(groups=[0, 40, 41], prompts=[7_001, 130], lens=_ragged(41, -1, 300, 13), Hq=32, Hkv=8,
                                        D=128, ps=64)),
    ("its rows in several blocks", dict(groups=[0, 60, 75, 80], prompts=[3_003, 2_050, 4_000], lens=_ragged(80, 0, 200, 14), Hq=21,
                                        Hkv=3, D=64, ps=48)),
    ("block kernel under a window", dict(groups=[0, 50, 90], prompts=[6_000, 5_555], lens=_ragged(90, 0, 1400, 15), Hq=32, Hkv=8,
                                         D=64, ps=16, window=1300)),
    ("wide and long", dict(groups=[0, 8], prompts=[3_000], lens=_ragged(8, 0, 900, 9), Hq=8, Hkv=2, D=512, ps=64)),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("case", LONG, ids=[c[0] for c in LONG])
def test_long_streams(case, bits):
    c = Case(**case[1], bits=bits, seed=31)
    out, lse = c.run()
    dk.dualkv_check_status()
    c.check(out, lse, only=range(0, c.B, max(1, c.B // 40)))


PIECES = [  # prompts of large groups, whose tiles are dealt by prompt, kv-head and block of 128 rows
    ("a few, with a rest", dict(groups=[0, 32, 64, 96, 128, 160], prompts=[129, 4_097, 0, 7_000, 5_000],
                                lens=_ragged(64, 0, 40, 16) + [-1] * 32 + _ragged(64, -1, 40, 17), Hq=8, Hkv=2, D=64, ps=16)),
    ("nobody left of the longest", dict(groups=[0, 40, 80], prompts=[9_000, 8_321], lens=[-1] * 40 + _ragged(40, 0, 40, 18),
                                        Hq=32, Hkv=8, D=128, ps=64)),
    ("more of them than blocks", dict(groups=list(range(0, 2881, 32)), prompts=_ragged(90, 100, 700, 19),
                                      lens=_ragged(2880, -1, 20, 20), Hq=8, Hkv=2, D=64, ps=16)),
    ("more prompts than blocks", dict(groups=list(range(0, 4001, 20)), prompts=_ragged(200, 400, 800, 21),
                                      lens=_ragged(4000, -1, 12, 22), Hq=2, Hkv=1, D=64, ps=16)),
    ("one and a half to a block", dict(groups=[0, 64, 128], prompts=[4_000, 4_000], lens=_ragged(128, 0, 20, 23), Hq=64, Hkv=8,
                                       D=64, ps=32)),
]


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("case", PIECES, ids=[c[0] for c in PIECES])
def test_prompts_dealt_in_pieces(case, bits):
    c = Case(**case[1], bits=bits, seed=32)
    out, lse = c.run()
    dk.dualkv_check_status()
    c.check(out, lse, only=range(0, c.B, max(1, c.B // 40)))


@pytest.mark.parametrize("seed", range(24))
def test_random_layouts(seed):
    r = np.random.default_rng(1000 + seed)
    G, Hkv, D = int(r.integers(1, 6)), int(r.choice([1, 2, 3])), int(r.choice([64, 128, 512]))
    sizes = r.integers(0, int(r.choice([3, 12, 70])), G)
    if not sizes.sum():
        sizes[0] = 1
    most = int(r.choice([20, 150, 700]))
    c = Case([0] + np.cumsum(sizes).tolist(), r.integers(0, most, G).tolist(), r.integers(-1, most, sizes.sum()).tolist(),
             Hkv * int(r.choice([1, 2, 4, 7, 8, 12, 16])), Hkv, D, int(r.choice([16, 32, 48, 64, 128])), int(r.choice([16, 4])),
             int(r.choice([0, 0, 64, r.integers(1, 500)])), seed, strided=bool(r.integers(0, 2)))
    out, lse = c.run()
    dk.dualkv_check_status()
    c.check(out, lse)


def test_repeats_bit_for_bit_on_another_stream_and_in_graphs():
    c = Case([0, 20, 33], [700, 90], _ragged(33, 0, 300, 40), 8, 2, 128, 16, 4, seed=41)
    want = c.run()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = c.run(stream=side)
    side.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    # two graphs that share outputs and workspace; between replays the responses grow
    ws = torch.empty(dk.dualkv_decode_workspace_bytes(c.G, c.groups, c.Hq, c.Hkv, c.D), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    groups = dk.offsets(c.groups)

    def step():
        dk.dualkv_decode(c.q, c.cache, c.d_tables[0], c.d_prompts, c.d_tables[1], c.d_lens, c.G, groups, c.Hq, c.Hkv, c.D,
                         c.scale, 0, out, lse, ws)

    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            step()
    for g in graphs + graphs:
        out.zero_()
        ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(want[0], out) and torch.equal(want[1], lse)
    short = [max(n - 5, -1) for n in c.lens]
    c.d_lens.copy_(torch.tensor(short, dtype=torch.int32))
    graphs[0].replay()
    torch.cuda.synchronize()
    c.lens = short
    c.check(out, lse)


@pytest.mark.parametrize("bits,D", [(16, 128), (4, 64), (16, 512)])
def test_the_most_sources(bits, D):
    # as many groups and responses as a call takes: their lengths leave room for fewer warps
    sizes = np.array([2] * 4094 + [4])
    r = np.random.default_rng(70)
    c = Case([0] + np.cumsum(sizes).tolist(), r.integers(0, 4, 4095).tolist(), r.integers(-1, 6, 8192).tolist(), 2, 1, D, 16, bits,
             seed=71)
    out, lse = c.run()
    dk.dualkv_check_status()
    c.check(out, lse, only=list(range(0, 8192, 97)) + [8191])


def test_two_streams_at_once():
    # two batches with prompts for the block kernel, each with its own workspace, on two streams in turn: their kernels share
    # the GPU in any order
    cases = [Case([0, 40], [6000], _ragged(40, 0, 200, 80 + i), 32, 8, 128, 64, bits, seed=80 + i) for i, bits in enumerate((16, 4))]
    want = [c.run() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = []
    for _ in range(12):
        for c, s in zip(cases, streams):
            got.append(c.run(stream=s))
    torch.cuda.synchronize()
    dk.dualkv_check_status()
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i % 2][0]) and torch.equal(lse, want[i % 2][1])


def test_in_graphs_behind_copies_and_other_kernels():
    # the calls' kernels may start before what is in front of them is done: copies, fills and other kernels whose results
    # they need, in a captured graph and out of it
    c = Case([0, 16], [900], _ragged(16, 1, 300, 42), 8, 2, 128, 32, 16, seed=43)
    big = Case([0, 32], [3000], _ragged(32, 1, 300, 44), 32, 8, 128, 64, 16, seed=45)
    for x in (c, big):
        want, want_lse = x.run()
        lens, q = x.d_lens.clone(), x.q.clone()
        ws = torch.empty(dk.dualkv_decode_workspace_bytes(x.G, x.groups, x.Hq, x.Hkv, x.D), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(want), torch.empty_like(want_lse)
        big_fill = torch.empty(1 << 26, device="cuda")

        def step():
            big_fill.fill_(1.0)      # takes long enough that a kernel that did not wait would be caught
            x.d_lens.copy_(lens)
            x.q.copy_(q)
            dk.dualkv_decode(x.q, x.cache, x.d_tables[0], x.d_prompts, x.d_tables[1], x.d_lens, x.G, x.groups, x.Hq, x.Hkv, x.D,
                             x.scale, 0, out, lse, ws)
            x.q.zero_()              # and what comes behind waits for them
            x.d_lens.fill_(-1)

        step()
        torch.cuda.synchronize()
        assert torch.equal(want, out) and torch.equal(want_lse, lse)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(want, out) and torch.equal(want_lse, lse)
    dk.dualkv_check_status()


def test_lengths_beyond_the_tables_and_pages_that_do_not_exist():
    c = Case([0, 4], [40], [30, 20, 10, 50], 4, 2, 64, 16, 16, seed=50)
    out, lse = c.run()
    dk.dualkv_check_status()
    # a response longer than its table, a page outside the pool: reported; the others keep their results
    c.d_lens[0] = 10_000
    c.d_tables[1][1, 1] = 1 << 30
    bad_out, bad_lse = c.run()
    with pytest.raises(dk.DualKVError):
        dk.dualkv_check_status()
    for b in (2, 3):
        assert torch.equal(bad_out[b], out[b]) and torch.equal(bad_lse[:, b], lse[:, b])
    # response 1 as if its tokens 16 .. 19 were not there, in place of counting what lies elsewhere
    assert bool(torch.isfinite(bad_out[1]).all()) and bool((bad_lse[:, 1] <= lse[:, 1]).all())


@pytest.mark.parametrize("bits", [16, 4])
def test_pools_past_32_bit_offsets(bits):
    # pages at both ends of a pool of 2.4 G values, the last ones beyond 2^31 values (4 bits: 2^30 bytes of codes); the
    # same tokens in a small pool give the same bits
    ps, Hkv, Hq, D = 64, 8, 32, 128
    c = Case([0, 2, 40], [300, 4000], _ragged(40, 0, 200, 60), Hq, Hkv, D, ps, bits, seed=61)
    want, want_lse = c.run()
    pool = 37_000
    far = dk.KVCache.empty(pool, Hkv, ps, D, bits)
    move = torch.arange(c.cache.pages, device="cuda") * 3
    move[::2] = pool - 1 - move[::2]
    pairs = [(far.k, c.cache.k), (far.v, c.cache.v)]
    if bits == 4:
        pairs += [(far.k_scale, c.cache.k_scale), (far.v_scale, c.cache.v_scale)]
    for a, b in pairs:
        a[move] = b
    tables = [torch.where(t >= 0, move[t.long().clamp(min=0)], -1).to(torch.int32) for t in c.d_tables]
    out, lse = dk.decode(c.q, far, tables[0], c.d_prompts, tables[1], c.d_lens, c.groups)
    dk.dualkv_check_status()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)


def test_without_prompts_and_without_lse():
    c = Case([0, 1, 2, 3], [0, 0, 0], [30, 0, 77], 4, 2, 64, 16, 16, seed=51)
    want, want_lse = c.run()
    c.check(want, want_lse)
    out, lse = dk.decode(c.q, c.cache, None, None, c.d_tables[1], c.d_lens, c.groups)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    out.zero_()
    ws = torch.empty(dk.dualkv_decode_workspace_bytes(c.G, c.groups, c.Hq, c.Hkv, c.D), dtype=torch.uint8, device="cuda")
    dk.dualkv_decode(c.q, c.cache, None, None, c.d_tables[1], c.d_lens, c.G, c.groups, c.Hq, c.Hkv, c.D, c.scale, 0, out, None,
                     ws)
    assert torch.equal(out, want)
    dk.dualkv_check_status()


def test_binding_refuses_what_does_not_fit():
    c = Case([0, 2], [20], [3, 4], 4, 2, 64, 16, 16, seed=52)
    ws = torch.empty(dk.dualkv_decode_workspace_bytes(1, c.groups, 4, 2, 64), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty(4, 2, device="cuda")

    def call(**kw):
        a = dict(q=c.q, cache=c.cache, pp=c.d_tables[0], pl=c.d_prompts, pages=c.d_tables[1], lens=c.d_lens, G=1, groups=c.groups,
                 Hq=4, out=out, lse=lse, ws=ws, wsb=None)
        a.update(kw)
        dk.dualkv_decode(a["q"], a["cache"], a["pp"], a["pl"], a["pages"], a["lens"], a["G"], a["groups"], a["Hq"], 2, 64, 0.125, 0,
                         a["out"], a["lse"], a["ws"], a["wsb"])

    call()
    for bad in (dict(q=c.q.float()), dict(q=c.q[:1]), dict(q=c.q.cpu()), dict(pp=None), dict(pl=None), dict(pl=c.d_prompts.long()),
                dict(pp=c.d_tables[1]), dict(pages=c.d_tables[1].long()), dict(lens=c.d_lens[:1]), dict(groups=[0, 3]), dict(G=2),
                dict(Hq=8), dict(out=out.float()), dict(lse=lse[:1]), dict(lse=lse.t()), dict(ws=ws.cpu()),
                dict(wsb=ws.numel() + 1), dict(cache=dk.KVCache.empty(2, 1, 16, 64))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(out=c.q), dict(ws=None), dict(wsb=16)):
        with pytest.raises(dk.DualKVError):
            call(**bad)
    dk.dualkv_check_status()
