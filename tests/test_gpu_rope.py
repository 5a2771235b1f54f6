"""GPU parity of dualkv_qk_norm_rope and its backward against ``oracle.rope`` (fp64).

Tolerances, with u = 2^-24 (half an fp32 step) and y one output value:
  forward   2^-8 |y| for the rounding to bf16, plus 32 u (|n_a| + |n_b|) for the fp32
            arithmetic on its pair: the sum of D squares loses at most 22 u and its root
            half of that, rsqrtf 4 u, w + w0 and the two products 3 u, a cosine or sine
            6 u (3.2 u from the angle, 2 u from the function), the rotation 3 u.
  dq, dk    2^-8 |dx| plus 100 u S, S = r (m |w| + |x r| mean(m |w x r|)) with m = |dy_a| + |dy_b|
            bounding the turned-back gradient: the same terms, r and the rotation twice.
  dweight   (heads per lane + 64) u sum m |x r|: sequential sums over a lane's heads, then trees.
"""
import numpy as np
import pytest
import torch

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


def _inv_freq(rope_dim, base):
    return (base ** (-2.0 * torch.arange(rope_dim // 2, dtype=torch.float64) / max(rope_dim, 1))).float().cuda()


def _inputs(P, off, Hq, Hkv, D, rope_dim, wdtype, fused, seed, base=1e4):
    g = torch.Generator(device="cuda").manual_seed(seed)
    T = P + off[-1]
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    if fused:
        row = rn(T, (Hq + 2 * Hkv) * D + 8)
        q, k = row[:, :Hq * D].view(T, Hq, D), row[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    else:
        q, k = rn(T, Hq, D), rn(T, Hkv, D)
    w = [None, None]
    if wdtype is not None:
        w = [(0.3 * torch.randn(D, generator=g, device="cuda") + 1).to(wdtype) for _ in range(2)]
    return q, k, w[0], w[1], _inv_freq(rope_dim, base), rn(T, Hq, D), rn(T, Hkv, D)


def _pair_abs(x, rope_dim, inter):
    """|a| + |b| of each value's pair (its own magnitude where it is not turned)."""
    m = np.abs(x)
    if rope_dim:
        a, b = orp._split(m.copy(), rope_dim, inter)
        ma, mb = orp._split(m, rope_dim, inter)
        ma[...] = mb[...] = a + b
    return m


def _check_forward(y, x, w, w0, pos, f, inter):
    want = orp.forward(x, w, w0, EPS, pos, f, inter)
    n = orp.forward(x, w, w0, EPS, pos, [], inter)
    tol = 2.0 ** -8 * np.abs(want) + 32 * U * _pair_abs(n, 2 * len(f), inter)
    err = np.abs(y - want)
    assert np.all(err <= tol), float(np.max(err - tol))


def _check_backward(dx, dw, x, dy, w, w0, pos, f, inter):
    want, want_w = orp.backward(x, dy, w, w0, EPS, pos, f, inter)
    m = _pair_abs(dy, 2 * len(f), inter)
    if w is None:
        tol = 2.0 ** -8 * np.abs(want) + 32 * U * m
    else:
        r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + EPS)
        aw, xh = np.abs(w + w0), np.abs(x * r)
        tol = 2.0 ** -8 * np.abs(want) + 100 * U * r * (m * aw + xh * np.mean(m * aw * xh, -1, keepdims=True))
        err = np.abs(dw - want_w)
        assert np.all(err <= (x.shape[1] + 64) * U * (m * xh).sum((0, 1))), float(err.max())
    err = np.abs(dx - want)
    assert np.all(err <= tol), float(np.max(err - tol))


CASES = [
    # name, P, offsets, Hq, Hkv, D, rope_dim, interleaved, weight dtype, weight offset, fused rows
    ("one-row", 1, [0, 0], 1, 1, 64, 64, False, torch.float32, 0.0, False),
    ("one-response-row", 0, [0, 1], 3, 1, 128, 128, False, BF, 0.0, False),
    ("ragged", 37, [0, 5, 5, 19, 20, 44], 4, 2, 128, 128, False, BF, 0.0, True),
    ("odd-heads", 9, [0, 3, 3, 20], 5, 5, 64, 64, False, torch.float32, 0.0, True),
    ("seven-to-one", 9, [0, 30], 7, 1, 128, 64, False, torch.float32, 1.0, True),
    ("interleaved", 20, [0, 11, 12], 6, 3, 64, 32, True, BF, 1.0, True),
    ("interleaved-full", 20, [0, 11, 12], 2, 1, 512, 512, True, BF, 0.0, False),
    ("wide", 33, [0, 17, 40], 4, 2, 512, 128, False, torch.float32, 1.0, True),
    ("wide-16", 33, [0, 17, 40], 3, 1, 512, 16, False, BF, 0.0, False),
    ("norm-only", 8, [0, 9], 4, 2, 128, 0, False, BF, 0.0, False),
    ("rotation-only", 8, [0, 9, 30], 4, 2, 128, 128, False, None, 0.0, True),
    ("rotation-only-part", 8, [0, 9, 30], 3, 3, 64, 48, True, None, 0.0, False),
    ("many-segments", 3, [0] + np.cumsum(np.arange(300) % 3).tolist(), 2, 2, 64, 64, False, BF, 0.0, False),
    ("most-segments", 2, [0] + np.cumsum(np.arange(4095) % 2).tolist(), 2, 1, 64, 32, True, torch.float32, 0.0, True),
    ("many-rows", 3001, [0, 4000, 9001], 3, 1, 64, 64, False, BF, 0.0, False),
]


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_matches_the_oracle(case):
    name, P, off, Hq, Hkv, D, rope_dim, inter, wdtype, w0, fused = case
    N = len(off) - 1
    q, k, qw, kw, f, dq_out, dk_out = _inputs(P, off, Hq, Hkv, D, rope_dim, wdtype, fused, 100 + D + Hq)
    T = P + off[-1]
    pos, fn = orp.positions(P, off), _np(f)
    q_out, k_out = (torch.full((T, H, D), float("nan"), dtype=BF, device="cuda") for H in (Hq, Hkv))
    dk.dualkv_qk_norm_rope(q, k, qw, kw, w0, EPS, f, rope_dim, inter, P, N, off, Hq, Hkv, D, q_out, k_out)
    # gradients into columns of one fused buffer whose other columns have to stay as they are
    row = torch.full((T, (Hq + 2 * Hkv) * D + 8), 7.0, dtype=BF, device="cuda")
    dq, dkk = row[:, :Hq * D].view(T, Hq, D), row[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)
    dw = [None, None] if qw is None else [torch.full((D,), float("nan"), device="cuda") for _ in range(2)]
    ws = torch.empty(dk.dualkv_qk_norm_rope_bwd_workspace_bytes(P, N, off, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    dk.dualkv_qk_norm_rope_bwd(q, k, dq_out, dk_out, qw, kw, w0, EPS, f, rope_dim, inter, P, N, off, Hq, Hkv, D, dq, dkk,
                               dw[0], dw[1], ws)
    torch.cuda.synchronize()
    assert bool((row[:, (Hq + Hkv) * D:] == 7.0).all())
    for y, x, w, dy, dx, g in ((q_out, q, qw, dq_out, dq, dw[0]), (k_out, k, kw, dk_out, dkk, dw[1])):
        wn = None if w is None else _np(w)
        _check_forward(_np(y), _np(x), wn, w0, pos, fn, inter)
        _check_backward(_np(dx), None if g is None else _np(g), _np(x), _np(dy), wn, w0, pos, fn, inter)


def test_far_positions_keep_their_angles():
    # positions up to 150,000 with frequencies up to 1: an angle formed in fp32 would be 0.008 off
    P, off = 149_900, [0, 50, 101]
    q, k, _, _, f, _, _ = _inputs(P, off, 1, 1, 64, 64, None, False, 5)
    q_out, k_out = dk.qk_norm_rope(q, k, P, off, f)
    pos = orp.positions(P, off)
    _check_forward(_np(q_out), _np(q), None, 0.0, pos, _np(f), False)
    _check_forward(_np(k_out), _np(k), None, 0.0, pos, _np(f), False)


def test_zero_row_and_gradient():
    # a head of zeros has no direction: eps keeps its norm finite, its output is 0
    P, off = 4, [0, 3]
    q, k, qw, kw, f, dq_out, dk_out = _inputs(P, off, 2, 1, 64, 64, BF, False, 6)
    q[2] = 0.0
    q_out, _ = dk.qk_norm_rope(q, k, P, off, f, qw, kw, eps=EPS)
    dq, _, _, _ = dk.qk_norm_rope_backward(q, k, dq_out, dk_out, P, off, f, qw, kw, eps=EPS)
    assert bool((q_out[2] == 0).all()) and bool(torch.isfinite(dq).all())


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    P, off, Hq, Hkv, D = 500, [0, 700, 1300], 4, 2, 128
    N, T = len(off) - 1, P + off[-1]
    q, k, qw, kw, f, dq_out, dk_out = _inputs(P, off, Hq, Hkv, D, D, torch.float32, True, 9)
    want = dk.qk_norm_rope(q, k, P, off, f, qw, kw) + dk.qk_norm_rope_backward(q, k, dq_out, dk_out, P, off, f, qw, kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = (dk.qk_norm_rope(q, k, P, off, f, qw, kw, stream=side)
           + dk.qk_norm_rope_backward(q, k, dq_out, dk_out, P, off, f, qw, kw, stream=side))
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    # two graphs that share buffers and workspace, replayed one after the other
    outs = [torch.zeros_like(t) for t in want]
    ws = torch.empty(dk.dualkv_qk_norm_rope_bwd_workspace_bytes(P, N, off, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    c_off = dk.offsets(off)

    def step(scale):
        dk.dualkv_qk_norm_rope(q, k, qw, kw, 0.0, 1e-6, f, D, False, P, N, c_off, Hq, Hkv, D, outs[0], outs[1])
        dk.dualkv_qk_norm_rope_bwd(q, k, dq_out, dk_out, qw, kw, 0.0, 1e-6, f, D, False, P, N, c_off, Hq, Hkv, D, outs[2],
                                   outs[3], outs[4], outs[5], ws)

    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, graph in enumerate(graphs):
        with torch.cuda.graph(graph):
            step(i)
    for graph in graphs + graphs:
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_rows_past_32_bit_offsets():
    # rows 65,536 values apart: the last ones lie beyond 2^31 values and 2^32 bytes
    T, Hq, Hkv, D, width = 33_001, 2, 1, 64, 65_536
    row = torch.empty(T, width, dtype=BF, device="cuda")
    cols = torch.randn(T, 4 * D, device="cuda").to(BF)
    row[:, 1024:1024 + 4 * D] = cols
    q, k = row[:, 1024:1024 + 2 * D].view(T, Hq, D), row[:, 1024 + 2 * D:1024 + 3 * D].view(T, Hkv, D)
    qc, kc = cols[:, :2 * D].contiguous().view(T, Hq, D), cols[:, 2 * D:3 * D].contiguous().view(T, Hkv, D)
    P, off = 1, [0, T - 1]
    g = torch.Generator(device="cuda").manual_seed(1)
    w = [1 + 0.1 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    f = _inv_freq(D, 1e4)
    got, want = dk.qk_norm_rope(q, k, P, off, f, *w), dk.qk_norm_rope(qc, kc, P, off, f, *w)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    dq, dkk = (torch.randn(T, H, D, generator=g, device="cuda").to(BF) for H in (Hq, Hkv))
    want = dk.qk_norm_rope_backward(qc, kc, dq, dkk, P, off, f, *w)
    out = torch.empty(T, width, dtype=BF, device="cuda")
    o = [out[:, 2048:2048 + 2 * D].view(T, Hq, D), out[:, 2048 + 2 * D:2048 + 3 * D].view(T, Hkv, D)]
    dw = [torch.empty(D, device="cuda") for _ in range(2)]
    ws = torch.empty(dk.dualkv_qk_norm_rope_bwd_workspace_bytes(P, 1, off, Hq, Hkv, D), dtype=torch.uint8, device="cuda")
    dk.dualkv_qk_norm_rope_bwd(q, k, dq, dkk, *w, 0.0, 1e-6, f, D, False, P, 1, off, Hq, Hkv, D, *o, *dw, ws)
    for a, b in zip(o + dw, want):
        assert torch.equal(a, b)


def test_binding_refuses_what_does_not_fit():
    P, off, Hq, Hkv, D = 4, [0, 3], 2, 1, 64
    q, k, qw, kw, f, dq_out, dk_out = _inputs(P, off, Hq, Hkv, D, D, BF, False, 1)
    T = P + off[-1]
    qo, ko = torch.empty_like(q), torch.empty_like(k)

    def call(**kw_):
        a = dict(q=q, k=k, q_weight=qw, k_weight=kw, inv_freq=f, rope_dim=D, q_out=qo, k_out=ko)
        a.update(kw_)
        dk.dualkv_qk_norm_rope(a["q"], a["k"], a["q_weight"], a["k_weight"], 0.0, EPS, a["inv_freq"], a["rope_dim"], False,
                               P, 1, off, Hq, Hkv, D, a["q_out"], a["k_out"])

    call()
    for bad in (dict(q=q[:-1]), dict(q=q.float()), dict(q=q.cpu()), dict(k_weight=None), dict(k_weight=kw.float()),
                dict(inv_freq=f[:-1]), dict(inv_freq=f.double()), dict(q_out=torch.empty(T, 2 * Hq, D, dtype=BF,
                     device="cuda")[:, ::2]), dict(q_weight=qw[:32]), dict(k=k.transpose(0, 1).contiguous().transpose(0, 1)
                     if Hkv > 1 else k[:, :, :32])):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(q_out=q), dict(q=q[:1].expand(T, Hq, D)), dict(rope_dim=24, inv_freq=f[:12])):
        with pytest.raises(dk.DualKVError):
            call(**bad)
    dk.dualkv_check_status()
