"""GPU parity of dualkv_token_logprobs and its backward against ``oracle.policy`` (fp64).

Tolerances, with u = 2^-24, p the row's probabilities, y = z - max z:
  With A = sum p |y| and A2 = sum p y^2, the running sum's relative error is at most
  u (2 A + K), K = 100 + V/128: 2 |y| u from each exponent (its rounding and that of
  scale log2 e), a few u from ex2, and one step per addition (V/512 by a thread, the trees,
  3 u per change of the maximum).
  lse      u (2 A + K + 4 |lse| + 4 |max z|)
  logp     u (2 A + K + 4 |z_t - max z| + 4 |max z| + 4 |logp|)
  entropy  u (1 + A + A2) (K + 8) + 4 u |H|
  dlogits  half a step of the output type times |d|, plus scale p ((3 |d| + |z| + 4) u c + 6 u c)
           with c = sum |g| + |h| (|d| + |H|), d = z - lse: the exponent's rounding, then the
           coefficient's; u |z| because scale is an fp32 argument: it moves z by up to u |z|
           against the oracle's (1.3 is 0.6 u off in fp32), while lse is given and does not
           move along; plus (N + 4) u scale sum |g| at a target; plus 2^-125 max(1, c) where ex2
           flushes a subnormal p and bf16 ends.
"""
import numpy as np
import pytest
import torch

from oracle import policy as opl
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(P, off, V, dtype, pad, seed, ignored=0.2, spread=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, M = off[-1], opl.rows_of(P, off)
    logits = (spread * torch.randn(M, V + pad, generator=g, device="cuda")).to(dtype)[:, :V]
    tok = torch.randint(0, V, (n,), generator=g, device="cuda")
    tok[torch.rand(n, generator=g, device="cuda") < ignored] = -100
    dlogp, dent = (torch.randn(n, generator=g, device="cuda") for _ in range(2))
    return logits, tok, dlogp, dent


def _check_forward(got, logits, tok, scale, P, off):
    logp, ent, lse = (None if t is None else _np(t) for t in got)
    want = opl.logprobs(_np(logits), tok.tolist(), scale, P, off)
    z = _np(logits) * scale
    V = z.shape[1]
    K = 100 + V / 128
    pred = opl.predictor(P, off)
    np.testing.assert_array_equal(np.isfinite(lse), np.isfinite(want[2]))
    live = np.zeros(len(lse), dtype=bool)
    for i, m in enumerate(pred):
        if m < 0 or tok[i] < 0:
            assert logp[i] == 0.0 and (ent is None or ent[i] == 0.0)
            continue
        live[m] = True
        top = z[m].max()
        if top == -np.inf:
            assert lse[m] == logp[i] == -np.inf and (ent is None or ent[i] == 0.0)
            continue
        p = np.exp(z[m] - top)
        p /= p.sum()
        y = np.where(p > 0, np.maximum(z[m] - top, -1e30), 0.0)
        A, A2 = (p * np.abs(y)).sum(), (p * y * y).sum()
        base = 2 * A + K + 4 * abs(top)
        assert abs(lse[m] - want[2][m]) <= U * (base + 4 * abs(want[2][m]))
        if want[0][i] == -np.inf:
            assert logp[i] == -np.inf
        else:
            assert abs(logp[i] - want[0][i]) <= U * (base + 4 * abs(z[m, tok[i]] - top) + 4 * abs(want[0][i]))
        if ent is not None:
            assert abs(ent[i] - want[1][i]) <= U * ((1 + A + A2) * (K + 8) + 4 * abs(want[1][i]))
    assert np.all(lse[~live] == 0.0)
    return want


def _check_backward(got, logits, tok, scale, P, off, lse, ent, dlogp, dent):
    lse, ent, dlogp = _np(lse), None if ent is None else _np(ent), _np(dlogp)
    dent = None if dent is None else _np(dent)
    want = opl.logprobs_backward(_np(logits), tok.tolist(), scale, P, off, lse, ent, dlogp, dent)
    z = _np(logits) * scale
    G, Hs, H = np.zeros(len(lse)), np.zeros(len(lse)), np.zeros(len(lse))
    at = np.zeros_like(z)
    for i, m in enumerate(opl.predictor(P, off)):
        if m >= 0 and tok[i] >= 0 and lse[m] != -np.inf:
            G[m] += abs(dlogp[i])
            at[m, tok[i]] = 1.0
            if dent is not None:
                Hs[m] += abs(dent[i])
                H[m] = ent[i]
    used = (G > 0) | (Hs > 0)
    with np.errstate(invalid="ignore"):
        d = np.where(used[:, None], np.maximum(z - lse[:, None], -1e4), -1e4)
    p = np.exp(d)
    c = G[:, None] + Hs[:, None] * (np.abs(d) * (p > 0) + np.abs(H[:, None]))
    absz = np.where(p > 0, np.abs(np.maximum(z, -1e4)), 0.0)
    step = 2.0 ** -8 if logits.dtype == BF else U
    N = len(off) - 1
    tol = (step * np.abs(want) + scale * p * ((3 * np.abs(d) + absz + 4) * U * c + 6 * U * c)
           + at * (N + 4) * U * scale * G[:, None] + 2.0 ** -125 * np.maximum(1.0, c))
    err = np.abs(_np(got) - want)
    assert np.all(err <= tol), float(np.max(err - tol))
    return want


CASES = [
    # name, P, offsets, V, dtype, row padding, scale
    ("one-token", 1, [0, 1], 1000, F32, 0, 1.0),
    ("one-entry", 3, [0, 2, 5], 1, BF, 0, 1.0),
    ("three-entries", 0, [0, 2, 5], 3, BF, 2, 1.0),
    ("no-token", 4, [0, 0, 0], 64, BF, 0, 1.0),
    ("odd-bf16", 7, [0, 5, 5, 19, 20, 44], 2049, BF, 0, 0.7),
    ("odd-f32", 7, [0, 5, 5, 19, 20, 44], 1023, F32, 0, 1.3),
    ("padded", 0, [0, 3, 9, 9, 30], 4097, BF, 7, 1.0),
    ("aligned", 2, [0, 16, 32], 4096, BF, 64, 1.0),
    ("wide-bf16", 1, [0, 2, 3], 70001, BF, 0, 1.0),
    ("wide-f32", 0, [0, 2, 5], 40003, F32, 1, 2.0),
    ("many-segments", 5, [0] + np.cumsum(np.arange(300) % 3).tolist(), 9, F32, 0, 1.0),
    ("most-segments", 5, [0] + np.cumsum(np.arange(4095) % 2).tolist(), 40, BF, 0, 1.0),
]


@pytest.mark.parametrize("entropy", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_matches_the_oracle(case, entropy):
    name, P, off, V, dtype, pad, scale = case
    logits, tok, dlogp, dent = _inputs(P, off, V, dtype, pad, 7 + V)
    N = len(off) - 1
    n, M = off[-1], opl.rows_of(P, off)
    nan = lambda k: torch.full((k,), float("nan"), device="cuda")  # noqa: E731
    logp, ent, lse = nan(n), nan(n) if entropy else None, nan(M)
    dk.dualkv_token_logprobs(logits, tok, scale, P, N, off, logp, ent, lse)
    _check_forward((logp, ent, lse), logits, tok, scale, P, off)
    # into rows of another padding, whose padding has to stay as it is
    full = torch.full((M, V + 5), 3.0, dtype=dtype, device="cuda")
    dlogits = full[:, :V]
    dk.dualkv_token_logprobs_bwd(logits, tok, scale, P, N, off, lse, ent, dlogp, dent if entropy else None, dlogits)
    dk.dualkv_check_status()
    _check_backward(dlogits, logits, tok, scale, P, off, lse, ent, dlogp, dent if entropy else None)
    assert bool((full[:, V:] == 3.0).all())
    # in place: the same bits
    dk.dualkv_token_logprobs_bwd(logits, tok, scale, P, N, off, lse, ent, dlogp, dent if entropy else None, logits)
    assert torch.equal(logits.view(torch.int16 if dtype == BF else torch.int32),
                       dlogits.contiguous().view(torch.int16 if dtype == BF else torch.int32))


def test_rows_that_start_anywhere():
    # a slice of an odd vocabulary's rows starts at any element
    V, P, off = 517, 3, [0, 4, 9]
    g = torch.Generator(device="cuda").manual_seed(3)
    for dtype in (BF, F32):
        for skip in range(9):
            flat = torch.randn(skip + 10 * V, generator=g, device="cuda").to(dtype)
            logits = flat[skip:].view(10, V)
            tok = torch.randint(0, V, (9,), generator=g, device="cuda")
            dlogp = torch.randn(9, generator=g, device="cuda")
            got = dk.token_logprobs(logits, tok, P, off, entropy=True)
            _check_forward(got, logits, tok, 1.0, P, off)
            d = dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off)
            _check_backward(d, logits, tok, 1.0, P, off, got[2], None, dlogp, None)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_masked_entries_and_rows(dtype):
    V, P, off = 300, 2, [0, 3, 7]
    logits, tok, dlogp, dent = _inputs(P, off, V, dtype, 0, 1, ignored=0.0)
    logits[:, 200:] = -float("inf")       # a padded vocabulary
    logits[0, :199] = -float("inf")       # one entry left
    tok[:] = torch.arange(7, device="cuda") * 20
    tok[0] = tok[3] = 199
    tok[4] = 250                          # a masked target: log probability -inf
    logits[2] = -float("inf")             # a row without any entry left
    logits[5, 7] = torch.finfo(dtype).min  # the type's lowest value
    tok[5] = 7
    got = dk.token_logprobs(logits, tok, P, off, entropy=True)
    _check_forward(got, logits, tok, 1.0, P, off)
    assert got[0][0] == 0.0 and got[1][0] == 0.0 and got[0][4] == -float("inf")
    d = dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off, entropy=got[1], dentropy=dent)
    want = _check_backward(d, logits, tok, 1.0, P, off, got[2], got[1], dlogp, dent)
    assert np.all(want[2] == 0) and bool(torch.isfinite(d).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_values_in_ignored_rows_do_not_matter(dtype):
    V, P, off = 129, 2, [0, 4, 8]
    logits, tok, dlogp, dent = _inputs(P, off, V, dtype, 0, 2, ignored=0.0)
    tok[2] = -1
    logits[2] = float("nan")
    logits[4] = float("inf")  # the last row of the first segment predicts nothing
    dlogp[2] = dent[2] = float("nan")
    got = dk.token_logprobs(logits, tok, P, off, entropy=True)
    d = dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off, entropy=got[1], dentropy=dent)
    for t in got + (d,):
        assert bool(torch.isfinite(t).all())
    assert got[0][2] == 0 and got[2][4] == 0 and not d[2].any() and not d[4].any()
    # in a live row they show, and only there
    logits[3, 5] = float("nan")
    logits[6, 5] = float("inf")
    lp, ent, lse = dk.token_logprobs(logits, tok, P, off, entropy=True)
    bad = torch.isnan(lp)
    assert bad.nonzero().flatten().tolist() == [3, 6] and bool(torch.isnan(ent[bad]).all())
    assert torch.isnan(lse).nonzero().flatten().tolist() == [3, 6]
    d = dk.token_logprobs_backward(logits, tok, lse, dlogp, P, off)
    assert torch.isnan(d).any(1).nonzero().flatten().tolist() == [3, 6]


def test_shared_row_with_equal_targets_and_cancelling_gradients():
    # the prompt's last row predicts one token per segment: the same one twice, gradients that sum to 0
    V, P = 50, 4
    off = list(range(7))
    logits, tok, _, _ = _inputs(P, off, V, F32, 0, 4, ignored=0.0)
    tok[:] = torch.tensor([3, 9, 3, 3, -1, 9])
    dlogp = torch.tensor([1.0, 2.0, -1.0, 0.5, 7.0, -2.5], device="cuda")
    logp, _, lse = dk.token_logprobs(logits, tok, P, off)
    d = dk.token_logprobs_backward(logits, tok, lse, dlogp, P, off)
    _check_backward(d, logits, tok, 1.0, P, off, lse, None, dlogp, None)
    assert d[0, 3] == 0.5 and d[0, 9] == -0.5 and not d[1:].any()


def test_zero_gradients_leave_zeros_without_reading():
    V, P, off = 77, 1, [0, 3]
    logits, tok, dlogp, _ = _inputs(P, off, V, BF, 0, 5, ignored=0.0)
    _, _, lse = dk.token_logprobs(logits, tok, P, off)
    dlogp[1] = 0.0
    logits[1] = float("nan")
    d = dk.token_logprobs_backward(logits, tok, lse, dlogp, P, off)
    assert not d[1].any() and bool(torch.isfinite(d).all())


def test_token_past_the_vocabulary_is_reported_and_ignored():
    V, P, off = 64, 2, [0, 2, 4]
    logits, tok, dlogp, _ = _inputs(P, off, V, BF, 0, 6, ignored=0.0)
    want = dk.token_logprobs(logits, tok, P, off)
    dk.dualkv_check_status()
    for at in (1, 2):  # a row of its own, and the shared row
        bad = tok.clone()
        bad[at] = V
        logp, _, lse = dk.token_logprobs(logits, bad, P, off)
        with pytest.raises(dk.DualKVError):
            dk.dualkv_check_status()
        keep = [i for i in range(4) if i != at]
        assert logp[at] == 0.0 and torch.equal(logp[keep], want[0][keep])
        d = dk.token_logprobs_backward(logits, bad, lse, dlogp, P, off)
        with pytest.raises(dk.DualKVError):
            dk.dualkv_check_status()
        assert bool(torch.isfinite(d).all())
    dk.dualkv_check_status()


def test_more_than_2_31_logits():
    # rows past the 32-bit range of elements: the last rows against the same rows alone
    V, n = 131072, 16385
    P, off = 1, [0, n]
    g = torch.Generator(device="cuda").manual_seed(8)
    logits = torch.randn(n + 1, V, generator=g, device="cuda", dtype=BF)
    tok = torch.full((n,), -1, dtype=torch.int64, device="cuda")
    tok[-3:] = torch.tensor([5, V - 1, 77], device="cuda")
    tok[0] = 9
    dlogp = torch.randn(n, generator=g, device="cuda")
    logp, _, lse = dk.token_logprobs(logits, tok, P, off)
    d = dk.token_logprobs_backward(logits, tok, lse, dlogp, P, off)
    small = torch.cat((logits[:1], logits[-4:])).contiguous()
    off2 = [0, 4]
    tok2 = torch.cat((tok[:1], tok[-3:]))
    dlogp2 = torch.cat((dlogp[:1], dlogp[-3:]))
    lp2, _, lse2 = dk.token_logprobs(small, tok2, P, off2)
    # rows n - 3 .. n - 1 predict tokens n - 3 .. n - 1; in the small batch they are rows 1 .. 3
    d2 = dk.token_logprobs_backward(small, tok2, lse2, dlogp2, P, off2)
    assert torch.allclose(logp[-3:], lp2[1:], rtol=0, atol=1e-5) and torch.allclose(logp[0], lp2[0], rtol=0, atol=1e-5)
    torch.testing.assert_close(d[-4:].float(), d2[1:].float(), rtol=2.0 ** -7, atol=1e-9)
    assert not d[1:-4].any()


def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph():
    P, off, V = 3, [0, 40, 90], 5003
    N = len(off) - 1
    logits, tok, dlogp, dent = _inputs(P, off, V, BF, 0, 9)
    want = dk.token_logprobs(logits, tok, P, off, entropy=True)
    want += (dk.token_logprobs_backward(logits, tok, want[2], dlogp, P, off, entropy=want[1], dentropy=dent),)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dk.token_logprobs(logits, tok, P, off, entropy=True, stream=side)
    got += (dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off, entropy=got[1], dentropy=dent, stream=side),)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    outs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dk.dualkv_token_logprobs(logits, tok, 1.0, P, N, off, outs[0], outs[1], outs[2])
        dk.dualkv_token_logprobs_bwd(logits, tok, 1.0, P, N, off, outs[2], outs[1], dlogp, dent, outs[3])
    for _ in range(2):
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_first_call_of_a_process_may_be_captured():
    dk.dualkv_release()  # the status word is set up again inside the capture
    P, off, V = 3, [0, 4], 65
    logits, tok, _, _ = _inputs(P, off, V, F32, 0, 10, ignored=0.0)
    logp, lse = torch.zeros(4, device="cuda"), torch.zeros(5, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        dk.dualkv_token_logprobs(logits, tok, 1.0, P, 1, off, logp, None, lse)
    graph.replay()
    torch.cuda.synchronize()
    _check_forward((logp, None, lse), logits, tok, 1.0, P, off)
    dk.dualkv_check_status()


def test_binding_refuses_what_does_not_fit():
    P, off, V = 2, [0, 3], 40
    logits, tok, dlogp, dent = _inputs(P, off, V, BF, 0, 11, ignored=0.0)
    logp, ent, lse = dk.token_logprobs(logits, tok, P, off, entropy=True)

    def fwd(**kw):
        a = dict(logits=logits, tokens=tok, scale=1.0, logp=logp, entropy=None, lse=lse)
        a.update(kw)
        dk.dualkv_token_logprobs(a["logits"], a["tokens"], a["scale"], P, 1, off, a["logp"], a["entropy"], a["lse"])

    def bwd(**kw):
        a = dict(lse=lse, entropy=ent, dlogp=dlogp, dentropy=dent, dlogits=torch.empty_like(logits))
        a.update(kw)
        dk.dualkv_token_logprobs_bwd(logits, tok, 1.0, P, 1, off, a["lse"], a["entropy"], a["dlogp"], a["dentropy"],
                                     a["dlogits"])

    fwd()
    bwd()
    for bad in (dict(logits=logits[1:]), dict(logits=logits.half()), dict(logits=logits.cpu()), dict(logits=logits[:, ::2]),
                dict(tokens=tok.int()), dict(tokens=tok[:-1]), dict(logp=lse), dict(lse=logp), dict(logp=logp.double())):
        with pytest.raises(ValueError):
            fwd(**bad)
    for bad in (dict(scale=0.0), dict(scale=float("nan")), dict(logits=logits[:1].expand(4, V))):
        with pytest.raises(dk.DualKVError):
            fwd(**bad)
    for bad in (dict(lse=None), dict(entropy=None), dict(dlogits=torch.empty_like(logits).float()), dict(dlogits=logits[:-1])):
        with pytest.raises(ValueError):
            bwd(**bad)
    two = torch.empty(8, V, dtype=BF, device="cuda")
    with pytest.raises(dk.DualKVError):  # overlapping, but not in place
        dk.dualkv_token_logprobs_bwd(two[:4], tok, 1.0, P, 1, off, lse, None, dlogp, None, two[1:5])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows", [1, 3, 40, 80, 160, 320])
def test_rows_split_over_blocks(rows, dtype):
    # few rows are split over a cluster (forward) or into smaller parts (backward): targets, masked
    # stretches and the maximum in different parts, an empty part, odd ends
    V, P, off = 70003, 1, [0, rows]
    logits, tok, dlogp, dent = _inputs(P, off, V, dtype, 3, rows, ignored=0.0)
    tok[0], tok[-1] = V - 1, 0
    logits[:, 20000:45000] = -float("inf")
    logits[0, 60000] = 30.0
    got = dk.token_logprobs(logits, tok, P, off, entropy=True)
    pick = sorted({0, rows // 2, rows - 1})
    few = logits[pick].contiguous()
    ftok, flse = tok[pick], got[2][pick]
    z = _np(few)
    want = opl.logprobs(np.concatenate([z, z[:1]]), ftok.tolist(), 1.0, 1, [0, len(pick)])
    for k, i in enumerate(pick):  # row i of the batch predicts token i, as row k of the few does token k
        top, p = z[k].max(), np.exp(z[k] - want[2][k])
        y = np.where(p > 0, np.maximum(z[k] - top, -1e30), 0.0)
        A, A2, K = (p * np.abs(y)).sum(), (p * y * y).sum(), 100 + V / 128
        base = 2 * A + K + 4 * abs(top)
        assert abs(float(flse[k]) - want[2][k]) <= U * (base + 4 * abs(want[2][k]))
        if want[0][k] == -np.inf:  # a masked target
            assert float(got[0][i]) == -np.inf
        else:
            assert abs(float(got[0][i]) - want[0][k]) <= U * (base + 4 * abs(z[k, ftok[k]] - top) + 4 * abs(want[0][k]))
        assert abs(float(got[1][i]) - want[1][k]) <= U * ((1 + A + A2) * (K + 8) + 4 * abs(want[1][k]))
    d = dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off, entropy=got[1], dentropy=dent)
    sub = torch.cat((few, few[:1]))
    lse2 = torch.cat((flse, torch.zeros(1, device="cuda")))
    dsub = torch.cat((d[pick], torch.zeros_like(d[:1])))
    _check_backward(dsub, sub, ftok, 1.0, 1, [0, len(pick)], lse2, got[1][pick], dlogp[pick], dent[pick])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 70003])
def test_rows_far_from_zero(V, dtype):
    # masked throughout with the type's lowest value (uniform probabilities), or far above or below 0:
    # an fp32 lse is too coarse there to normalise with
    P, off = 1, [0, 4]
    logits, tok, dlogp, dent = _inputs(P, off, V, dtype, 0, 13, ignored=0.0)
    lowest = torch.finfo(dtype).min
    logits[0] = lowest
    logits[1, : V // 2] = lowest
    logits[2] += 3e4 if dtype == F32 else 2.0 ** 14
    logits[3] -= 1e5 if dtype == F32 else 2.0 ** 15
    got = dk.token_logprobs(logits, tok, P, off, entropy=True)
    _check_forward(got, logits, tok, 1.0, P, off)
    z = _np(logits)
    lse = opl.logprobs(z, tok.tolist(), 1.0, P, off)[2]  # fp64
    want = np.zeros_like(z)
    tol = np.zeros_like(z)
    step = 2.0 ** -8 if dtype == BF else U
    for i in range(4):  # row i predicts token i
        top = z[i].max()
        y = np.maximum(z[i] - top, -1e4)
        d = y - np.log(np.exp(y).sum())
        p, g, h = np.exp(d), float(dlogp[i]), float(dent[i])
        H = -(p * np.where(p > 0, d, 0.0)).sum()
        want[i] = -g * p - h * p * (np.where(p > 0, d, 0.0) + H)
        want[i, tok[i]] += g
        # the row's sum (as the forward's) moves d as well: u (K + V/128 + 100); the given entropy its own error
        A = (p * np.abs(np.where(p > 0, d, 0.0))).sum()
        K = 100 + V / 128
        c = abs(g) + abs(h) * (np.abs(d) * (p > 0) + abs(H))
        tol[i] = step * np.abs(want[i]) + p * U * ((3 * np.abs(d) + 2 * A + K + 10) * c + abs(h) * (1 + A) ** 2 * (K + 8))
        tol[i, tok[i]] += 8 * U * abs(g)
    for entropy in (False, True):
        kw = dict(entropy=got[1], dentropy=dent) if entropy else {}
        for inplace in (False, True):
            x = logits.clone()
            out = dk.token_logprobs_backward(x, tok, got[2], dlogp, P, off, inplace=inplace, **kw)
            if entropy:
                err = np.abs(_np(out)[:4] - want[:4])
                assert np.all(err <= tol[:4] + 2.0 ** -125), float(np.max(err - tol[:4]))
            else:
                sums = _np(out)[:4].sum(1)  # a softmax gradient sums to 0
                assert np.all(np.abs(sums) <= step * np.abs(_np(out)[:4]).sum(1) + U * (K + 100))
            assert not out[4].any()


def test_calls_of_two_threads():
    import threading
    P, off, V = 3, [0, 40, 90], 5003
    logits, tok, dlogp, dent = _inputs(P, off, V, BF, 0, 14)
    want = dk.token_logprobs(logits, tok, P, off, entropy=True)
    grad = dk.token_logprobs_backward(logits, tok, want[2], dlogp, P, off, entropy=want[1], dentropy=dent)
    x = dict(logp=want[0], old=want[0] - 0.1 * dent, adv=torch.tensor([1.0, -1.0], device="cuda"))
    loss = dk.policy_loss(x["logp"], x["old"], x["adv"], off)
    torch.cuda.synchronize()
    wrong = []

    def work():
        stream = torch.cuda.Stream()
        for _ in range(20):
            got = dk.token_logprobs(logits, tok, P, off, entropy=True, stream=stream)
            g = dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off, entropy=got[1], dentropy=dent, stream=stream)
            l3 = dk.policy_loss(x["logp"], x["old"], x["adv"], off, stream=stream)
            stream.synchronize()
            wrong.extend(k for k, (a, b) in enumerate(zip(want + (grad,) + loss, got + (g,) + l3)) if not torch.equal(a, b))

    threads = [threading.Thread(target=work) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


@pytest.mark.parametrize("V", [65, 70003])
def test_forward_without_log_sums(V):
    # scoring alone needs neither lse nor entropies
    P, off = 2, [0, 3, 5]
    logits, tok, _, _ = _inputs(P, off, V, BF, 0, 15)
    want = dk.token_logprobs(logits, tok, P, off)
    logp = torch.full((5,), float("nan"), device="cuda")
    dk.dualkv_token_logprobs(logits, tok, 1.0, P, 2, off, logp, None, None)
    assert torch.equal(logp, want[0])


def test_tensors_of_another_device_are_refused():
    # the binding compares with the calling thread's current device (here: a device that these are not on)
    t = torch.zeros(3, device="cuda")
    with pytest.raises(ValueError, match="current device"):
        dk._arg("call", "t", t, (3,), (F32,), t.get_device() + 1)
    with pytest.raises(ValueError, match="current device"):
        dk._workspace_args("call", t, None, t.get_device() + 1)
