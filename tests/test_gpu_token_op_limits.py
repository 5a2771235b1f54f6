"""The per-token operators at the ends of what their entry points accept, against fp64."""
import numpy as np
import pytest
import torch

import test_gpu_logprobs as tl
import test_gpu_policy as tp
import test_gpu_rope as tr
from oracle import policy as opl
from oracle import rope as orp
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


@pytest.mark.parametrize("wdtype", [BF, F32])
@pytest.mark.parametrize("Hq,Hkv,D", [(3, 3, 128), (4, 2, 128), (8, 1, 128), (5, 5, 64), (8, 4, 64), (3, 1, 512)])
def test_norm_without_eps(monkeypatch, Hq, Hkv, D, wdtype):
    # heads that do not fill a warp leave lanes without one, which must add nothing to the weight gradients
    monkeypatch.setattr(tr, "EPS", 0.0)  # the checks' eps
    P, off = 9, [0, 5, 5, 40]
    q, k, qw, kw, f, dq_out, dk_out = tr._inputs(P, off, Hq, Hkv, D, D, wdtype, True, 31)
    y = dk.qk_norm_rope(q, k, P, off, f, qw, kw, eps=0.0)
    g = dk.qk_norm_rope_backward(q, k, dq_out, dk_out, P, off, f, qw, kw, eps=0.0)
    pos, fn = orp.positions(P, off), tr._np(f)
    for i, (x, w, dy) in enumerate(((q, qw, dq_out), (k, kw, dk_out))):
        tr._check_forward(tr._np(y[i]), tr._np(x), tr._np(w), 0.0, pos, fn, False)
        assert bool(torch.isfinite(g[2 + i]).all())
        tr._check_backward(tr._np(g[i]), tr._np(g[2 + i]), tr._np(x), tr._np(dy), tr._np(w), 0.0, pos, fn, False)


@pytest.mark.parametrize("off", [[0, 40, 90], [0, 3000, 3001, 30000]], ids=["one-cluster", "two-launches"])
@pytest.mark.parametrize("entropies", [INF, float("nan")])
def test_terms_without_a_coefficient_stay_out_of_the_loss(off, entropies):
    # KL and entropies may be passed for the statistics alone; what they hold then does not reach the loss
    x = tp._inputs(off, 41, False, 0.2)
    x["mask"][:3] = True
    x["ref"][0] = -INF                  # what token_logprobs returns for a masked target
    x["ref"][1] = x["logp"][1] + 100.0  # e^100 is beyond fp32
    x["ent"][2] = entropies
    args = dict(mask=x["mask"], reduction="seq_mean")
    want = dk.policy_loss(x["logp"], x["old"], x["adv"], off, **args)
    loss, stats, w = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["ref"], x["ent"], **args)
    assert bool(torch.isfinite(want[0]).all()) and torch.equal(loss, want[0]) and torch.equal(w, want[2])
    assert torch.equal(stats[[0, 3]], want[1][[0, 3]])
    assert float(stats[1]) == INF and not bool(torch.isfinite(stats[2]))
    # each for itself with the other's coefficient set
    e_only = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["ref"], x["old"], entropy_coef=0.5, **args)
    assert bool(torch.isfinite(e_only[0]).all()) and float(e_only[1][1]) == INF
    kl_only = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["old"], x["ent"], kl_coef=0.5, **args)
    assert bool(torch.isfinite(kl_only[0]).all()) and not bool(torch.isfinite(kl_only[1][2]))
    # with a coefficient they do
    both = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["ref"], x["ent"], kl_coef=0.5, **args)
    assert float(both[0]) == INF


def _gradients_from_the_logits(logits, tok, scale, P, off, dlogp, dent):
    """fp64 gradient of the logits with each row's own sum, and its tolerance per value.

    With p, d = z - lse, A, A2 and K as in test_gpu_logprobs: the kernel normalises with the forward's lse, off by
    u (2 A + K + 4 |lse| + 4 |max z|), in rows whose lse is at most 128 (bf16: 1024) from 0, and with a sum of its
    own, off by u (2 A + K), in all others; the entropy that it is given is off by u ((1 + A + A2) (K + 8) + 4 |H|).  The rest as
    there; scales are exact in fp32 here."""
    z, tok = tl._np(logits) * scale, torch.as_tensor(tok).tolist()
    M, V = z.shape
    want, tol = np.zeros_like(z), np.zeros_like(z)
    K = 100 + V / 128
    step = 2.0 ** -8 if logits.dtype == BF else U
    for m in range(M):
        mine = [i for i, r in enumerate(opl.predictor(P, off)) if r == m and tok[i] >= 0]
        if not mine:
            continue
        top = z[m].max()
        y = np.maximum(z[m] - top, -1e4)
        s = np.exp(y).sum()
        d, lse = y - np.log(s), top + np.log(s)
        p = np.exp(d)
        dp = np.where(p > 0, d, 0.0)
        H = -(p * dp).sum()
        A, A2 = (p * np.abs(dp)).sum(), (p * dp * dp).sum()
        g, h = dlogp[mine].sum(), dent[mine].sum() if dent is not None else 0.0
        ga, ha = np.abs(dlogp[mine]).sum(), np.abs(dent[mine]).sum() if dent is not None else 0.0
        want[m] = -g * p - h * p * (dp + H)
        for i in mine:
            want[m, tok[i]] += dlogp[i]
        want[m] *= scale
        holds = 1024.01 if logits.dtype == BF else 128.001
        sum_off = 2 * A + K + (8 * max(abs(lse), abs(top)) if abs(lse) <= holds else 0.0)
        c = ga + ha * (np.abs(dp) + abs(H))
        # p moves by its own relative error, and with it (by ha p) the factor d + H
        e = p * ((3 * np.abs(dp) + sum_off + 10) * (c + ha) + ha * ((1 + A + A2) * (K + 8) + 4 * abs(H)))
        tol[m] = step * np.abs(want[m]) + scale * U * e + 2.0 ** -125 * np.maximum(1.0, c)
        for i in mine:
            tol[m, tok[i]] += scale * U * (len(off) + 4) * ga
    return want, tol


@pytest.mark.parametrize("scale", [0.75, 1.25])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 70003])
def test_rows_of_the_lowest_value_at_any_scale(V, dtype, scale):
    # scale times the type's lowest value passes fp32's range: the log-sum stays finite, -inf keeps its one meaning
    P, off = 1, [0, 5]
    logits, tok, dlogp, dent = tl._inputs(P, off, V, dtype, 0, 61, ignored=0.0)
    most = torch.finfo(dtype).max
    logits[0] = -most              # uniform probabilities
    logits[1, : V // 2] = -most
    logits[2] = -INF               # a row without any entry
    logits[3] = most
    logits[4] = -most
    logits[4, int(tok[4])] = most  # one sure entry
    lp, ent, lse = (tl._np(t) for t in dk.token_logprobs(logits, tok, P, off, scale=scale, entropy=True))
    bound = float(np.finfo(np.float32).max)
    for m, p in ((0, 1 / V), (3, 1 / V), (4, 1.0)):
        K = 100 + V / 128
        assert abs(lp[m] - np.log(p)) <= U * (K + 4 * abs(np.log(p)))
        assert abs(ent[m] + np.log(p)) <= U * (2 * (K + 8) + 4 * abs(np.log(p)))
        want = np.clip(tl._np(logits[m]).max() * scale, -bound, bound)
        assert np.isfinite(lse[m]) and abs(lse[m] - want) <= 2 * U * abs(want)
    assert lp[2] == lse[2] == -INF and ent[2] == 0.0
    keep = [0, 1, 3, 4]
    full = dk.token_logprobs(logits, tok, P, off, scale=scale, entropy=True)
    for inplace in (False, True):
        x = logits.clone()
        out = dk.token_logprobs_backward(x, tok, full[2], dlogp, P, off, scale=scale, entropy=full[1], dentropy=dent,
                                         inplace=inplace)
        some = torch.cat((logits[keep], logits[:1]))  # the last row predicts nothing
        want, tol = _gradients_from_the_logits(some, tok[keep], scale, P, [0, 4], tl._np(dlogp)[keep],
                                               tl._np(dent)[keep])
        err = np.abs(tl._np(out)[keep] - want[:4])
        assert np.all(err <= tol[:4]), float(np.max(err - tol[:4]))
        assert not out[2].any() and not out[5].any()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 70003])
def test_masked_entries_under_large_gradients(V, dtype):
    # a masked entry's gradient is 0 whatever flows into its row (0 times a large factor, not 0 times infinity)
    P, off = 1, [0, 4, 7]
    logits, tok, dlogp, dent = tl._inputs(P, off, V, dtype, 0, 71, ignored=0.0)
    tok %= V // 2
    logits[:, V // 2:] = -INF
    logits[1, V // 4: V // 2] = torch.finfo(dtype).min
    got = dk.token_logprobs(logits, tok, P, off, entropy=True)
    dent *= 1e12
    d = dk.token_logprobs_backward(logits, tok, got[2], dlogp, P, off, entropy=got[1], dentropy=dent)
    assert bool(torch.isfinite(d).all()) and not d[:, V // 2:].any()
    tl._check_backward(d, logits, tok, 1.0, P, off, got[2], got[1], dlogp, dent)


@pytest.mark.parametrize("scale", [1.0, 1.25])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("V", [40, 4096, 70003])
def test_gradients_of_rows_off_zero(V, dtype, scale):
    # the rounding of an fp32 lse would be up to 2^-13 of every probability, and more than g (1 - p) at a sure target
    P, off = 2, [0, 9, 12, 13]
    for k, shift in enumerate((0.0, 45.0, 70.0, 200.0, -1000.0, 1030.0, 4000.0, 4090.0)):
        logits, tok, dlogp, dent = tl._inputs(P, off, V, dtype, 0, 50 + k, ignored=0.0)
        rows = torch.tensor(opl.predictor(P, off), device="cuda")
        logits[rows[::2], tok[::2]] += 14.0 + logits.float().amax().to(dtype)  # every other target is sure
        logits = (logits.float() + shift + 3.7 * torch.arange(len(logits), device="cuda")[:, None]).to(dtype)
        lp, ent, lse = dk.token_logprobs(logits, tok, P, off, scale=scale, entropy=True)
        for entropy in (False, True):
            kw = dict(entropy=ent, dentropy=dent) if entropy else {}
            want, tol = _gradients_from_the_logits(logits, tok, scale, P, off, tl._np(dlogp),
                                                   tl._np(dent) if entropy else None)
            out = dk.token_logprobs_backward(logits, tok, lse, dlogp, P, off, scale=scale, **kw)
            err = np.abs(tl._np(out) - want)
            assert np.all(err <= tol), (shift, float(np.max(err / np.maximum(tol, 1e-300))))
            # rows that start elsewhere within 16 bytes, and in place: the same bits
            full = torch.full((len(logits), V + 3), 7.0, dtype=dtype, device="cuda")
            dk.dualkv_token_logprobs_bwd(logits, tok, scale, P, len(off) - 1, off, lse, ent, dlogp,
                                         dent if entropy else None, full[:, 1:V + 1])
            assert torch.equal(full[:, 1:V + 1], out) and bool((full[:, V + 1:] == 7.0).all())
            x = logits.clone()
            dk.token_logprobs_backward(x, tok, lse, dlogp, P, off, scale=scale, inplace=True, **kw)
            assert torch.equal(x, out)
    dk.dualkv_check_status()


@pytest.mark.parametrize("reduction", ["token_mean", "seq_mean", "seq_sum"])
def test_loss_of_more_records_than_the_join_holds(reduction):
    # 1,024 tokens a record: 4,096 records and more are read twice
    for n in (4_100_000, 4_300_007, 9_000_001):
        off = [0, 5, 5, n // 3, n]
        x = tp._inputs(off, n, True, 0.3)
        args = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.05, entropy_coef=0.01)
        loss, stats, w = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["ref"], x["ent"], x["mask"], reduction=reduction,
                                        per_token=True, **args)
        lp, old, ref, ent, A = (x[k].double() for k in ("logp", "old", "ref", "ent", "adv"))
        seg = torch.repeat_interleave(torch.arange(4, device="cuda"), torch.tensor(np.diff(off), device="cuda"))
        live = torch.zeros(4, dtype=torch.float64, device="cuda").index_add_(0, seg, x["mask"].double())
        per = {"token_mean": live.sum().expand(4), "seq_mean": 4 * live, "seq_sum": torch.full_like(live, 4.0)}[reduction]
        want_w = torch.where(live > 0, 1.0 / per, torch.zeros_like(live))
        on = want_w[seg] * x["mask"]
        ratio = torch.exp(lp - old)
        pg = -torch.minimum(ratio * A, ratio.clamp(0.8, 1.28) * A)
        d = ref - lp
        kl = torch.expm1(d) - d
        far = torch.where(A > 0, ratio > 1.28, ratio < 0.8) & (A != 0) & x["mask"]
        want = torch.stack([(on * pg).sum(), (on * kl).sum(), (on * ent).sum(), far.sum() / live.sum()])
        # tolerances as in test_gpu_policy; a weight's division and its count beyond 2^24 round twice
        tol = U * torch.stack([24 * (on * pg.abs()).sum(), 24 * (on * (kl + (d.exp() + 1) * d.abs())).sum(),
                               16 * (on * ent.abs()).sum(), torch.zeros_like(want[0])]) + 2 * U * want.abs()
        assert bool(((w.double() - want_w).abs() <= 2 * U * want_w).all())
        assert bool(((stats.double() - want).abs() <= tol).all()), ((stats.double() - want) / tol)
        total = want[0] + 0.05 * want[1] - 0.01 * want[2]
        assert abs(float(loss) - float(total)) <= float(tol[0] + 0.05 * tol[1] + 0.01 * tol[2] + U * total.abs())
