"""The per-token operators at the ends of what their entry points accept, against fp64."""
import numpy as np
import pytest
import torch

import test_gpu_policy as tp
import test_gpu_rope as tr
from oracle import rope as orp
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
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
