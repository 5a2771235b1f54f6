"""GPU parity of dualkv_policy_loss and its backward against ``oracle.policy`` (fp64).

Tolerances, with u = 2^-24 (sums over a thread's at most 8 tokens in fp32, then fp64):
  loss, stats  24 u sum w |policy term| (expf 4 u, the difference 2 u, products 2 u, 8 additions),
               24 u sum w (kl + (e^x + 1) |x|), 16 u sum w |H|, and the final rounding
  dlogp        16 u |dloss| w (|A| ratio + b (|e^x - 1| + e^x |x|))
  weights      u each; the share of clipped tokens is a quotient of exact counts: u
"""
import numpy as np
import pytest
import torch

from oracle import policy as opl
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


def _np(t):
    return t.detach().double().cpu().numpy()


def _inputs(off, seed, per_token, masked, sigma=0.2):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, N = off[-1], len(off) - 1
    rn = lambda k: torch.randn(k, generator=g, device="cuda")  # noqa: E731
    logp = -rn(n).abs()
    mask = None if masked is None else torch.rand(n, generator=g, device="cuda") >= masked
    return dict(logp=logp, old=logp + sigma * rn(n), ref=logp + 0.7 * rn(n), ent=rn(n).abs(), adv=rn(n if per_token else N),
                mask=mask)


def _want(x, off, per_token, **kw):
    adv = _np(x["adv"])
    if not per_token:
        adv = np.repeat(adv, np.diff(off))
    return opl.loss(_np(x["logp"]), _np(x["old"]), None if x["ref"] is None else _np(x["ref"]),
                    None if x["ent"] is None else _np(x["ent"]), adv, None if x["mask"] is None else _np(x["mask"]), off, **kw)


def _run_and_check(x, off, lo, hi, dual, b, e, reduction, per_token, dloss=0.75):
    N = len(off) - 1
    loss, stats, w = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["ref"], x["ent"], x["mask"], lo, hi, dual, b, e,
                                    reduction, per_token=per_token)
    up = torch.tensor(dloss, device="cuda")
    dlogp, dent = dk.policy_loss_backward(x["logp"], x["old"], x["adv"], off, up, w, x["ref"], x["mask"], lo, hi, dual, b, e,
                                          per_token=per_token)
    r = _want(x, off, per_token, lo=lo, hi=hi, dual=dual, b=b, e=e, reduction=reduction, dloss=dloss)
    tp, tk, te = 24 * U * r["mag"], 24 * U * r["klmag"], 16 * U * r["entmag"]
    got = _np(stats)
    assert np.all(np.abs(_np(w) - r["weights"]) <= U * np.abs(r["weights"]))
    assert abs(got[0] - r["stats"][0]) <= tp + U * abs(r["stats"][0])
    if x["ref"] is not None:
        assert abs(got[1] - r["stats"][1]) <= tk + U * abs(r["stats"][1])
    else:
        assert got[1] == 0.0
    assert abs(got[2] - r["stats"][2]) <= te + U * abs(r["stats"][2])
    assert abs(got[3] - r["stats"][3]) <= U * r["stats"][3]
    assert abs(float(loss) - r["loss"]) <= tp + abs(b) * tk + abs(e) * te + U * abs(r["loss"])
    rb = _want(x, off, per_token, lo=lo, hi=hi, dual=dual, b=b, e=e, reduction=reduction, dloss=dloss, w=_np(w))
    err = np.abs(_np(dlogp) - rb["dlogp"])
    assert np.all(err <= 16 * U * rb["tol"] + U * np.abs(rb["dlogp"])), float(np.max(err - 16 * U * rb["tol"]))
    if e:
        assert np.all(np.abs(_np(dent) - rb["dentropy"]) <= 2 * U * np.abs(rb["dentropy"]))
    else:
        assert dent is None
    return loss, stats, w, dlogp, dent


LAYOUTS = [
    ("one-token", [0, 1]),
    ("tiny", [0, 32, 64, 96, 128]),
    ("empty-segments", [0, 0, 5, 5, 17, 17]),
    ("chunk-edges", [0, 2048, 4096, 8193, 8193, 10240, 10241]),
    ("chunks-of-one-block", [0, 1023, 2047, 2048, 3073, 4097]),
    ("cluster-edge", [0, 1024, 1024, 2048, 3050]),
    ("past-the-cluster", [0, 1024, 1024, 2048, 4096]),
    ("long", [0, 30011]),
    ("many-segments", [0] + np.cumsum(np.arange(600) % 5).tolist()),
    ("most-segments", [0] + np.cumsum(np.arange(4095) % 3).tolist()),
]


@pytest.mark.parametrize("reduction", ["token_mean", "seq_mean", "seq_sum"])
@pytest.mark.parametrize("name,off", LAYOUTS, ids=[c[0] for c in LAYOUTS])
def test_matches_the_oracle(name, off, reduction):
    for k, (per_token, masked, dual, b, e) in enumerate([(False, None, 0.0, 0.04, 0.0), (True, 0.3, 1.1, 0.0, 0.01),
                                                         (False, 0.9, 2.0, 0.1, -0.02)]):
        x = _inputs(off, 50 + k, per_token, masked)
        if b == 0.0:
            x["ref"] = None
        if e == 0.0:
            x["ent"] = None
        _run_and_check(x, off, 0.2, 0.28, dual, b, e, reduction, per_token)


def test_masks_that_leave_nothing():
    off = [0, 40, 90]
    x = _inputs(off, 3, False, None)
    x["mask"] = torch.ones(90, dtype=torch.uint8, device="cuda")
    x["mask"][:40] = 0
    for name in ("logp", "old", "ref", "ent"):
        x[name][:40] = float("nan")
    x["adv"][0] = float("inf")
    for reduction in dk.LOSS_REDUCTIONS:
        args = dict(ref_logp=x["ref"], mask=x["mask"], kl_coef=0.1, entropy_coef=0.1)
        loss, stats, w = dk.policy_loss(x["logp"], x["old"], x["adv"], off, entropy=x["ent"], reduction=reduction, **args)
        one = torch.ones(1, device="cuda")
        dlogp, dent = dk.policy_loss_backward(x["logp"], x["old"], x["adv"], off, one, w, **args)
        for t in (loss, stats, w, dlogp, dent):
            assert bool(torch.isfinite(t).all())
        assert not dlogp[:40].any() and not dent[:40].any() and w[0] == 0 and bool(dent[40:].all())
    x["mask"][:] = 0
    for reduction in dk.LOSS_REDUCTIONS:
        loss, stats, w = dk.policy_loss(x["logp"], x["old"], x["adv"], off, entropy=x["ent"], reduction=reduction, **args)
        assert float(loss) == 0.0 and not stats.any() and not w.any()
    # no token at all
    none = torch.empty(0, device="cuda")
    loss, stats, w = dk.policy_loss(none, none, x["adv"], [0, 0, 0])
    assert float(loss) == 0.0 and not stats.any() and not w.any()
    dk.policy_loss_backward(none, none, x["adv"], [0, 0, 0], loss, w)


def test_nothing_changes_sides_at_a_bound():
    """Differences a few fp32 steps around each bound, from pairs whose difference rounds."""
    lo, hi, dual = 0.2, 0.28, 3.0
    rng = np.random.default_rng(0)
    logp, old, adv = [], [], []
    for bound, sign in ((1 + hi, 1.0), (1 - lo, -1.0), (dual, -1.0)):
        for base in (0.0, 0.3, -1.7, -23.1):
            o = np.float32(base) * np.ones(200, dtype=np.float32)
            o = (o * (1 + rng.random(200) * 0.1)).astype(np.float32)
            lp = (o.astype(np.float64) + np.log(bound)).astype(np.float32)
            for _ in range(2):
                lp = np.where(rng.random(200) < 0.5, np.nextafter(lp, np.float32(9)), np.nextafter(lp, np.float32(-99)))
            logp.append(lp)
            old.append(o)
            adv.append(np.full(200, sign, dtype=np.float32))
    logp, old, adv = (torch.from_numpy(np.concatenate(v)).cuda() for v in (logp, old, adv))
    off = [0, logp.shape[0]]
    x = dict(logp=logp, old=old, ref=None, ent=None, adv=adv, mask=None)
    r = _run_and_check(x, off, lo, hi, dual, 0.0, 0.0, "token_mean", True)
    share = float(r[1][3])
    assert 0.2 < share < 0.8  # both sides are met


def test_small_and_large_differences():
    # the KL term near 0 would cancel; ratios that overflow stay where they belong
    x0 = torch.tensor([0.0, 1e-7, -1e-5, 1e-3, -0.02, 0.3, 0.4999, -0.5, 0.7, -3.0, 5.0], device="cuda")
    n = x0.shape[0]
    off = [0, n]
    logp = torch.zeros(n, device="cuda")
    z = torch.zeros(n, device="cuda")
    loss, stats, w = dk.policy_loss(logp, z, z, off, ref_logp=x0, kl_coef=1.0, reduction="seq_sum", per_token=True)
    for i in range(n):
        l1, s1, w1 = dk.policy_loss(logp[i:i + 1], z[:1], z[:1], [0, 1], ref_logp=x0[i:i + 1], kl_coef=1.0)
        v = float(x0[i])
        want = opl.token_terms(0.0, 0.0, v, 0.0, 0.2, 0.2, 0.0)
        assert abs(float(s1[1]) - want[3]) <= 8 * U * (want[3] + (abs(v) if abs(v) >= 0.5 else 0.0))
        g, _ = dk.policy_loss_backward(logp[i:i + 1], z[:1], z[:1], [0, 1], torch.ones(1, device="cuda"), w1,
                                       ref_logp=x0[i:i + 1], kl_coef=1.0)
        assert abs(float(g) - want[4]) <= 8 * U * abs(want[4])
    big = torch.tensor([200.0, 200.0, -200.0, 200.0], device="cuda")
    adv = torch.tensor([1.0, 0.0, -1.0, -1.0], device="cuda")
    old = torch.zeros(4, device="cuda")
    loss, stats, w = dk.policy_loss(big, old, adv, [0, 4], per_token=True, dual_clip=3.0)
    assert abs(float(loss) - (-1.2 + 0.0 + 0.8 + 3.0) / 4) < 1e-6
    g, _ = dk.policy_loss_backward(big, old, adv, [0, 4], loss, w, per_token=True, dual_clip=3.0)
    assert not g.any()


def test_pointers_that_start_anywhere_and_repeats():
    off = [0, 700, 705, 4000]
    x = _inputs(off, 21, True, 0.2)
    want = _run_and_check(x, off, 0.2, 0.28, 0.0, 0.05, 0.01, "seq_mean", True)
    shifted = {}
    for i, (k, v) in enumerate(x.items()):
        t = torch.empty(v.shape[0] + 7, dtype=v.dtype, device="cuda")[i + 1:][:v.shape[0]]
        shifted[k] = t.copy_(v)
    got = _run_and_check(shifted, off, 0.2, 0.28, 0.0, 0.05, 0.01, "seq_mean", True)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


def test_streams_and_graphs_that_share_a_workspace():
    off = [0, 3000, 3001, 9000]
    N, n = 3, 9000
    x = _inputs(off, 22, False, 0.2)
    args = (N, off, 0.2, 0.28, 3.0, 0.05, 0.01)
    want = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["ref"], x["ent"], x["mask"], *args[2:])
    one = torch.ones(1, device="cuda")
    want += dk.policy_loss_backward(x["logp"], x["old"], x["adv"], off, one, want[2], x["ref"], x["mask"], *args[2:])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = dk.policy_loss(x["logp"], x["old"], x["adv"], off, x["ref"], x["ent"], x["mask"], *args[2:], stream=side)
    got += dk.policy_loss_backward(x["logp"], x["old"], x["adv"], off, one, got[2], x["ref"], x["mask"], *args[2:],
                                   stream=side)
    side.synchronize()
    for a, b in zip(want, got):
        assert torch.equal(a, b)
    outs = [torch.zeros_like(t) for t in want]
    ws = torch.empty(dk.dualkv_policy_loss_workspace_bytes(N, off), dtype=torch.uint8, device="cuda")
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for graph in graphs:
        with torch.cuda.graph(graph):
            dk.dualkv_policy_loss(x["logp"], x["old"], x["ref"], x["ent"], x["adv"], x["mask"], *args, "token_mean",
                                  outs[0], outs[1], outs[2], ws)
            dk.dualkv_policy_loss_bwd(x["logp"], x["old"], x["ref"], x["adv"], x["mask"], *args, "token_mean", one, outs[2],
                                      outs[3], outs[4])
    for graph in graphs + graphs:
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, outs):
            assert torch.equal(a, b)


def test_binding_refuses_what_does_not_fit():
    off = [0, 3, 5]
    x = _inputs(off, 1, False, None)

    def call(**kw):
        a = dict(old_logp=x["old"], advantages=x["adv"], R_offsets=off, ref_logp=x["ref"], kl_coef=0.1)
        a.update(kw)
        return dk.policy_loss(x["logp"], **a)

    call()
    for bad in (dict(old_logp=x["old"][:-1]), dict(old_logp=x["old"].double()), dict(ref_logp=None), dict(entropy_coef=0.1),
                dict(reduction="mean"), dict(advantages=x["old"][:4]), dict(mask=x["old"]), dict(advantages=x["adv"].cpu()),
                dict(advantages=x["old"], per_token=False)):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(clip_low=1.0), dict(clip_low=-0.1), dict(clip_high=float("nan")), dict(dual_clip=1.0),
                dict(dual_clip=-3.0), dict(kl_coef=float("inf"))):
        with pytest.raises(dk.DualKVError):
            call(**bad)
    # three values for three segments of three tokens: which of the two has to be said
    t = torch.ones(3, device="cuda")
    with pytest.raises(ValueError, match="per_token"):
        dk.policy_loss(t, t, t, [0, 2, 2, 3])
    dk.policy_loss(t, t, t, [0, 2, 2, 3], per_token=True)
    dk.policy_loss(t, t, t, [0, 1, 2, 3])
