"""The per-token operators together with the attention, as a policy update uses them.

One attention layer between a fused projection and an output head, on packed rows:
projection -> qk_norm_rope -> dualkv attention -> output projection + residual -> logits of rows
P - 1 .. T - 1 -> token_logprobs -> policy_loss, and all the way back.  The reference is
fp64 autograd on the N replicated sequences, each with its own copy of the prompt, from the
operators' definitions alone.  Gradients are compared normwise with the 2e-2 that the
attention's own gradients are held to: every tensor between two operators is rounded to
bf16 (at most 2^-8 of a value, about a dozen times on the way), the log-probabilities to
5e-2 absolute (logits of size 3 rounded to bf16: 2^-7 each for the target and for the sum, behind
values that carry the rounding of the layers before).
"""
import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


class Case:
    def __init__(self, P, R, Hq, Hkv, D, V, E=192, seed=0):
        self.P, self.R, self.Hq, self.Hkv, self.D, self.V, self.E = P, R, Hq, Hkv, D, V, E
        self.off = [0]
        for r in R:
            self.off.append(self.off[-1] + r)
        self.n, self.N, self.T = self.off[-1], len(R), P + self.off[-1]
        g = torch.Generator(device="cuda").manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.x = rn(self.T, E).to(BF)
        self.w = dict(qkv=(rn(E, (Hq + 2 * Hkv) * D) / E ** 0.5).to(BF), o=(rn(Hq * D, E) / (Hq * D) ** 0.5).to(BF),
                      head=(rn(E, V) * 1.5 / E ** 0.5).to(BF), qn=1 + 0.2 * rn(D), kn=1 + 0.2 * rn(D))
        self.f = (1e4 ** (-torch.arange(D // 2, device="cuda") * 2.0 / D)).float()
        self.tok = torch.randint(0, V, (self.n,), generator=g, device="cuda")
        self.mask = torch.rand(self.n, generator=g, device="cuda") > 0.2
        self.noise = 0.3 * rn(2, self.n)
        self.adv = rn(self.N)
        self.kw = dict(clip_low=0.2, clip_high=0.28, kl_coef=0.05, entropy_coef=0.01)


def _reference(c, old, ref):
    """Token log-probabilities and gradients of fp64 autograd on the replicated sequences."""
    w = {k: v.double().cpu().requires_grad_() for k, v in c.w.items()}
    x = c.x.double().cpu().requires_grad_()
    f, tok, mask, adv, old, ref = (t.cpu() for t in (c.f.double(), c.tok, c.mask, c.adv.double(), old.double(),
                                                      ref.double()))
    half = c.D // 2
    parts, entropies = [], []
    for s in range(c.N):
        rows = torch.cat((torch.arange(c.P), c.P + torch.arange(c.off[s], c.off[s + 1])))
        L = rows.numel()
        h = x[rows]
        q, k, v = (h @ w["qkv"]).split((c.Hq * c.D, c.Hkv * c.D, c.Hkv * c.D), 1)
        a = torch.arange(L).double()[:, None] * f

        def norm_turn(t, H, g):
            t = t.reshape(L, H, c.D)
            t = t * (t.square().mean(-1, keepdim=True) + EPS).rsqrt() * g
            cos, sin = a.cos()[:, None], a.sin()[:, None]
            u, z = t[..., :half], t[..., half:]
            return torch.cat((u * cos - z * sin, z * cos + u * sin), -1)

        q, k = norm_turn(q, c.Hq, w["qn"]), norm_turn(k, c.Hkv, w["kn"])
        k = k.repeat_interleave(c.Hq // c.Hkv, 1)
        v = v.reshape(L, c.Hkv, c.D).repeat_interleave(c.Hq // c.Hkv, 1)
        S = torch.einsum("qhd,khd->hqk", q, k) / c.D ** 0.5
        S = S.masked_fill(torch.ones(L, L).triu(1).bool(), -float("inf"))
        o = torch.einsum("hqk,khd->qhd", S.softmax(-1), v).reshape(L, -1)
        lp = torch.log_softmax((h + o @ w["o"])[c.P - 1:L - 1] @ w["head"], -1)
        parts.append(lp.gather(1, tok[c.off[s]:c.off[s + 1], None])[:, 0])
        entropies.append(-(lp.exp() * lp).sum(-1))
    logp, ent = torch.cat(parts), torch.cat(entropies)
    A = torch.repeat_interleave(adv, torch.tensor(c.R))
    ratio = (logp - old).exp()
    pg = -torch.minimum(ratio * A, ratio.clamp(1 - c.kw["clip_low"], 1 + c.kw["clip_high"]) * A)
    d = ref - logp
    per = pg + c.kw["kl_coef"] * (d.exp() - d - 1) - c.kw["entropy_coef"] * ent
    loss = torch.zeros((), dtype=torch.float64)
    for s in range(c.N):
        m = mask[c.off[s]:c.off[s + 1]]
        if m.any():
            loss = loss + per[c.off[s]:c.off[s + 1]][m].mean() / c.N
    loss.backward()
    return logp.detach(), x.grad, {k: v.grad for k, v in w.items()}


def _forward(c):
    s = {}
    s["qkv"] = c.x @ c.w["qkv"]
    a, b = c.Hq * c.D, (c.Hq + c.Hkv) * c.D
    s["q0"], s["k0"] = s["qkv"][:, :a].view(c.T, c.Hq, c.D), s["qkv"][:, a:b].view(c.T, c.Hkv, c.D)
    s["v"] = s["qkv"][:, b:].contiguous().view(c.T, c.Hkv, c.D)
    s["q"], s["k"] = dk.qk_norm_rope(s["q0"], s["k0"], c.P, c.off, c.f, c.w["qn"], c.w["kn"], eps=EPS)
    s["o"], s["lse"] = dk.forward(s["q"], s["k"], s["v"], c.P, c.off)
    s["h"] = (c.x + s["o"].view(c.T, -1) @ c.w["o"])[c.P - 1:]
    s["logits"] = s["h"] @ c.w["head"]
    s["logp"], s["ent"], s["tlse"] = dk.token_logprobs(s["logits"], c.tok, c.P, c.off, entropy=True)
    return s


def _step(c, s, old, ref):
    loss, stats, weights = dk.policy_loss(s["logp"], old, c.adv, c.off, ref, s["ent"], c.mask, reduction="seq_mean", **c.kw)
    one = torch.ones(1, device="cuda")
    dlogp, dent = dk.policy_loss_backward(s["logp"], old, c.adv, c.off, one, weights, ref, c.mask, **c.kw)
    dlogits = dk.token_logprobs_backward(s["logits"], c.tok, s["tlse"], dlogp, c.P, c.off, entropy=s["ent"], dentropy=dent,
                                         inplace=True)
    g = dict(head=s["h"].T @ dlogits)
    dh = torch.zeros(c.T, c.E, dtype=BF, device="cuda")
    dh[c.P - 1:] = dlogits @ c.w["head"].T
    g["o"] = s["o"].view(c.T, -1).T @ dh
    do = (dh @ c.w["o"].T).view(c.T, c.Hq, c.D)
    dq, dkk, dv = dk.backward(s["q"], s["k"], s["v"], s["o"], s["lse"], do, c.P, c.off)
    dq0, dk0, g["qn"], g["kn"] = dk.qk_norm_rope_backward(s["q0"], s["k0"], dq, dkk, c.P, c.off, c.f, c.w["qn"], c.w["kn"],
                                                          eps=EPS)
    dqkv = torch.cat([t.view(c.T, -1) for t in (dq0, dk0, dv)], 1)
    g["qkv"] = c.x.T @ dqkv
    return loss, dh + dqkv @ c.w["qkv"].T, g


CASES = [
    ("ragged", Case, dict(P=70, R=[33, 0, 5, 120], Hq=4, Hkv=2, D=64, V=501)),
    ("wide", Case, dict(P=1, R=[40, 1], Hq=2, Hkv=1, D=128, V=257, seed=1)),
]


@pytest.mark.parametrize("name,make,kw", CASES, ids=[c[0] for c in CASES])
def test_policy_step_matches_replicated_sequences(name, make, kw):
    c = make(**kw)
    s = _forward(c)
    # the sampling policy and the reference model scored the same tokens a little differently
    old, ref = s["logp"] + c.noise[0], s["logp"] + c.noise[1]
    _, dx, g = _step(c, s, old, ref)
    dk.dualkv_check_status()
    want_logp, want_dx, want = _reference(c, old, ref)
    assert float((s["logp"].double().cpu() - want_logp).abs().max()) <= 5e-2
    rel = lambda a, b: float((a.double().cpu() - b).norm() / b.norm())  # noqa: E731
    assert rel(dx, want_dx) <= 2e-2
    for k, v in want.items():
        assert rel(g[k], v) <= 2e-2, (k, rel(g[k], v))
