"""Performance cases of the packed policy update's operators around attention.

Three operators, each with its backward pass, on the packed layout of one
prompt of P tokens and N response segments:

  rope   per-head RMS norm of q and k with the position rotation
  logp   log-probabilities (and entropies) of the response tokens from logits
  loss   clipped policy loss with a KL term and an entropy bonus

``own`` selects what ``run`` calls: False computes the plain form from
elementary torch operations, True calls this package's kernels.
"""
import ctypes
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ layouts
def _lengths(c):
    """Response lengths of a case: equal, or ragged from the case's own seed, some of them zero."""
    if c["r_lo"] == c["r_hi"]:
        r = [c["r_lo"]] * c["N"]
    else:
        r = np.random.default_rng(c["r_seed"]).integers(c["r_lo"], c["r_hi"] + 1, c["N"]).tolist()
    for n in range(c["empty"]):
        r[(3 * n + 1) % c["N"]] = 0
    if not any(r):
        r[0] = 1
    return r


def _offsets(c):
    return [0] + np.cumsum(_lengths(c)).tolist()


def _positions(P, off):
    pos = [torch.arange(P)]
    pos += [P + torch.arange(b - a) for a, b in zip(off, off[1:])]
    return torch.cat(pos).to(torch.int64).to(DEV)


def _segments(off):
    n = torch.arange(len(off) - 1)
    return torch.repeat_interleave(n, torch.tensor(off).diff()).to(DEV)


def _predictor(P, off):
    """Logits row that predicts each response token; -1 where no row does."""
    rows = torch.arange(off[-1]) - (1 if P == 0 else 0)
    first = torch.tensor([a for a, b in zip(off, off[1:]) if b > a], dtype=torch.int64)
    rows[first] = 0 if P > 0 else -1
    return rows.to(DEV)


# -------------------------------------------------------------------- cases
def _rope(name, dir, P, N, r_lo, r_hi, Hq, Hkv, D, rope_dim, interleaved=False, fused=False, w="bf16", w0=0.0, r_seed=1,
          empty=0, base=1e6):
    return dict(name=name, op="rope", dir=dir, P=P, N=N, r_lo=r_lo, r_hi=r_hi, r_seed=r_seed, empty=empty, Hq=Hq, Hkv=Hkv,
                D=D, rope_dim=rope_dim, interleaved=interleaved, fused=fused, weights=w, w0=w0, base=base)


def _logp(name, dir, P, N, r_lo, r_hi, V, dtype, entropy, ignored=0.0, pad=0, masked=0, scale=1.0, r_seed=2, empty=0):
    return dict(name=name, op="logp", dir=dir, P=P, N=N, r_lo=r_lo, r_hi=r_hi, r_seed=r_seed, empty=empty, V=V, dtype=dtype,
                entropy=entropy, ignored=ignored, pad=pad, masked=masked, scale=scale)


def _loss(name, dir, N, r_lo, r_hi, reduction, per_token, masked, kl, ent, dual=0.0, lo=0.2, hi=0.2, r_seed=3, empty=0):
    return dict(name=name, op="loss", dir=dir, P=0, N=N, r_lo=r_lo, r_hi=r_hi, r_seed=r_seed, empty=empty,
                reduction=reduction, per_token=per_token, masked=masked, kl=kl, ent=ent, dual=dual, lo=lo, hi=hi)


def listed():
    return [
        # the package's smallest workload: one prompt of 64, four responses of 32, D = 64; launch latency is all of it
        _rope("rope fwd tiny", "fwd", 64, 4, 32, 32, 2, 2, 64, 64, w="f32"),
        # the GRPO layer of the benchmark (32 responses of 2048 behind a prompt of 6144), q and k read out of the fused
        # projection's rows
        _rope("rope fwd grpo", "fwd", 6144, 32, 2048, 2048, 32, 8, 128, 128, fused=True),
        # ragged DAPO-like responses, gradients of a training step written into the fused projection's gradient
        _rope("rope bwd ragged", "bwd", 8192, 32, 257, 4096, 32, 8, 128, 128, fused=True, w="f32", r_seed=20260518),
        # wide heads of a global layer, a quarter of each head rotated, weights stored as their distance from one
        _rope("rope bwd wide heads", "bwd", 16384, 16, 1001, 1500, 8, 2, 512, 128, interleaved=True, w0=1.0, base=1e4),
        # scoring a handful of short answers: few rows, so one row has to be spread over many SMs
        _logp("logp fwd short", "fwd", 512, 4, 1, 3, 50001, "f32", False),
        # scoring pass over a long micro-batch; more than 2^31 logits
        _logp("logp fwd long", "fwd", 2048, 8, 1850, 2550, 131072, "bf16", True, scale=1.25),
        # fp32 logits of an odd vocabulary, prompt-like stretches of the responses ignored, one response empty
        _logp("logp bwd odd", "bwd", 100, 6, 300, 900, 32001, "f32", False, ignored=0.25, empty=1),
        # training step with an entropy bonus; rows of a padded vocabulary whose padding is masked
        _logp("logp bwd long", "bwd", 2048, 8, 900, 1900, 131072, "bf16", True, ignored=0.05, pad=64, masked=128),
        # four responses of 32 tokens: latency
        _loss("loss fwd tiny", "fwd", 4, 32, 32, "seq_mean", False, 0.0, 0.04, 0.0),
        # a large rollout batch in one reduction: token mean, ragged, per-token advantages, masked tokens
        _loss("loss fwd large", "fwd", 1024, 1000, 7000, "token_mean", True, 0.1, 0.001, 0.01, dual=3.0, hi=0.28),
        # the GRPO micro-batch: 32 responses of 2048, sequence mean, one advantage per response
        _loss("loss bwd grpo", "bwd", 32, 2048, 2048, "seq_mean", False, 0.05, 0.04, 0.0),
        # the large batch's gradients
        _loss("loss bwd large", "bwd", 1024, 1000, 7000, "token_mean", True, 0.1, 0.001, 0.01, dual=3.0, hi=0.28, empty=2),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_layout(rng, tokens, most_n, prompt=True):
    """P, N, r_lo, r_hi, r_seed, empty of a layout with about `tokens` rows."""
    P = int(tokens * rng.uniform(0.0, 0.6)) if prompt else 0
    rest = max(1, tokens - P)
    N = min(_log_int(rng, 1, most_n), rest)
    mean = max(1, rest // N)
    ragged = rng.random() < 0.7
    lo, hi = (max(0, mean // 2), max(1, mean + mean // 2)) if ragged else (mean, mean)
    return dict(P=P, N=N, r_lo=lo, r_hi=hi, r_seed=rng.randrange(1 << 20), empty=rng.choice([0, 0, 1]) if N > 1 else 0)


def draw(rng):
    op = rng.choice(["rope", "logp", "loss"])
    dir = rng.choice(["fwd", "bwd"])
    if op == "rope":
        D = rng.choice([64, 128, 128, 512])
        Hkv = rng.choice([1, 2, 3, 4, 8])
        Hq = Hkv * rng.choice([1, 2, 4, 5, 8])
        most = max(2, min(60000, 250_000_000 // ((Hq + Hkv) * D)))
        lay = _draw_layout(rng, _log_int(rng, 1, most), 64)
        return dict(op=op, dir=dir, **lay, Hq=Hq, Hkv=Hkv, D=D, rope_dim=rng.choice([16, D // 2, D, D]),
                    interleaved=rng.random() < 0.3, fused=rng.random() < 0.5, weights=rng.choice(["bf16", "f32", "none"]),
                    w0=rng.choice([0.0, 1.0]), base=rng.choice([1e4, 1e6]))
    if op == "logp":
        dtype = rng.choice(["bf16", "bf16", "f32"])
        V = _log_int(rng, 500, 160000)
        most = max(2, min(20000, (1_000_000_000 if dtype == "bf16" else 500_000_000) // V))
        lay = _draw_layout(rng, _log_int(rng, 1, most), 64, prompt=False)
        # without a prompt a segment's first token has no row that predicts it: leave that to batches of some size
        few = lay["N"] * lay["r_hi"] < 100 * (1 + lay["N"])
        lay["P"] = rng.choice([1, 77, 4096] if few else [0, 1, 77, 4096])
        masked = rng.choice([0, 0, rng.randrange(1, V // 8)])
        return dict(op=op, dir=dir, **lay, V=V, dtype=dtype, entropy=rng.random() < 0.5, ignored=0.0 if few else rng.choice([0.0, 0.1, 0.5]),
                    pad=rng.choice([0, 0, rng.randrange(1, 130)]), masked=masked, scale=rng.choice([1.0, 0.7, 1.25]))
    tokens = _log_int(rng, 4, 2_500_000)
    lay = _draw_layout(rng, tokens, 1500, prompt=False)
    return dict(op=op, dir=dir, **lay, reduction=rng.choice(["token_mean", "seq_mean", "seq_sum"]),
                per_token=rng.random() < 0.5, masked=0.0 if tokens < 100 else rng.choice([0.0, 0.1, 0.5]), kl=rng.choice([0.0, 0.001, 0.04]),
                ent=rng.choice([0.0, 0.01]), dual=rng.choice([0.0, 3.0]), lo=rng.choice([0.1, 0.2]), hi=rng.choice([0.2, 0.28]))


# ------------------------------------------------------------------ prepare
def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 17)
    off = _offsets(case)
    s = dict(c=case, off=off, c_off=(ctypes.c_int32 * len(off))(*off))
    return {"rope": _prepare_rope, "logp": _prepare_logp, "loss": _prepare_loss}[case["op"]](case, g, s)


def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _qk_rows(c, T, make):
    """q [T, Hq, D] and k [T, Hkv, D]: views of one fused [T, (Hq + 2 Hkv) D] tensor, or tensors of their own."""
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    if not c["fused"]:
        return make(T, Hq * D).view(T, Hq, D), make(T, Hkv * D).view(T, Hkv, D)
    row = make(T, (Hq + 2 * Hkv) * D)
    return row[:, :Hq * D].view(T, Hq, D), row[:, Hq * D:(Hq + Hkv) * D].view(T, Hkv, D)


def _prepare_rope(c, g, s):
    T, D, bf = c["P"] + s["off"][-1], c["D"], torch.bfloat16
    s["q"], s["k"] = _qk_rows(c, T, lambda *shape: _randn(g, *shape, dtype=bf))
    s["pos"] = _positions(c["P"], s["off"])
    j = torch.arange(c["rope_dim"] // 2, dtype=torch.float64, device=DEV)
    s["inv_freq"] = (c["base"] ** (-2.0 * j / c["rope_dim"])).float()
    s["qw"] = s["kw"] = None
    if c["weights"] != "none":
        wt = {"bf16": bf, "f32": torch.float32}[c["weights"]]
        s["qw"], s["kw"] = ((1.0 - c["w0"] + 0.2 * _randn(g, D)).to(wt) for _ in range(2))
    if c["dir"] == "fwd":
        s["q_out"] = torch.empty(T, c["Hq"], D, dtype=bf, device=DEV)
        s["k_out"] = torch.empty(T, c["Hkv"], D, dtype=bf, device=DEV)
        return s
    s["dq_out"], s["dk_out"] = _randn(g, T, c["Hq"], D, dtype=bf), _randn(g, T, c["Hkv"], D, dtype=bf)
    s["dq"], s["dk"] = _qk_rows(c, T, lambda *shape: torch.empty(*shape, dtype=bf, device=DEV))
    s["dqw"] = s["dkw"] = None
    if s["qw"] is not None:
        s["dqw"], s["dkw"] = (torch.empty(D, device=DEV) for _ in range(2))
    # enough for any layout: two fp32 rows of D for each of a few thousand thread blocks
    s["ws"] = torch.empty(32 << 20, dtype=torch.uint8, device=DEV)
    return s


def _prepare_logp(c, g, s):
    P, n, V = c["P"], s["off"][-1], c["V"]
    M = n + (1 if P > 0 else 0)
    dt = {"bf16": torch.bfloat16, "f32": torch.float32}[c["dtype"]]
    s["rows"] = _predictor(P, s["off"])
    full = _randn(g, M, V + c["pad"], dtype=dt).mul_(2.5)
    s["logits"] = full[:, :V]
    if c["masked"]:
        s["logits"][:, V - c["masked"]:] = -math.inf
    tok = torch.randint(0, V - c["masked"], (n,), generator=g, device=DEV)
    here = s["rows"] >= 0
    # a trained model gives most of its tokens a high probability
    s["logits"][s["rows"][here], tok[here]] = (8.0 + 3.0 * _randn(g, n))[here].to(dt)
    if c["ignored"]:
        tok[torch.rand(n, generator=g, device=DEV) < c["ignored"]] = -100
    s["tokens"] = tok
    f32 = dict(dtype=torch.float32, device=DEV)
    if c["dir"] == "fwd":
        s["logp"], s["lse"] = torch.empty(n, **f32), torch.empty(M, **f32)
        s["entropy"] = torch.empty(n, **f32) if c["entropy"] else None
        return s
    # what the forward pass left: the rows' log-sum-exp and the tokens' entropies
    s["lse"], ent = torch.empty(M, **f32), torch.empty(M, **f32)
    for a in range(0, M, 1024):
        z = s["logits"][a:a + 1024].float() * c["scale"]
        lse = torch.logsumexp(z, 1)
        s["lse"][a:a + 1024] = lse
        if c["entropy"]:
            p = torch.exp(z - lse[:, None])
            ent[a:a + 1024] = lse - torch.where(p > 0, p * z, torch.zeros_like(p)).sum(1)
    live = here & (tok >= 0)
    dead = torch.ones(M, dtype=torch.bool, device=DEV)
    dead[s["rows"][live]] = False
    s["lse"][dead] = 0.0
    s["entropy"] = s["dentropy"] = None
    if c["entropy"]:
        s["entropy"] = torch.where(live, ent[s["rows"].clamp(min=0)], torch.zeros_like(s["rows"], dtype=torch.float32))
        s["dentropy"] = torch.full((n,), -0.01 / max(n, 1), **f32)
    s["dlogp"] = _randn(g, n) / max(n, 1)
    s["dlogits"] = torch.empty(M, V + c["pad"], dtype=dt, device=DEV)[:, :V]
    return s


def _prepare_loss(c, g, s):
    n, N = s["off"][-1], c["N"]
    s["seg"] = _segments(s["off"])
    s["logp"] = -_randn(g, n).abs_()
    s["old"] = s["logp"] + 0.15 * _randn(g, n)
    s["ref"] = s["logp"] + 0.3 * _randn(g, n) if c["kl"] else None
    s["entropy"] = _randn(g, n).abs_() if c["ent"] else None
    s["adv"] = _randn(g, n if c["per_token"] else N)
    s["mask"] = None
    if c["masked"]:
        s["mask"] = torch.rand(n, generator=g, device=DEV) >= c["masked"]
    f32 = dict(dtype=torch.float32, device=DEV)
    s["weights"] = torch.empty(N, **f32)
    if c["dir"] == "fwd":
        s["loss"], s["stats"] = torch.empty(1, **f32), torch.empty(4, **f32)
        s["ws"] = torch.empty((N + n // 1024 + 16) * 64, dtype=torch.uint8, device=DEV)
        return s
    s["weights"].copy_(_weights_plain(s))  # what the forward pass left
    s["dloss"] = torch.full((), 0.5, **f32) + 0.1 * _randn(g, ())
    s["dlogp"] = torch.empty(n, **f32)
    s["dentropy"] = torch.empty(n, **f32) if c["ent"] else None
    return s


# ---------------------------------------------------------------------- run
def run(s):
    c = s["c"]
    return {("rope", "fwd"): _rope_fwd, ("rope", "bwd"): _rope_bwd, ("logp", "fwd"): _logp_fwd, ("logp", "bwd"): _logp_bwd,
            ("loss", "fwd"): _loss_fwd, ("loss", "bwd"): _loss_bwd}[c["op"], c["dir"]](c, s)


EPS = 1e-6


def _rotation_plain(c, s):
    """cos and sin of every row's angles, [T, 1, rope_dim / 2]: the angle in 64 bits, its cosine in 32."""
    a = s["pos"].double()[:, None] * s["inv_freq"].double()
    return a.cos().float()[:, None], a.sin().float()[:, None]


def _rotate_plain(c, x, cos, sin):
    r = c["rope_dim"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _rope_fwd(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_qk_norm_rope(s["q"], s["k"], s["qw"], s["kw"], c["w0"], EPS, s["inv_freq"], c["rope_dim"],
                                   c["interleaved"], c["P"], c["N"], s["c_off"], c["Hq"], c["Hkv"], c["D"], s["q_out"],
                                   s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    cos, sin = _rotation_plain(c, s)

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.float() + c["w0"])
        return _rotate_plain(c, x, cos, sin).to(torch.bfloat16)

    return {"q": one(s["q"], s["qw"]), "k": one(s["k"], s["kw"])}


def _rope_bwd(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_qk_norm_rope_bwd(s["q"], s["k"], s["dq_out"], s["dk_out"], s["qw"], s["kw"], c["w0"], EPS,
                                       s["inv_freq"], c["rope_dim"], c["interleaved"], c["P"], c["N"], s["c_off"], c["Hq"],
                                       c["Hkv"], c["D"], s["dq"], s["dk"], s["dqw"], s["dkw"], s["ws"])
        return {"dq": s["dq"], "dk": s["dk"], "dqw": s["dqw"], "dkw": s["dkw"]}
    cos, sin = _rotation_plain(c, s)

    def one(x, dy, w):
        dn = _rotate_plain(c, dy.float(), cos, -sin)
        if w is None:
            return dn.to(torch.bfloat16), None
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
        xh = x * r
        dw = (dn * xh).sum((0, 1), dtype=torch.float64).float()
        u = dn * (w.float() + c["w0"])
        dx = r * (u - xh * (u * xh).mean(-1, keepdim=True))
        return dx.to(torch.bfloat16), dw

    dq, dqw = one(s["q"], s["dq_out"], s["qw"])
    dk, dkw = one(s["k"], s["dk_out"], s["kw"])
    return {"dq": dq, "dk": dk, "dqw": dqw, "dkw": dkw}


def _live_rows(s, M):
    """Rows that predict at least one token which is not ignored."""
    on = (s["rows"] >= 0) & (s["tokens"] >= 0)
    live = torch.zeros(M, dtype=torch.float32, device=DEV)
    live.index_fill_(0, s["rows"][on], 1.0)
    return on, live > 0


def _logp_fwd(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_token_logprobs(s["logits"], s["tokens"], c["scale"], c["P"], c["N"], s["c_off"], s["logp"],
                                     s["entropy"], s["lse"])
        return {"logp": s["logp"], "entropy": s["entropy"], "lse": s["lse"]}
    z = s["logits"].float() * c["scale"]
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1)
    on, live = _live_rows(s, z.shape[0])
    lse = m[:, 0] + total.log()
    row, tok = s["rows"].clamp(min=0), s["tokens"].clamp(min=0)
    zero = torch.zeros_like(row, dtype=torch.float32)
    logp = torch.where(on, z[row, tok] - lse[row], zero)
    ent = None
    if c["entropy"]:
        ent = lse - torch.where(e > 0, e * z, torch.zeros_like(z)).sum(1) / total
        ent = torch.where(on, ent[row], zero)
    return {"logp": logp, "entropy": ent, "lse": torch.where(live, lse, torch.zeros_like(lse))}


def _logp_bwd(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_token_logprobs_bwd(s["logits"], s["tokens"], c["scale"], c["P"], c["N"], s["c_off"], s["lse"],
                                         s["entropy"], s["dlogp"], s["dentropy"], s["dlogits"])
        return s["dlogits"]
    M = s["lse"].shape[0]
    on, live = _live_rows(s, M)
    row, tok = s["rows"][on], s["tokens"][on]
    g = torch.zeros(M, dtype=torch.float32, device=DEV).index_add_(0, row, s["dlogp"][on])
    lp = s["logits"].float() * c["scale"] - s["lse"][:, None]
    p = torch.exp(lp)
    dz = -g[:, None] * p
    if c["entropy"]:
        h = torch.zeros(M, dtype=torch.float32, device=DEV).index_add_(0, row, s["dentropy"][on])
        ent = torch.zeros(M, dtype=torch.float32, device=DEV)
        ent[row] = s["entropy"][on]
        dz -= h[:, None] * torch.where(p > 0, p * (lp + ent[:, None]), torch.zeros_like(p))
    dz.index_put_((row, tok), s["dlogp"][on], accumulate=True)
    dz = torch.where(live[:, None], dz * c["scale"], torch.zeros_like(dz))
    return dz.to(s["logits"].dtype)


def _mask_plain(s):
    return torch.ones_like(s["seg"], dtype=torch.bool) if s["mask"] is None else s["mask"]


def _weights_plain(s):
    """Weight of a live token of each segment in the loss."""
    c, N = s["c"], s["c"]["N"]
    n = torch.zeros(N, dtype=torch.float64, device=DEV).index_add_(0, s["seg"], _mask_plain(s).double())
    if c["reduction"] == "token_mean":
        return torch.where(n > 0, 1.0 / n.sum().clamp(min=1), torch.zeros_like(n)).float()
    if c["reduction"] == "seq_mean":
        return torch.where(n > 0, 1.0 / (N * n.clamp(min=1)), torch.zeros_like(n)).float()
    return torch.where(n > 0, 1.0 / N, torch.zeros_like(n)).float()


def _loss_args(c, s):
    return (c["N"], s["c_off"], c["lo"], c["hi"], c["dual"], c["kl"], c["ent"], c["reduction"])


def _terms_plain(c, s):
    """Each token's policy term, KL term and clip flag, in 64 bits: the clipping borders decide on close values."""
    adv = s["adv"].double() if c["per_token"] else s["adv"].double()[s["seg"]]
    ratio = torch.exp(s["logp"].double() - s["old"].double())
    up = torch.where(adv > 0, ratio > 1.0 + c["hi"], torch.zeros_like(s["seg"], dtype=torch.bool))
    down = torch.where(adv < 0, ratio < 1.0 - c["lo"], torch.zeros_like(up))
    far = torch.where(adv < 0, ratio > c["dual"], torch.zeros_like(up)) if c["dual"] else torch.zeros_like(up)
    bounded = torch.where(up, torch.full_like(ratio, 1.0 + c["hi"]), ratio)
    bounded = torch.where(down, torch.full_like(ratio, 1.0 - c["lo"]), bounded)
    bounded = torch.where(far, torch.full_like(ratio, c["dual"]), bounded)
    x = s["ref"].double() - s["logp"].double() if c["kl"] else None
    return adv, ratio, bounded, up | down | far, x


def _loss_fwd(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_policy_loss(s["logp"], s["old"], s["ref"], s["entropy"], s["adv"], s["mask"], *_loss_args(c, s),
                                  s["loss"], s["stats"], s["weights"], s["ws"])
        return {"loss": s["loss"], "stats": s["stats"], "weights": s["weights"]}
    on = _mask_plain(s)
    adv, ratio, bounded, clipped, x = _terms_plain(c, s)
    weights = _weights_plain(s)
    w = torch.where(on, weights.double()[s["seg"]], torch.zeros_like(ratio))
    zero = torch.zeros((), dtype=torch.float64, device=DEV)
    policy = (w * (-adv * bounded)).sum()
    kl = (w * (torch.exp(x) - x - 1.0)).sum() if c["kl"] else zero
    ent = (w * s["entropy"].double()).sum() if c["ent"] else zero
    count = on.double().sum()
    share = (clipped & on).double().sum() / count.clamp(min=1)
    loss = policy + c["kl"] * kl - c["ent"] * ent
    return {"loss": loss.float()[None], "stats": torch.stack((policy, kl, ent, share)).float(), "weights": weights}


def _loss_bwd(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_policy_loss_bwd(s["logp"], s["old"], s["ref"], s["adv"], s["mask"], *_loss_args(c, s), s["dloss"],
                                      s["weights"], s["dlogp"], s["dentropy"])
        return {"dlogp": s["dlogp"], "dentropy": s["dentropy"]}
    on = _mask_plain(s)
    adv, ratio, bounded, clipped, x = _terms_plain(c, s)
    w = torch.where(on, s["weights"].double()[s["seg"]], torch.zeros_like(ratio)) * s["dloss"].double()
    d = torch.where(clipped, torch.zeros_like(ratio), -adv * ratio)
    if c["kl"]:
        d = d - c["kl"] * (torch.exp(x) - 1.0)
    return {"dlogp": (w * d).float(), "dentropy": (-c["ent"] * w).float() if c["ent"] else None}


# --------------------------------------------------------------------- work
def work(case):
    c, off = case, _offsets(case)
    n = off[-1]
    if c["op"] == "rope":
        x = (c["P"] + n) * (c["Hq"] + c["Hkv"]) * c["D"]
        w = 0 if c["weights"] == "none" else 2 * c["D"] * (2 if c["weights"] == "bf16" else 4)
        if c["dir"] == "fwd":
            return {"bytes": 4 * x + w + 2 * c["rope_dim"], "flops": 7 * x}
        return {"bytes": 6 * x + w + 2 * c["rope_dim"] + (8 * c["D"] if w else 0), "flops": 14 * x}
    if c["op"] == "logp":
        e = 2 if c["dtype"] == "bf16" else 4
        M = n + (1 if c["P"] > 0 else 0)
        live = max(1.0, M * (1.0 - c["ignored"]))
        if c["dir"] == "fwd":
            return {"bytes": live * c["V"] * e + 12 * n + 4 * M + (4 * n if c["entropy"] else 0),
                    "flops": live * c["V"] * (6 if c["entropy"] else 4)}
        return {"bytes": (live + M) * c["V"] * e + 12 * n + 4 * M + (8 * n if c["entropy"] else 0),
                "flops": live * c["V"] * (6 if c["entropy"] else 4)}
    inputs = 8 + (4 if c["kl"] else 0) + (4 if c["per_token"] else 0) + (1 if c["masked"] else 0)
    if c["dir"] == "fwd":
        return {"bytes": n * (inputs + (4 if c["ent"] else 0)) + 8 * c["N"] + 24, "flops": 20 * n}
    return {"bytes": n * (inputs + 4 + (4 if c["ent"] else 0)) + 8 * c["N"], "flops": 16 * n}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits: derivatives by automatic differentiation of the
    definition where the operator's inputs are all leaves of it."""
    s = prepare(case, seed)
    return {"rope": _rope_exact, "logp": _logp_exact, "loss": _loss_exact}[case["op"]](case, s)


def _rope_exact(c, s):
    half = c["rope_dim"] // 2
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(s["pos"].double(), s["inv_freq"].double())).unsqueeze(1)

    def forward(x, w):
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * (c["w0"] + w)
        head, tail = x[..., :c["rope_dim"]], x[..., c["rope_dim"]:]
        if c["interleaved"]:
            v = torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) * turn
            head = torch.view_as_real(v).flatten(-2)
        else:
            v = torch.complex(head[..., :half], head[..., half:]) * turn
            head = torch.cat((v.real, v.imag), -1)
        return torch.cat((head, tail), -1)

    out = {}
    for name in ("q", "k"):
        x, w = s[name].double(), s[name + "w"]
        w = None if w is None else w.double()
        if c["dir"] == "fwd":
            out[name] = forward(x, w)
            continue
        x.requires_grad_()
        leaves = [x] if w is None else [x, w.requires_grad_()]
        got = torch.autograd.grad(forward(x, w), leaves, s["d%s_out" % name].double())
        out["d" + name], out["d%sw" % name] = got[0], None if w is None else got[1]
        del x, got
    return out


def _logp_exact(c, s):
    on = (s["rows"] >= 0) & (s["tokens"] >= 0)
    at, tok = s["rows"][on], s["tokens"][on]
    M = s["lse"].shape[0]
    if c["dir"] == "fwd":
        lp = torch.log_softmax(s["logits"].double() * c["scale"], 1)
        logp = torch.zeros(on.shape, dtype=torch.float64, device=DEV)
        logp[on] = lp[at, tok]
        lse = torch.zeros(M, dtype=torch.float64, device=DEV)
        lse[at] = s["logits"][at, tok].double() * c["scale"] - lp[at, tok]
        ent = None
        if c["entropy"]:
            ent = torch.zeros_like(logp)
            ent[on] = torch.special.entr(lp.exp_()).sum(1)[at]
        return {"logp": logp, "entropy": ent, "lse": lse}
    # the gradients for the saved log-sum-exp and entropies as they are given
    lp = s["logits"].double().mul_(c["scale"]).sub_(s["lse"].double()[:, None])
    coef, bonus, ent = (torch.zeros(M, 1, dtype=torch.float64, device=DEV) for _ in range(3))
    coef.index_add_(0, at, s["dlogp"][on].double()[:, None])
    if c["entropy"]:
        bonus.index_add_(0, at, s["dentropy"][on].double()[:, None])
        ent[at] = s["entropy"][on].double()[:, None]
    d = lp.clamp(min=-1e4).add_(ent).mul_(bonus).add_(coef).mul_(lp.exp_()).neg_()
    d.index_put_((at, tok), s["dlogp"][on].double(), accumulate=True)
    dead = torch.ones(M, dtype=torch.bool, device=DEV)
    dead[at] = False
    d[dead] = 0.0
    return d.mul_(c["scale"])


def _loss_exact(c, s):
    on = torch.ones(s["seg"].shape, dtype=torch.bool, device=DEV) if s["mask"] is None else s["mask"]
    seg, N = s["seg"][on], c["N"]
    live = torch.bincount(seg, minlength=N).double()
    if c["dir"] == "fwd":
        per = {"token_mean": live.sum().clamp(min=1).expand(N), "seq_mean": N * live.clamp(min=1),
               "seq_sum": torch.full_like(live, N)}[c["reduction"]]
        weights = (live > 0).double() / per
    else:
        weights = s["weights"].double()
    logp = s["logp"].double()[on].requires_grad_()
    old = s["old"].double()[on]
    adv = s["adv"].double()
    adv = adv[on] if c["per_token"] else adv[seg]
    ratio = (logp - old).exp()
    gain = torch.minimum(ratio * adv, ratio.clamp(1.0 - c["lo"], 1.0 + c["hi"]) * adv)
    if c["dual"]:
        gain = torch.where(adv < 0, torch.maximum(gain, c["dual"] * adv), gain)
    w = weights[seg]
    policy = -(w * gain).sum()
    kl = ent = torch.zeros((), dtype=torch.float64, device=DEV)
    if c["kl"]:
        x = s["ref"].double()[on] - logp
        kl = (w * (torch.expm1(x) - x)).sum()
    if c["ent"]:
        ent = (w * s["entropy"].double()[on]).sum()
    loss = policy + c["kl"] * kl - c["ent"] * ent
    if c["dir"] == "fwd":
        beyond = torch.where(adv > 0, ratio > 1.0 + c["hi"], (adv < 0) & (ratio < 1.0 - c["lo"]))
        if c["dual"]:
            beyond |= (adv < 0) & (ratio > c["dual"])
        stats = torch.stack((policy, kl, ent, beyond.double().sum() / live.sum().clamp(min=1)))
        return {"loss": loss.detach()[None], "stats": stats.detach(), "weights": weights}
    d = torch.zeros(on.shape, dtype=torch.float64, device=DEV)
    if seg.numel():
        d[on] = torch.autograd.grad(loss, logp)[0] * s["dloss"].double()
    dent = None
    if c["ent"]:
        dent = torch.zeros_like(d)
        dent[on] = -c["ent"] * s["dloss"].double() * w
    return {"dlogp": d, "dentropy": dent}
