"""Performance cases of the operators that generate responses behind shared prompts.

Three operators on a paged key/value cache, whose pages hold bf16 values or 4-bit
codes with a scale for every 32 of them:

  append  per-head norm and position rotation of new rows' q and k; the keys and the
          values go into the cache
  read    rows of the cache back as dense keys and values
  decode  attention of one new token per response over its prompt's pages, which a
          whole group of responses shares, and over its own

``own`` selects what ``run`` calls: False computes the plain form from
elementary torch operations, True calls this package's kernels.
"""
import ctypes
import math

import numpy as np
import torch

own = False

DEV = "cuda"
BF = torch.bfloat16
EPS = 1e-6
GROUP = 32  # values that share a scale in a 4-bit cache


# ------------------------------------------------------------------- layouts
def _draw_lengths(seed, n, lo, hi):
    return [lo] * n if lo == hi else np.random.default_rng(seed).integers(lo, hi + 1, n).tolist()


def _append_layout(c):
    """Of each stream: rows of this call, tokens held afterwards, position of its first token.  Stream 0 is the
    prompt where the case has one."""
    rows = _draw_lengths(c["r_seed"], c["N"], c["r_lo"], c["r_hi"])
    held = _draw_lengths(c["r_seed"] + 1, c["N"], c["held_lo"], c["held_hi"])
    lens, starts = [a + b for a, b in zip(rows, held)], [c["start"]] * c["N"]
    if c["P"]:
        rows, lens, starts = [c["P"]] + rows, [c["P"]] + lens, [0] + [c["P"]] * c["N"]
    if not any(rows):
        rows[0], lens[0] = 1, lens[0] + 1
    return rows, lens, starts


def _decode_layout(c):
    """Responses before each group's first, tokens of each prompt and of each response (-1: one that has ended)."""
    prompts = _draw_lengths(c["r_seed"], c["G"], c["p_lo"], c["p_hi"])
    lens = _draw_lengths(c["r_seed"] + 1, c["G"] * c["N"], c["r_lo"], c["r_hi"])
    for i in range(c["ended"]):
        lens[(5 * i + 2) % len(lens)] = -1 if i % 2 else 0
    return [c["N"] * g for g in range(c["G"] + 1)], prompts, lens


def _offsets(rows):
    return [0] + np.cumsum(rows).tolist()


# -------------------------------------------------------------------- cases
def _append(name, bits, P, N, r_lo, r_hi, Hq, Hkv, D, rope_dim, ps, held_lo=0, held_hi=0, start=0, interleaved=False,
            fused=True, w="bf16", w0=0.0, r_seed=1, base=1e6):
    return dict(name=name, op="append", bits=bits, P=P, N=N, r_lo=r_lo, r_hi=r_hi, r_seed=r_seed, held_lo=held_lo,
                held_hi=held_hi, start=start, Hq=Hq, Hkv=Hkv, D=D, rope_dim=rope_dim, ps=ps, interleaved=interleaved,
                fused=fused, weights=w, w0=w0, base=base)


def _read(name, bits, N, r_lo, r_hi, held_lo, held_hi, Hkv, D, ps, r_seed=2):
    return dict(name=name, op="read", bits=bits, P=0, N=N, r_lo=r_lo, r_hi=r_hi, r_seed=r_seed, held_lo=held_lo,
                held_hi=held_hi, start=0, Hkv=Hkv, D=D, ps=ps)


def _decode(name, bits, G, N, p_lo, p_hi, r_lo, r_hi, Hq, Hkv, D, ps, window=0, ended=0, r_seed=3):
    return dict(name=name, op="decode", bits=bits, G=G, N=N, p_lo=p_lo, p_hi=p_hi, r_lo=r_lo, r_hi=r_hi, r_seed=r_seed,
                Hq=Hq, Hkv=Hkv, D=D, ps=ps, window=window, ended=ended)


def listed():
    return [
        # one generation step of four responses, the package's smallest heads: latency is all of it
        _append("append step tiny", 16, 0, 4, 1, 1, 2, 2, 64, 64, 16, held_lo=0, held_hi=40, start=64, fused=False, w="f32"),
        # a generation step of 256 responses far into long contexts, cache of 4 bits; the new rows are read back
        _append("append step 4-bit", 4, 0, 256, 1, 1, 32, 8, 128, 128, 64, held_lo=0, held_hi=200, start=100000),
        # the benchmark's GRPO micro-batch (32 responses of 2048 behind a prompt of 6144) put into a cache to go on from
        _append("append packed grpo", 16, 6144, 32, 2048, 2048, 32, 8, 128, 128, 64),
        # wide heads of a global layer, a quarter of each head rotated, ragged responses, 4 bits, read back
        _append("append ragged wide 4-bit", 4, 4097, 24, 100, 1500, 8, 2, 512, 128, 32, interleaved=True, w0=1.0, r_seed=11,
                base=1e4),
        # the last tokens of a few short streams, narrow heads, 4 bits
        _read("read short 4-bit", 4, 9, 1, 77, 0, 50, 7, 64, 16),
        # a long prompt's keys and values for a dense pass over them
        _read("read long", 16, 1, 131072, 131072, 0, 0, 8, 128, 64),
        # a step of four short responses behind a short prompt: latency
        _decode("decode tiny", 16, 1, 4, 64, 64, 1, 32, 2, 2, 64, 16),
        # one answer behind 131,071 tokens of its own: few rows, so its keys have to be spread over all SMs
        _decode("decode long 4-bit", 4, 1, 1, 0, 0, 131071, 131071, 32, 8, 128, 64),
        # the GRPO layer half way through its responses: 32 of up to 2048 tokens behind one prompt of 6144
        _decode("decode grpo", 16, 1, 32, 6144, 6144, 1, 2048, 32, 8, 128, 64),
        # a rollout server's step: six prompts, 32 responses each, 4 bits
        _decode("decode groups 4-bit", 4, 6, 32, 1000, 5000, 500, 2900, 32, 8, 128, 32, r_seed=5),
        # a sliding-window layer of wide heads, the window spanning the end of the prompt in young responses
        _decode("decode wide window", 16, 2, 16, 16384, 16384, 100, 2000, 8, 2, 512, 64, window=1024),
        # seven queries to a key, narrow heads, small pages, odd lengths, some responses not begun and some ended
        _decode("decode odd 4-bit", 4, 3, 11, 1, 999, 1, 777, 21, 3, 64, 16, ended=3, r_seed=8),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _spread(rng, mean):
    """Bounds of lengths around a mean, equal or ragged."""
    return (max(1, mean // 2), mean + mean // 2) if rng.random() < 0.7 else (mean, mean)


def draw(rng):
    op = rng.choice(["append", "append", "read", "decode", "decode", "decode"])
    D = rng.choice([64, 128, 128, 512])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    c = dict(op=op, bits=rng.choice([16, 4]), Hkv=Hkv, D=D, ps=rng.choice([16, 32, 64, 128]), r_seed=rng.randrange(1 << 20))
    if op == "decode":
        c["Hq"] = Hkv * rng.choice([1, 2, 4, 4, 5, 7, 8, 16])
        c["G"], c["N"] = _log_int(rng, 1, 8), _log_int(rng, 1, 64)
        most = max(40, min(60000, 900_000_000 // (c["G"] * c["N"] * Hkv * D)))
        total = _log_int(rng, 20, most)
        prompt = int(total * rng.uniform(0.0, 0.9))
        c["p_lo"], c["p_hi"] = _spread(rng, prompt) if prompt else (0, 0)
        c["r_lo"], c["r_hi"] = _spread(rng, max(1, (total - prompt) * 2 // 3))
        c["window"] = rng.choice([0, 0, 0, 1024, rng.randrange(1, 3000)])
        c["ended"] = rng.choice([0, 0, 1, 2]) if c["G"] * c["N"] > 3 else 0
        return c
    heads = Hkv
    if op == "append":
        c["Hq"] = Hkv * rng.choice([1, 2, 4, 5, 8])
        heads += c["Hq"]
        c.update(rope_dim=rng.choice([16, D // 2, D, D]), interleaved=rng.random() < 0.3, fused=rng.random() < 0.6,
                 weights=rng.choice(["bf16", "f32", "none"]), w0=rng.choice([0.0, 1.0]), base=rng.choice([1e4, 1e6]))
    rows = _log_int(rng, 1, max(2, min(60000, 250_000_000 // (heads * D))))
    c["N"] = min(_log_int(rng, 1, 200), rows)
    c["P"] = int(rows * rng.uniform(0.1, 0.6)) if op == "append" and rng.random() < 0.4 else 0
    mean = max(1, (rows - c["P"]) // c["N"])
    c["r_lo"], c["r_hi"] = _spread(rng, mean) if mean > 1 else (1, 1)
    c["held_lo"], c["held_hi"] = rng.choice([(0, 0), (0, 200), (17, 90)])
    c["start"] = 0 if c["P"] else rng.choice([0, 1, 5000, 100000])
    return c


# ------------------------------------------------------------------ prepare
def _randn(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _page_tables(g, ps, *lengths):
    """One [streams, most pages] int32 table for each list of lengths, all from one shuffled pool; the places behind
    a stream's last page hold -1.  Returns the pool's pages and the tables."""
    need = [[max(0, -(-n // ps)) for n in ns] for ns in lengths]
    pool = sum(map(sum, need)) + 3
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32).cpu()
    tables, at = [], 0
    for counts in need:
        t = torch.full((len(counts), max(counts + [1])), -1, dtype=torch.int32)
        for i, k in enumerate(counts):
            t[i, :k] = order[at:at + k]
            at += k
        tables.append(t.to(DEV))
    return pool, tables


def _new_cache(g, c, pool):
    """k, v and their scales (None in bf16) of a cache that holds a model's keys and values: some channels of the
    keys are larger than others."""
    shape = (pool, c["Hkv"], c["ps"], c["D"])
    k = _randn(g, *shape, dtype=BF)
    k *= (0.6 + torch.rand(c["Hkv"], 1, c["D"], generator=g, device=DEV)).to(BF)
    v = _randn(g, *shape, dtype=BF)
    if c["bits"] == 16:
        return k, v, None, None
    (kc, ks), (vc, vs) = _quantise(k), _quantise(v)
    return kc, vc, ks, vs


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 29)
    return (_prepare_decode if case["op"] == "decode" else _prepare_rows)(case, g)


def _prepare_rows(c, g):
    rows, lens, starts = _append_layout(c)
    off = _offsets(rows)
    T, Hkv, D = off[-1], c["Hkv"], c["D"]
    pool, (pages,) = _page_tables(g, c["ps"], lens)
    s = dict(c=c, S=len(rows), off=off, c_off=(ctypes.c_int32 * len(off))(*off), pages=pages, lens=_int32(lens),
             starts=_int32(starts))
    s["cache"] = _new_cache(g, c, pool)
    stream = torch.repeat_interleave(torch.arange(s["S"]), torch.tensor(rows))
    index = torch.arange(T) - torch.tensor(off[1:])[stream] + torch.tensor(lens)[stream]
    s["stream"], s["index"] = stream.to(DEV), index.to(DEV)
    s["k_out"], s["v_out"] = (torch.empty(T, Hkv, D, dtype=BF, device=DEV) for _ in range(2))
    if c["op"] == "read":
        return s
    Hq = c["Hq"]
    if c["fused"]:
        row = _randn(g, T, (Hq + 2 * Hkv) * D, dtype=BF)
        cut = (0, Hq * D, (Hq + Hkv) * D, (Hq + 2 * Hkv) * D)
        s["q"], s["k"], s["v"] = (row[:, a:b].view(T, (b - a) // D, D) for a, b in zip(cut, cut[1:]))
    else:
        s["q"], s["k"], s["v"] = (_randn(g, T, h, D, dtype=BF) for h in (Hq, Hkv, Hkv))
    s["q_out"] = torch.empty(T, Hq, D, dtype=BF, device=DEV)
    j = torch.arange(c["rope_dim"] // 2, dtype=torch.float64, device=DEV)
    s["inv_freq"] = (c["base"] ** (-2.0 * j / c["rope_dim"])).float()
    s["qw"] = s["kw"] = None
    if c["weights"] != "none":
        wt = {"bf16": BF, "f32": torch.float32}[c["weights"]]
        s["qw"], s["kw"] = ((1.0 - c["w0"] + 0.2 * _randn(g, D)).to(wt) for _ in range(2))
    return s


def _prepare_decode(c, g):
    groups, prompts, lens = _decode_layout(c)
    B, Hq, D = len(lens), c["Hq"], c["D"]
    pool, (prompt_pages, pages) = _page_tables(g, c["ps"], prompts, lens)
    s = dict(c=c, B=B, groups=groups, c_groups=(ctypes.c_int32 * len(groups))(*groups), prompt_pages=prompt_pages,
             prompt_lens=_int32(prompts), pages=pages, lens=_int32(lens))
    s["cache"] = _new_cache(g, c, pool)
    s["q"] = _randn(g, B, Hq, D, dtype=BF)
    s["out"] = torch.empty(B, Hq, D, dtype=BF, device=DEV)
    s["lse"] = torch.empty(Hq, B, dtype=torch.float32, device=DEV)
    # enough for any case here: partial results of every response's and prompt's heads and of every thread block
    s["ws"] = torch.empty((B * Hq * 6 + 64 * 1024) * (D + 2) * 4, dtype=torch.uint8, device=DEV)
    s["most"] = max(prompts), max(max(lens), 0)
    return s


# ---------------------------------------------------------------- 4-bit form
def _quantise(x):
    """Codes (two to a byte, the even value in the low half) and scales of rows of D values: value = scale (code - 8).
    The scale is a seventh of the largest magnitude of its 32 values, rounded up to five significant bits; a value
    goes to its nearest code, from half way between two to the larger magnitude."""
    x = x.float().unflatten(-1, (-1, GROUP))
    top = x.abs().amax(-1)
    t = top / torch.full_like(top, 7.0)  # a quotient of two tensors is rounded once; one by a number is a product
    step = ((t.view(torch.int32) + 0x7FFFF) & ~0x7FFFF).view(torch.float32)
    n = torch.floor(x.abs() / torch.where(step > 0, step, torch.ones_like(step))[..., None] + 0.5)
    code = (n * torch.sign(x) + 8.0).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), step.to(BF)


def _dequantise(codes, scale):
    n = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float() - 8.0
    return (n.unflatten(-1, (-1, GROUP)) * scale.float()[..., None]).flatten(-2)


def _gathered(cache, page, slot):
    """Keys and values in fp32 at the given pages and places in them, heads behind the places' dimensions."""
    k, v, ks, vs = cache
    if ks is None:
        return k[page, :, slot].float(), v[page, :, slot].float()
    return _dequantise(k[page, :, slot], ks[page, :, slot]), _dequantise(v[page, :, slot], vs[page, :, slot])


# ---------------------------------------------------------------------- run
def run(s):
    return {"append": _run_append, "read": _run_read, "decode": _run_decode}[s["c"]["op"]](s["c"], s)


def _places(c, s):
    return s["pages"][s["stream"], s["index"] // c["ps"]].long(), s["index"] % c["ps"]


def _rotate(c, x, cos, sin):
    r = c["rope_dim"]
    if c["interleaved"]:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        y = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = x[..., :r // 2], x[..., r // 2:r]
        y = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((y, x[..., r:]), -1)


def _run_append(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        cache = dualkv.KVCache(*s["cache"])
        dualkv.dualkv_cache_append(s["q"], s["k"], s["v"], s["qw"], s["kw"], c["w0"], EPS, s["inv_freq"], c["rope_dim"],
                                   c["interleaved"], cache, s["pages"], s["lens"], s["starts"], s["S"], s["c_off"], c["Hq"],
                                   c["Hkv"], c["D"], s["q_out"], None)
        if c["bits"] == 4:
            dualkv.dualkv_cache_read(cache, s["pages"], s["lens"], s["S"], s["c_off"], c["Hkv"], c["D"], s["k_out"],
                                     s["v_out"])
            return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}
        return {"q": s["q_out"], "k": s["cache"][0], "v": s["cache"][1]}
    angle = (s["starts"].long()[s["stream"]] + s["index"]).double()[:, None] * s["inv_freq"].double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, w):
        x = x.float()
        if w is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (w.float() + c["w0"])
        return _rotate(c, x, cos, sin)

    q, k = one(s["q"], s["qw"]).to(BF), one(s["k"], s["kw"])
    page, slot = _places(c, s)
    ck, cv, cks, cvs = s["cache"]
    if c["bits"] == 16:
        ck[page, :, slot], cv[page, :, slot] = k.to(BF), s["v"]
        return {"q": q, "k": ck, "v": cv}
    (ck[page, :, slot], cks[page, :, slot]), (cv[page, :, slot], cvs[page, :, slot]) = _quantise(k), _quantise(s["v"])
    k, v = _gathered(s["cache"], page, slot)
    return {"q": q, "k": k.to(BF), "v": v.to(BF)}


def _run_read(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_cache_read(dualkv.KVCache(*s["cache"]), s["pages"], s["lens"], s["S"], s["c_off"], c["Hkv"], c["D"],
                                 s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    k, v = _gathered(s["cache"], *_places(c, s))
    return {"k": k.to(BF), "v": v.to(BF)}


def _run_decode(c, s):
    if own:
        from shared_prompt_exact_gb300 import dualkv
        dualkv.dualkv_decode(s["q"], dualkv.KVCache(*s["cache"]), s["prompt_pages"], s["prompt_lens"], s["pages"], s["lens"],
                             c["G"], s["c_groups"], c["Hq"], c["Hkv"], c["D"], c["D"] ** -0.5, c["window"], s["out"],
                             s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    B, Hkv, D, ps = s["B"], c["Hkv"], c["D"], c["ps"]
    group = torch.arange(B, device=DEV) // c["N"]
    plen, rlen = s["prompt_lens"].long()[group][:, None], s["lens"].long()[:, None]
    # places of the prompt's tokens, then of the response's; position of each, and whether the query sees it
    i, j = torch.arange(s["most"][0], device=DEV), torch.arange(s["most"][1], device=DEV)
    place = torch.cat((i, j))
    page = torch.cat((s["prompt_pages"].long()[group][:, i // ps], s["pages"].long()[:, j // ps]), 1)
    pos = torch.cat((i.expand(B, -1), plen + j), 1)
    seen = torch.cat((i < plen, j < rlen), 1) & (rlen >= 0)
    if c["window"]:
        seen &= plen + rlen - 1 - pos < c["window"]
    k, v = _gathered(s["cache"], page.clamp(min=0), (place % ps).expand(B, -1))  # [B, keys, Hkv, D]
    v = torch.where(seen[:, :, None, None], v, torch.zeros((), device=DEV))
    x = torch.matmul(s["q"].float().view(B, Hkv, -1, D), k.permute(0, 2, 3, 1)) * D ** -0.5  # [B, Hkv, queries, keys]
    x = torch.where(seen[:, None, None], x, torch.full((), -math.inf, device=DEV))
    m = x.amax(-1, keepdim=True).clamp(min=-3e38)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    out = torch.matmul(e, v.transpose(1, 2)) / total
    out = torch.where(total > 0, out, torch.zeros((), device=DEV))
    lse = torch.where(total > 0, m + total.log(), torch.full((), -math.inf, device=DEV))
    return {"out": out.to(BF).flatten(1, 2), "lse": lse.flatten(1).t().contiguous()}


# --------------------------------------------------------------------- work
def _row_bytes(c):
    """Bytes of one token's key, or value, in one head of the cache."""
    return 2 * c["D"] if c["bits"] == 16 else c["D"] // 2 + c["D"] // GROUP * 2


def work(case):
    c = case
    if c["op"] == "decode":
        _, prompts, lens = _decode_layout(c)
        keys = pairs = 0
        for g, p in enumerate(prompts):
            first = p  # the first token of the prompt that a response of the group sees
            for n in lens[g * c["N"]:(g + 1) * c["N"]]:
                if n >= 0:
                    lo = max(0, p + n - c["window"]) if c["window"] else 0
                    first = min(first, lo)
                    keys += p + n - max(lo, p)
                    pairs += p + n - lo
            keys += p - first
        B = len(lens)
        return {"bytes": keys * c["Hkv"] * 2 * _row_bytes(c) + B * c["Hq"] * (4 * c["D"] + 4) + 4 * keys // c["ps"],
                "flops": 4 * c["D"] * c["Hq"] * pairs}
    T, kv = sum(_append_layout(c)[0]), c["Hkv"] * c["D"]
    held = T * c["Hkv"] * 2 * _row_bytes(c)
    if c["op"] == "read":
        return {"bytes": held + T * 4 * kv, "flops": T * 2 * kv}
    w = 0 if c["weights"] == "none" else 2 * c["D"] * (2 if c["weights"] == "bf16" else 4)
    x = T * (c["Hq"] + c["Hkv"]) * c["D"]
    back = held + T * 4 * kv if c["bits"] == 4 else 0
    return {"bytes": T * (4 * c["Hq"] * c["D"] + 4 * kv) + held + back + w + 2 * c["rope_dim"], "flops": 7 * x}


# -------------------------------------------------------------------- exact
def exact(case, seed):
    """What run() returns, from the definitions in 64 bits, stream by stream and response by response."""
    s = prepare(case, seed)
    return {"append": _exact_append, "read": _exact_read, "decode": _exact_decode}[case["op"]](case, s)


def _stream_rows(c, cache, table, lo, hi):
    """Keys and values of a stream's tokens [lo, hi) in fp64, [tokens, Hkv, D]."""
    ids = table[lo // c["ps"]:-(-hi // c["ps"])].long()
    got = []
    for x, scale in zip(cache[:2], cache[2:]):
        x = x.index_select(0, ids)
        if scale is None:
            x = x.double()
        else:
            low = torch.remainder(x, 16)
            x = torch.stack((low, torch.div(x - low, 16, rounding_mode="floor")), -1).double().flatten(-2) - 8
            x = x * torch.repeat_interleave(scale.index_select(0, ids).double(), GROUP, -1)
        x = x.permute(0, 2, 1, 3).flatten(0, 1)
        got.append(x[lo % c["ps"]:lo % c["ps"] + hi - lo])
    return got


def _exact_read(c, s):
    ks, vs = [], []
    lens = s["lens"].tolist()
    for i, (a, b) in enumerate(zip(s["off"], s["off"][1:])):
        if b > a:
            k, v = _stream_rows(c, s["cache"], s["pages"][i], lens[i] - (b - a), lens[i])
            ks.append(k)
            vs.append(v)
    return {"k": torch.cat(ks), "v": torch.cat(vs)}


def _nearest(x):
    """The values that 4-bit codes stand for, [rows, Hkv, D] in fp64."""
    x = x.unflatten(-1, (-1, GROUP))
    t = x.abs().amax(-1, keepdim=True) / 7
    unit = torch.exp2(torch.floor(torch.log2(t)) - 4)
    step = torch.where(t > 0, torch.ceil(t / unit) * unit, torch.ones_like(t))
    below = torch.trunc(x / step)
    return ((below + torch.trunc(2 * (x / step - below))) * step).flatten(-2)


def _exact_append(c, s):
    lens, starts = s["lens"].tolist(), s["starts"].tolist()
    pos = torch.cat([torch.arange(n - (b - a), n, dtype=torch.float64, device=DEV) + p0
                     for n, p0, a, b in zip(lens, starts, s["off"], s["off"][1:])])
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                       torch.outer(pos, s["inv_freq"].double())).unsqueeze(1)
    half = c["rope_dim"] // 2

    def one(x, w):
        x = x.double()
        if w is not None:
            x = x / ((x ** 2).sum(-1, keepdim=True) / c["D"] + EPS).sqrt() * (c["w0"] + w.double())
        head, tail = x[..., :c["rope_dim"]], x[..., c["rope_dim"]:]
        if c["interleaved"]:
            head = torch.view_as_real(torch.view_as_complex(head.unflatten(-1, (half, 2)).contiguous()) * turn).flatten(-2)
        else:
            z = torch.complex(head[..., :half].contiguous(), head[..., half:].contiguous()) * turn
            head = torch.cat((z.real, z.imag), -1)
        return torch.cat((head, tail), -1)

    q, k, v = one(s["q"], s["qw"]), one(s["k"], s["kw"]), s["v"].double()
    if c["bits"] == 4:
        return {"q": q, "k": _nearest(k), "v": _nearest(v)}
    ck, cv = (x.double() for x in s["cache"][:2])
    for i, (a, b) in enumerate(zip(s["off"], s["off"][1:])):
        at = torch.arange(lens[i] - (b - a), lens[i], device=DEV)
        flat = s["pages"][i].long()[at // c["ps"]] * c["ps"] + at % c["ps"]
        for cache, x in ((ck, k), (cv, v)):
            for h in range(c["Hkv"]):
                cache[flat // c["ps"], h, flat % c["ps"]] = x[a:b, h]
    return {"q": q, "k": ck, "v": cv}


def _exact_decode(c, s):
    out = torch.zeros(s["B"], c["Hq"], c["D"], dtype=torch.float64, device=DEV)
    lse = torch.full((c["Hq"], s["B"]), -math.inf, dtype=torch.float64, device=DEV)
    prompts, lens = s["prompt_lens"].tolist(), s["lens"].tolist()
    for g, p in enumerate(prompts):
        for b in range(s["groups"][g], s["groups"][g + 1]):
            n = lens[b]
            lo = max(0, p + n - c["window"]) if c["window"] else 0
            if n < 0 or p + n <= lo:
                continue
            parts = []
            if lo < p:
                parts.append(_stream_rows(c, s["cache"], s["prompt_pages"][g], lo, p))
            if n > max(lo - p, 0):
                parts.append(_stream_rows(c, s["cache"], s["pages"][b], max(lo - p, 0), n))
            k, v = (torch.cat(x) for x in zip(*parts))
            q = s["q"][b].double().view(c["Hkv"], -1, c["D"])
            x = torch.einsum("hgd,thd->hgt", q, k) / math.sqrt(c["D"])
            total = torch.logsumexp(x, -1)
            out[b] = torch.einsum("hgt,thd->hgd", (x - total[..., None]).exp(), v).flatten(0, 1)
            lse[:, b] = total.flatten()
    return {"out": out, "lse": lse}
