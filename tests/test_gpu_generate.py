"""The operators of generation together, as a rollout uses them, against the packed operators of training.

A prompt goes into a cache once, responses grow behind it token by token (append, then decode), and in the end the
cache is read back.  The packed operators (qk_norm_rope and dualkv_fwd) on the finished micro-batch give what every step
should have given: each step's row is the packed layout's row of that token.  bf16 caches hold the same keys up to
one rounding, so outputs agree as far as the two attentions' own bounds reach (2^-8 of the value and of
sum p |v| <= max |v| each, for the output's rounding and the weights').  With a cache of 4 bits the attention is compared with
dualkv_fwd on the keys and values that are read back.
"""
import numpy as np
import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    pbuild.build()
    dk.load()


@pytest.mark.parametrize("bits", [16, 4])
@pytest.mark.parametrize("P,R,Hq,Hkv,D,ps,window", [(70, [9, 1, 20], 8, 2, 128, 16, 0), (33, [5, 17], 4, 1, 64, 32, 24),
                                                    (20, [6, 3], 4, 2, 512, 16, 0)])
def test_generation_matches_the_packed_operators(P, R, Hq, Hkv, D, ps, window, bits):
    off = [0] + np.cumsum(R).tolist()
    T, N = P + off[-1], len(R)
    g = torch.Generator(device="cuda").manual_seed(P + bits)
    x = torch.randn(T, (Hq + 2 * Hkv) * D, generator=g, device="cuda").to(BF)
    cut = lambda t: (t[:, :Hq * D].view(-1, Hq, D), t[:, Hq * D:(Hq + Hkv) * D].view(-1, Hkv, D),  # noqa: E731
                     t[:, (Hq + Hkv) * D:].view(-1, Hkv, D))
    w = [1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    f = (1e4 ** (-torch.arange(D // 2, device="cuda") * 2.0 / D)).float()
    i32 = lambda t: torch.tensor(t, dtype=torch.int32, device="cuda")  # noqa: E731
    most = -(-max(R) // ps)
    p_pages = -(-P // ps)
    cache = dk.KVCache.empty(p_pages + N * most, Hkv, ps, D, bits)
    prompt_table = torch.arange(p_pages, dtype=torch.int32, device="cuda")[None]
    table = (p_pages + torch.arange(N * most, dtype=torch.int32, device="cuda")).view(N, most)
    prompt_len = i32([P])
    q, k, v = cut(x[:P])
    dk.cache_append(q, k, v, cache, prompt_table, prompt_len, i32([0]), [0, P], f, *w)
    lens = torch.zeros(N, dtype=torch.int32, device="cuda")
    got, rows, queries = [], [], []
    for r in range(max(R)):
        live = [n for n in range(N) if r < R[n]]
        lens.copy_(i32([r + 1 if n in live else -1 for n in range(N)]))
        step_off = [0] + np.cumsum([1 if n in live else 0 for n in range(N)]).tolist()
        where = [P + off[n] + r for n in live]
        q, k, v = cut(x[torch.tensor(where, device="cuda")])
        q1 = dk.cache_append(q, k, v, cache, table, lens, i32([P] * N), step_off, f, *w)
        full = torch.zeros(N, Hq, D, dtype=BF, device="cuda")
        full[live] = q1
        out, lse = dk.decode(full, cache, prompt_table, prompt_len, table, lens, [0, N], window)
        ended = [n for n in range(N) if n not in live]
        assert not bool(out[ended].any()) and bool(torch.isneginf(lse[:, ended]).all())
        got.append((out[live], lse[:, live]))
        queries.append(q1)
        rows += where
    dk.dualkv_check_status()
    out, lse = torch.cat([o for o, _ in got]), torch.cat([s for _, s in got], 1)
    rows = torch.tensor(rows, device="cuda")
    q_all, k_all = dk.qk_norm_rope(*cut(x)[:2], P, off, f, *w)
    v_all = cut(x)[2].contiguous()
    assert torch.equal(torch.cat(queries), q_all[rows])
    kc, vc = (torch.cat(t) for t in zip(dk.cache_read(cache, prompt_table, prompt_len, [0, P]),
                                        dk.cache_read(cache, table, i32(R), off)))
    if bits == 16:
        assert torch.equal(kc, k_all) and torch.equal(vc, v_all)
    want, want_lse = dk.forward(q_all, kc, vc, P, off, window)
    tol = 2 * 2.0 ** -8 * (want[rows].abs().max() + vc.abs().max()).item()
    assert float((out.float() - want[rows].float()).abs().max()) <= tol
    assert float((lse - want_lse[:, rows]).abs().max()) <= 1e-3
