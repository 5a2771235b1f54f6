"""The generation loop as the README has it, with responses that end on the way: they get no row, see nothing and
write nothing from then on, also when their pages have gone to another response."""
import numpy as np
import pytest
import torch

from oracle import cache as oc
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF = torch.bfloat16


def _np(t):
    return t.detach().double().cpu().numpy()


@pytest.mark.parametrize("bits", [16, 4])
def test_ended_responses_stay_ended(bits):
    pbuild.build()
    P, N, Hq, Hkv, D, ps, steps = 21, 5, 4, 2, 64, 16, 24
    ends = [steps, 3, steps, 17, 0]  # steps that each response takes
    g = torch.Generator(device="cuda").manual_seed(bits)
    rn = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF)  # noqa: E731
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    f = (1e4 ** (-torch.arange(D // 2, device="cuda") * 2.0 / D)).float()
    w = [1 + 0.2 * torch.randn(D, generator=g, device="cuda") for _ in range(2)]
    cache = dk.KVCache.empty(2 + N + 2, Hkv, ps, D, bits)
    for t in (cache.k, cache.v) if bits == 16 else (cache.k_scale, cache.v_scale):
        t.fill_(float("nan"))
    prompt_table, prompt_lens = i32([[0, 1]]), i32([P])
    dk.cache_append(rn(P, Hq, D), rn(P, Hkv, D), rn(P, Hkv, D), cache, prompt_table, prompt_lens, i32([0]), [0, P], f, *w)
    prompt_k, prompt_v = dk.cache_read(cache, prompt_table, prompt_lens, [0, P])
    # responses 0 and 2 go on, past their first page, in the pages of 1 and 4, which end before that
    table = i32([[2, 3], [3, 7], [4, 6], [5, 8], [6, 7]])
    lens = i32([0 if n else -1 for n in ends])
    q_all = torch.full((N, Hq, D), float("nan"), dtype=BF, device="cuda")
    for step in range(steps):
        for n, end in enumerate(ends):
            if step == end:
                lens[n] = -1
                q_all[n] = float("nan")  # what an ended one has is not used
        live = [n for n, end in enumerate(ends) if step < end]
        rows = [0] + np.cumsum([n in live for n in range(N)]).tolist()
        lens += (lens >= 0).int()
        assert lens.tolist() == [step + 1 if n in live else -1 for n in range(N)]
        q = dk.cache_append(rn(len(live), Hq, D), rn(len(live), Hkv, D), rn(len(live), Hkv, D), cache, table, lens, i32([P] * N),
                            rows, f, *w)
        q_all[live] = q
        out, lse = dk.decode(q_all, cache, prompt_table, prompt_lens, table, lens, [0, N])
        dk.dualkv_check_status()
        k, v = dk.cache_read(cache, table, lens, [0] + np.cumsum([step + 1 if n in live else 0 for n in range(N)]).tolist())
        for n in range(N):
            if n not in live:
                assert not bool(out[n].any()) and bool(torch.isneginf(lse[:, n]).all())
                continue
            at = live.index(n) * (step + 1)
            kn, vn = (np.concatenate([_np(a), _np(b[at:at + step + 1])]) for a, b in ((prompt_k, k), (prompt_v, v)))
            pos = (np.arange(P), P + np.arange(step + 1))
            ref, ref_lse, A, X = oc.attend(_np(q_all[n]), kn, vn, D ** -0.5, P + step, pos, 0)
            d = (4 * D + 32) * U * X  # as in test_gpu_decode
            assert np.all(np.abs(_np(out[n]) - ref) <= 2.0 ** -8 * (np.abs(ref) + A) + (2 * d[:, None] + 2.0 ** -20) * A)
            assert np.all(np.abs(_np(lse[:, n]) - ref_lse) <= d + 2.0 ** -20 + 4 * U * np.abs(ref_lse))
