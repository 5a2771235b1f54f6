"""The per-token operators at the ends of what their entry points accept, against fp64."""
import numpy as np
import pytest
import torch

import test_gpu_rope as tr
from oracle import rope as orp
from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


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
