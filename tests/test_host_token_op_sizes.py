"""Sizes past 32 bits: the C calls take 32-bit counts, and a count that does not fit must not wrap into a small one.
Tensors without storage stand for ones that fill the GPU."""
import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk
from test_host_token_ops import _logp

BF, F32 = torch.bfloat16, torch.float32
FAR = 1 << 32


@pytest.fixture(autouse=True)
def _lib(monkeypatch):
    pbuild.build()
    dk.load()
    monkeypatch.setattr(torch.cuda, "current_device", lambda: -1)  # where tensors without storage are


def _empty(*shape, dtype=F32):
    return torch.empty(*shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("off", [[0, FAR + 3], [0, 1 << 31], [0, -FAR, 3], [0, FAR]])
def test_offsets(off):
    with pytest.raises(ValueError, match="32 bits"):
        dk.offsets(off)


def test_loss_of_too_many_tokens():
    n = FAR + 5
    t, one, w = _empty(n), _empty(1), _empty(1)
    with pytest.raises(ValueError, match="32 bits"):
        dk.dualkv_policy_loss(t, t, None, None, w, None, 1, [0, n], 0.2, 0.2, 0.0, 0.0, 0.0, "token_mean", one, _empty(4), w,
                              None, stream=0)
    with pytest.raises(ValueError, match="32 bits"):
        dk.dualkv_policy_loss_bwd(t, t, None, w, None, 1, [0, n], 0.2, 0.2, 0.0, 0.0, 0.0, "token_mean", one, w, _empty(n),
                                  None, stream=0)
    with pytest.raises(ValueError, match="32 bits"):
        dk.dualkv_policy_loss_workspace_bytes(1, [0, n])


def test_vocabulary_of_too_many_entries():
    V, off = FAR + 64, [0, 2]
    x, tok, lp, lse = _empty(3, V, dtype=BF), _empty(2, dtype=torch.int64), _empty(2), _empty(3)
    with pytest.raises(ValueError, match="32 bits"):
        dk.dualkv_token_logprobs(x, tok, 1.0, 1, 1, off, lp, None, lse, stream=0)
    with pytest.raises(ValueError, match="32 bits"):
        dk.dualkv_token_logprobs_bwd(x, tok, 1.0, 1, 1, off, lse, None, lp, None, _empty(3, V, dtype=BF), stream=0)


@pytest.mark.parametrize("Hq,Hkv,D,rope_dim", [(1, 1, FAR + 64, 64), (FAR + 2, 1, 64, 64), (FAR + 2, FAR + 2, 64, 0),
                                               (1, 1, 64, FAR + 64)])
def test_heads_of_too_many_values(Hq, Hkv, D, rope_dim):
    off = [0, 1]
    q, k, f = _empty(2, Hq, D, dtype=BF), _empty(2, Hkv, D, dtype=BF), _empty(rope_dim // 2)
    args = (None, None, 0.0, 1e-6, f, rope_dim, False, 1, 1, off, Hq, Hkv, D)
    with pytest.raises(ValueError, match="32 bits"):
        dk.dualkv_qk_norm_rope(q, k, *args, q, k, stream=0)
    with pytest.raises(ValueError, match="32 bits"):
        dk.dualkv_qk_norm_rope_bwd(q, k, q, k, *args, q, k, None, None, None, stream=0)
    if rope_dim < FAR:
        with pytest.raises(ValueError, match="32 bits"):
            dk.dualkv_qk_norm_rope_bwd_workspace_bytes(1, 1, off, Hq, Hkv, D)


def test_prompt_of_too_many_tokens():
    with pytest.raises(ValueError):
        dk.dualkv_qk_norm_rope_bwd_workspace_bytes(FAR + 4, 1, [0, 1], 2, 1, 64)


@pytest.mark.parametrize("backward", [False, True])
def test_scale_whose_base_2_form_overflows(backward):
    # scale * log2(e) has to be finite: 0 * inf would make a row's largest entry NaN
    for scale in (2.4e38, 3.4e38):
        assert _logp(dk.load(), backward, scale=scale) == dk.DUALKV_ERR_INVALID
