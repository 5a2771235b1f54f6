"""Host-side argument validation of the per-token operators around attention: every
case below is refused before any device work; no pointer is dereferenced."""
import ctypes

import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

OK_OFF = [0, 2, 3]


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return dk.load()


def _vp(x):
    return ctypes.c_void_p(x)


def _rope(lib, backward=False, **kw):
    a = dict(q=0x100000, qs=256, k=0x200000, ks=128, qw=0x300000, kw=0x301000, wd=dk.DUALKV_BF16, w0=0.0, eps=1e-6,
             f=0x302000, rd=64, inter=0, P=4, N=2, off=OK_OFF, Hq=4, Hkv=2, D=64, qo=0x400000, qos=256, ko=0x500000, kos=128,
             gq=0x600000, gk=0x700000, dqw=0x800000, dkw=0x801000, ws=0x900000, wsb=1 << 20)
    a.update(kw)
    off = None if a["off"] is None else (ctypes.c_int32 * len(a["off"]))(*a["off"])
    head = [_vp(a["q"]), a["qs"], _vp(a["k"]), a["ks"]]
    mid = [_vp(a["qw"]), _vp(a["kw"]), a["wd"], a["w0"], a["eps"], _vp(a["f"]), a["rd"], a["inter"], a["P"], a["N"], off,
           a["Hq"], a["Hkv"], a["D"]]
    if not backward:
        return lib.dualkv_qk_norm_rope(*head, *mid, _vp(a["qo"]), _vp(a["ko"]), None)
    return lib.dualkv_qk_norm_rope_bwd(*head, _vp(a["gq"]), _vp(a["gk"]), *mid, _vp(a["qo"]), a["qos"], _vp(a["ko"]),
                                       a["kos"], _vp(a["dqw"]), _vp(a["dkw"]), _vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("backward", [False, True])
def test_rope_refusals(lib, backward):
    def rc(**kw):
        return _rope(lib, backward, **kw)

    bad = dk.DUALKV_ERR_INVALID
    for kw in (dict(P=-1), dict(N=0), dict(off=None), dict(off=[0, 3, 2]), dict(off=[1, 2, 3]), dict(P=0, off=[0, 0, 0]),
               dict(Hkv=3), dict(D=96), dict(q=0), dict(k=0), dict(qo=0), dict(ko=0), dict(qs=255), dict(qs=248),
               dict(qs=1 << 40), dict(qs=-256), dict(ks=0), dict(kw=0), dict(qw=0), dict(wd=2), dict(wd=-1), dict(eps=-1.0),
               dict(eps=float("nan")), dict(w0=float("inf")), dict(rd=-16), dict(rd=80), dict(rd=8), dict(rd=64, f=0),
               dict(Hq=1 << 26, Hkv=1, qs=1 << 31),
               # an output over an input or over the other output
               dict(qo=0x100000), dict(qo=0x200040), dict(ko=0x400040), dict(qo=0x301000), dict(ko=0x302000)):
        assert rc(**kw) == bad, kw
    for kw in (dict(q=0x100008), dict(ko=0x500008), dict(qw=0x300002), dict(f=0x302004)):
        assert rc(**kw) == dk.DUALKV_ERR_ALIGN, kw
    many = [0] * 4096 + [1]
    assert rc(N=4096, off=many) == dk.DUALKV_ERR_UNSUPPORTED


def test_rope_backward_refusals(lib):
    for kw in (dict(gq=0), dict(gk=0), dict(dqw=0), dict(dkw=0), dict(qos=128), dict(kos=2), dict(dqw=0x801000),
               # interleaved gradients whose columns overlap: q takes columns 0..255 of rows of 384
               dict(qos=384, kos=384, ko=0x400000 + 2 * 248), dict(qos=384, kos=384, ko=0x400000 + 2 * 264),
               dict(dkw=0x900000)):
        assert _rope(lib, True, **kw) == dk.DUALKV_ERR_INVALID, kw
    for kw in (dict(ws=0), dict(ws=0x900010), dict(wsb=16)):
        assert _rope(lib, True, **kw) == dk.DUALKV_ERR_WORKSPACE, kw
    off = dk.offsets(OK_OFF)
    need = lib.dualkv_qk_norm_rope_bwd_workspace_bytes(4, 2, off, 4, 2, 64)
    assert need > 0 and _rope(lib, True, wsb=need - 1) == dk.DUALKV_ERR_WORKSPACE
    assert lib.dualkv_qk_norm_rope_bwd_workspace_bytes(4, 2, off, 4, 3, 64) == 0
    assert lib.dualkv_qk_norm_rope_bwd_workspace_bytes(4, 2, off, 4, 2, 80) == 0


def test_offsets_are_converted_once():
    off = dk.offsets(OK_OFF)
    assert dk.offsets(off) is off and list(off) == OK_OFF


def _logp(lib, backward=False, **kw):
    a = dict(x=0x100000, xs=64, dt=dk.DUALKV_BF16, V=64, scale=1.0, tok=0x200000, P=4, N=2, off=OK_OFF, lp=0x300000,
             ent=0x301000, lse=0x302000, dlp=0x303000, dent=0x304000, dx=0x400000, dxs=64)
    a.update(kw)
    off = None if a["off"] is None else (ctypes.c_int32 * len(a["off"]))(*a["off"])
    head = [_vp(a["x"]), a["xs"], a["dt"], a["V"], a["scale"], _vp(a["tok"]), a["P"], a["N"], off]
    if not backward:
        return lib.dualkv_token_logprobs(*head, _vp(a["lp"]), _vp(a["ent"]), _vp(a["lse"]), None)
    return lib.dualkv_token_logprobs_bwd(*head, _vp(a["lse"]), _vp(a["ent"]), _vp(a["dlp"]), _vp(a["dent"]), _vp(a["dx"]),
                                         a["dxs"], None)


@pytest.mark.parametrize("backward", [False, True])
def test_logprobs_refusals(lib, backward):
    for kw in (dict(P=-1), dict(N=0), dict(off=None), dict(off=[0, 3, 2]), dict(P=0, off=[0, 0, 0]), dict(dt=2), dict(V=0),
               dict(xs=63), dict(xs=1 << 40), dict(scale=0.0), dict(scale=float("inf")), dict(x=0), dict(tok=0)):
        assert _logp(lib, backward, **kw) == dk.DUALKV_ERR_INVALID, kw
    for kw in (dict(x=0x100001), dict(x=0x100002, dt=dk.DUALKV_F32), dict(tok=0x200004), dict(lse=0x302002)):
        assert _logp(lib, backward, **kw) == dk.DUALKV_ERR_ALIGN, kw
    assert _logp(lib, backward, N=4096, off=[0] * 4096 + [1]) == dk.DUALKV_ERR_UNSUPPORTED


def test_logprobs_overlaps(lib):
    bad = dk.DUALKV_ERR_INVALID
    for kw in (dict(lp=0), dict(lp=0x100000), dict(lse=0x200008), dict(ent=0x300008)):
        assert _logp(lib, **kw) == bad, kw
    for kw in (dict(lse=0), dict(dlp=0), dict(ent=0), dict(dx=0), dict(dxs=63), dict(dx=0x100080), dict(dx=0x1fff80),
               dict(dx=0x303000), dict(dx=0x100000, dxs=65), dict(dx=0x304000)):
        assert _logp(lib, True, **kw) == bad, kw
    assert _logp(lib, True, dx=0x400001) == dk.DUALKV_ERR_ALIGN


def _policy(lib, backward=False, **kw):
    a = dict(lp=0x100000, old=0x101000, ref=0x102000, ent=0x103000, adv=0x104000, pt=0, mask=0x105000, N=2, off=OK_OFF, lo=0.2,
             hi=0.2, dual=0.0, kl=0.1, ec=0.1, red=0, loss=0x106000, stats=0x107000, w=0x108000, ws=0x109000, wsb=1 << 20,
             dl=0x300000, g=0x301000, gh=0x302000)
    a.update(kw)
    off = None if a["off"] is None else (ctypes.c_int32 * len(a["off"]))(*a["off"])
    mid = [_vp(a["adv"]), a["pt"], _vp(a["mask"]), a["N"], off, a["lo"], a["hi"], a["dual"], a["kl"], a["ec"]]
    if not backward:
        return lib.dualkv_policy_loss(_vp(a["lp"]), _vp(a["old"]), _vp(a["ref"]), _vp(a["ent"]), *mid, a["red"],
                                      _vp(a["loss"]), _vp(a["stats"]), _vp(a["w"]), _vp(a["ws"]), a["wsb"], None)
    return lib.dualkv_policy_loss_bwd(_vp(a["lp"]), _vp(a["old"]), _vp(a["ref"]), *mid, _vp(a["dl"]), _vp(a["w"]),
                                      _vp(a["g"]), _vp(a["gh"]), None)


@pytest.mark.parametrize("backward", [False, True])
def test_policy_refusals(lib, backward):
    nan = float("nan")
    for kw in (dict(N=0), dict(off=None), dict(off=[0, 3, 2]), dict(off=[1, 2, 3]), dict(lp=0), dict(old=0), dict(ref=0),
               dict(adv=0), dict(w=0), dict(lo=1.0), dict(lo=-0.1), dict(lo=nan), dict(hi=-1.0), dict(hi=nan), dict(dual=1.0),
               dict(dual=nan), dict(kl=nan), dict(ec=float("inf")), dict(hi=1e31), dict(dual=1e31), dict(kl=-1e31)):
        assert _policy(lib, backward, **kw) == dk.DUALKV_ERR_INVALID, kw
    for kw in (dict(lp=0x100002), dict(adv=0x104001), dict(w=0x108003)):
        assert _policy(lib, backward, **kw) == dk.DUALKV_ERR_ALIGN, kw
    assert _policy(lib, backward, N=4096, off=[0] * 4096 + [1]) == dk.DUALKV_ERR_UNSUPPORTED


def test_policy_outputs_and_workspace(lib):
    bad = dk.DUALKV_ERR_INVALID
    for kw in (dict(red=3), dict(red=-1), dict(loss=0), dict(stats=0), dict(ent=0), dict(loss=0x100000), dict(stats=0x106000 - 8),
               dict(w=0x105000), dict(loss=0x109010)):
        assert _policy(lib, **kw) == bad, kw
    for kw in (dict(ws=0), dict(ws=0x109010), dict(wsb=8)):
        assert _policy(lib, **kw) == dk.DUALKV_ERR_WORKSPACE, kw
    for kw in (dict(dl=0), dict(g=0), dict(g=0x100004), dict(gh=0x301004), dict(g=0x105000), dict(gh=0x300000)):
        assert _policy(lib, True, **kw) == bad, kw
    assert lib.dualkv_policy_loss_workspace_bytes(2, dk.offsets(OK_OFF)) > 0
    assert lib.dualkv_policy_loss_workspace_bytes(2, dk.offsets([0, 3, 1])) == 0


@pytest.mark.parametrize("backward", [False, True])
def test_logprobs_vocabulary_limit(lib, backward):
    far = dict(x=1 << 44, dx=1 << 45, xs=1 << 31, dxs=1 << 31)
    for V in ((1 << 30) + 1, (1 << 31) - 1):
        assert _logp(lib, backward, V=V, **far) == dk.DUALKV_ERR_INVALID
    if not torch.cuda.is_available():  # the largest passes the checks, and there is no device to run it
        assert _logp(lib, backward, V=1 << 30, **far) == dk.DUALKV_ERR_CUDA
