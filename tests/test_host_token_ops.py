"""Host-side argument validation of the per-token operators around attention: every
case below is refused before any device work; no pointer is dereferenced."""
import ctypes

import pytest

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
