"""Host-side argument validation of the paged cache and the attention over it: every case below is refused
before any device work; no pointer is dereferenced."""
import ctypes

import pytest
import torch

from shared_prompt_exact_gb300 import build as pbuild
from shared_prompt_exact_gb300 import dualkv as dk

OFF = [0, 2, 3]
BAD, ALIGN = dk.DUALKV_ERR_INVALID, dk.DUALKV_ERR_ALIGN


@pytest.fixture(scope="module")
def lib():
    pbuild.build()
    return dk.load()


def _vp(x):
    return ctypes.c_void_p(x)


def _off(values):
    return None if values is None else (ctypes.c_int32 * len(values))(*values)


# pools of 4 pages x 2 heads x 16 tokens x 64 values: 16 KB in bf16, 4 KB + 512 B in 4 bits
CACHE = dict(ck=0x1000000, cv=0x1100000, cks=0, cvs=0, pool=4, ps=16, bits=16)
CACHE4 = dict(CACHE, cks=0x1200000, cvs=0x1300000, bits=4)


def _cache(a):
    if a.get("no_cache"):
        return None
    return ctypes.byref(dk._CacheStruct(a["ck"], a["cv"], a["cks"] or None, a["cvs"] or None, a["pool"], a["ps"], a["bits"]))


def _append(lib, **kw):
    a = dict(CACHE, q=0x100000, qs=256, k=0x200000, ks=128, v=0x280000, vs=128, qw=0x300000, kw=0x301000, wd=dk.DUALKV_BF16,
             w0=0.0, eps=1e-6, f=0x302000, rd=64, inter=0, pages=0x303000, mp=3, lens=0x304000, starts=0x305000, S=2, off=OFF,
             Hq=4, Hkv=2, D=64, qo=0x400000)
    a.update(kw)
    return lib.dualkv_cache_append(_vp(a["q"]), a["qs"], _vp(a["k"]), a["ks"], _vp(a["v"]), a["vs"], _vp(a["qw"]),
                                   _vp(a["kw"]), a["wd"], a["w0"], a["eps"], _vp(a["f"]), a["rd"], a["inter"], _cache(a),
                                   _vp(a["pages"]), a["mp"], _vp(a["lens"]), _vp(a["starts"]), a["S"], _off(a["off"]),
                                   a["Hq"], a["Hkv"], a["D"], _vp(a["qo"]), None)


def _read(lib, **kw):
    a = dict(CACHE, pages=0x303000, mp=3, lens=0x304000, S=2, off=OFF, Hkv=2, D=64, ko=0x400000, vo=0x500000)
    a.update(kw)
    return lib.dualkv_cache_read(_cache(a), _vp(a["pages"]), a["mp"], _vp(a["lens"]), a["S"], _off(a["off"]), a["Hkv"],
                                 a["D"], _vp(a["ko"]), _vp(a["vo"]), None)


def _decode(lib, **kw):
    a = dict(CACHE, q=0x100000, qs=256, pp=0x301000, mpp=2, pl=0x302000, pages=0x303000, mp=3, lens=0x304000, G=2, off=OFF,
             Hq=4, Hkv=2, D=64, scale=0.125, window=0, out=0x400000, lse=0x500000, ws=0x2000000, wsb=1 << 40)
    a.update(kw)
    return lib.dualkv_decode(_vp(a["q"]), a["qs"], _cache(a), _vp(a["pp"]), a["mpp"], _vp(a["pl"]), _vp(a["pages"]), a["mp"],
                             _vp(a["lens"]), a["G"], _off(a["off"]), a["Hq"], a["Hkv"], a["D"], a["scale"], a["window"],
                             _vp(a["out"]), _vp(a["lse"]), _vp(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("call", [_append, _read, _decode])
def test_cache_refusals(lib, call):
    for kw in (dict(no_cache=True), dict(D=96), dict(Hkv=0), dict(Hkv=-2), dict(pool=0), dict(pool=1 << 31), dict(ps=0), dict(ps=8),
               dict(ps=24), dict(ps=1 << 17), dict(bits=8), dict(ck=0), dict(cv=0), dict(cks=0x1200000, cvs=0x1300000),
               dict(CACHE4, cks=0), dict(CACHE4, cvs=0), dict(bits=4), dict(mp=0), dict(mp=-1), dict(mp=(1 << 27) + 1),
               dict(pages=0), dict(lens=0), dict(off=None), dict(off=[0, 3, 2]), dict(off=[1, 2, 3])):
        assert call(lib, **kw) == BAD, kw
    for kw in (dict(ck=0x1000008), dict(cv=0x1100002), dict(CACHE4, cks=0x1200004), dict(pages=0x303002), dict(lens=0x304001)):
        assert call(lib, **kw) == ALIGN, kw


def test_append_refusals(lib):
    for kw in (dict(S=0), dict(S=-1), dict(Hq=3), dict(Hq=0), dict(q=0), dict(k=0), dict(v=0), dict(qo=0), dict(starts=0),
               dict(qs=248), dict(qs=255), dict(ks=120), dict(vs=0), dict(vs=129), dict(qs=1 << 40), dict(kw=0), dict(qw=0),
               dict(wd=2), dict(eps=-1.0), dict(eps=float("nan")), dict(w0=float("inf")), dict(rd=-16), dict(rd=80), dict(rd=8),
               dict(f=0),
               # the cache or q_out over an input or one another
               dict(qo=0x100000), dict(qo=0x200080), dict(qo=0x280000), dict(qo=0x1003ff0), dict(ck=0x200000), dict(cv=0x303000 - 16),
               dict(cv=0x1000000), dict(CACHE4, cks=0x1000ff0), dict(CACHE4, cvs=0x304000 - 0x1f0), dict(qo=0x305000)):
        assert _append(lib, **kw) == BAD, kw
    for kw in (dict(q=0x100008), dict(v=0x280008), dict(qo=0x400008), dict(f=0x302004), dict(starts=0x305002)):
        assert _append(lib, **kw) == ALIGN, kw
    assert _append(lib, S=4096, off=[0] * 4096 + [1]) == dk.DUALKV_ERR_UNSUPPORTED
    # no rows: nothing to do, nothing looked at but the layout
    assert _append(lib, off=[0, 0, 0], q=0, k=0, v=0, qo=0, pages=0) == dk.DUALKV_OK


def test_read_refusals(lib):
    for kw in (dict(S=0), dict(ko=0), dict(vo=0), dict(ko=0x500000), dict(vo=0x1000000), dict(ko=0x304000), dict(CACHE4, vo=0x1200000)):
        assert _read(lib, **kw) == BAD, kw
    for kw in (dict(ko=0x400008), dict(vo=0x500004)):
        assert _read(lib, **kw) == ALIGN, kw
    assert _read(lib, S=4096, off=[0] * 4096 + [1]) == dk.DUALKV_ERR_UNSUPPORTED
    assert _read(lib, off=[0, 0, 0], ko=0, vo=0) == dk.DUALKV_OK


def test_decode_refusals(lib):
    nan = float("nan")
    for kw in (dict(G=0), dict(Hq=3), dict(Hq=1 << 20), dict(scale=0.0), dict(scale=-1.0), dict(scale=nan), dict(scale=3e38),
               dict(qs=248), dict(qs=250), dict(q=0), dict(out=0), dict(pp=0), dict(pl=0), dict(pp=0, pl=0), dict(mpp=0),
               dict(mpp=(1 << 27) + 1), dict(out=0x100000), dict(out=0x1000000), dict(lse=0x400000), dict(lse=0x304000),
               dict(out=0x301000), dict(ws=0x400000)):
        assert _decode(lib, **kw) == BAD, kw
    for kw in (dict(q=0x100004), dict(out=0x400008), dict(lse=0x500002), dict(pp=0x301001), dict(pl=0x302002)):
        assert _decode(lib, **kw) == ALIGN, kw
    off = dk.offsets(OFF)
    need = lib.dualkv_decode_workspace_bytes(2, off, 4, 2, 64)
    assert need > 0
    for kw in (dict(ws=0), dict(ws=0x2000080), dict(wsb=need - 1)):
        assert _decode(lib, **kw) == dk.DUALKV_ERR_WORKSPACE, kw
    assert _decode(lib, G=4096, off=[0] * 4096 + [1]) == dk.DUALKV_ERR_UNSUPPORTED
    assert _decode(lib, G=1, off=[0, 8193]) == dk.DUALKV_ERR_UNSUPPORTED
    assert _decode(lib, mp=(1 << 27) - 1, ps=16, G=1, off=[0, 4096]) == dk.DUALKV_ERR_UNSUPPORTED
    assert _decode(lib, off=[0, 0, 0], q=0, out=0, ws=0) == dk.DUALKV_OK
    assert lib.dualkv_decode_workspace_bytes(2, off, 4, 3, 64) == 0 and lib.dualkv_decode_workspace_bytes(2, off, 4, 2, 96) == 0


def test_binding_refuses_on_the_host():
    for bad in (dict(bits=8), dict(bits=4, D=48)):
        with pytest.raises(ValueError):
            dk.KVCache.empty(4, 2, 16, **{"D": 64, **bad}, device="cpu")
    with pytest.raises(ValueError):
        dk.KVCache(*(torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16) for _ in range(2)))
    with pytest.raises(ValueError):
        dk.dualkv_decode_workspace_bytes(2, [0, 1], 4, 2, 64)
    with pytest.raises(ValueError):
        dk.dualkv_decode_workspace_bytes(1, [0, 1], 1 << 33, 2, 64)
