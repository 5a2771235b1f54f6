"""ctypes binding of libdualkv.so (declared in include/dualkv.h).

Argument marshalling only: every step of the attention path runs in the
library's CUDA kernels.  The functions keep the C names and signatures
(tensors in place of raw pointers); ``forward``/``backward`` add buffer
allocation on top.  If the library is missing, loading raises: there is no
fallback implementation.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import os
import threading
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libdualkv.so")

DUALKV_OK = 0
DUALKV_ERR_INVALID = 1
DUALKV_ERR_ALIGN = 2
DUALKV_ERR_WORKSPACE = 3
DUALKV_ERR_CUDA = 4
DUALKV_ERR_DEVICE = 5
DUALKV_ERR_UNSUPPORTED = 6

# every symbol the header declares
EXPORTS = ("dualkv_fwd", "dualkv_bwd_workspace_bytes", "dualkv_bwd", "dualkv_build_index", "dualkv_rho",
           "dualkv_pairs", "dualkv_check_status", "dualkv_error_string", "dualkv_profile_enable",
           "dualkv_profile_read", "dualkv_selftest_timeout", "dualkv_bwd_noalloc", "dualkv_release",
           "dualkv_pack", "dualkv_unpack", "dualkv_fold", "dualkv_fwd_heads", "dualkv_bwd_heads",
           "dualkv_fwd_layers", "dualkv_bwd_layers", "dualkv_bwd_layers_workspace_bytes",
           "dualkv_selftest_kernel", "dualkv_plan_cache_info", "dualkv_qk_norm_rope",
           "dualkv_qk_norm_rope_bwd", "dualkv_qk_norm_rope_bwd_workspace_bytes", "dualkv_token_logprobs",
           "dualkv_token_logprobs_bwd", "dualkv_policy_loss", "dualkv_policy_loss_bwd",
           "dualkv_policy_loss_workspace_bytes", "dualkv_cache_append", "dualkv_cache_read", "dualkv_decode",
           "dualkv_decode_workspace_bytes")
NOALLOC_SCRATCH_BYTES = 32 << 20
_TOO_FAR = 1 << 31  # counts from here on would wrap on their way into a C int
KERNEL_KINDS = ("fwd", "prep", "dkv", "reduce", "dq", "pack", "rope", "logprobs", "policy", "cache", "decode")
DUALKV_BF16 = 0
DUALKV_F32 = 1
LOSS_REDUCTIONS = {"token_mean": 0, "seq_mean": 1, "seq_sum": 2}

_lock = threading.Lock()
_lib = None


class DualKVError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {error_string(code)} (code {code})")


class _CacheStruct(ctypes.Structure):
    """dualkv_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("pages", ctypes.c_int64), ("page_size", ctypes.c_int32),
                ("bits", ctypes.c_int32)]


def load(path: Optional[str] = None):
    """Load libdualkv.so; raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"{p} is missing: build it with shared_prompt_exact_gb300.build.build()")
        lib = ctypes.CDLL(p)
        vp, ci, cf = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
        i32p = ctypes.POINTER(ctypes.c_int32)
        lib.dualkv_fwd.argtypes = [vp, vp, vp, ci, ci, i32p, ci, ci, ci, cf, ci, vp, vp, vp]
        lib.dualkv_fwd.restype = ci
        lib.dualkv_bwd_workspace_bytes.argtypes = [ci, ci, i32p, ci, ci, ci, ci]
        lib.dualkv_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.dualkv_bwd.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, i32p, ci, ci, ci, cf, ci, vp, vp, vp, vp,
                                   ctypes.c_size_t, vp]
        lib.dualkv_bwd.restype = ci
        lib.dualkv_fwd_heads.argtypes = [vp, vp, vp, ci, ci, i32p, ci, ci, ci, cf, ci, ci, ci, vp, vp, vp]
        lib.dualkv_fwd_heads.restype = ci
        lib.dualkv_bwd_heads.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, i32p, ci, ci, ci, cf, ci, ci, ci, vp, vp,
                                         vp, vp, ctypes.c_size_t, vp]
        lib.dualkv_bwd_heads.restype = ci
        lib.dualkv_build_index.argtypes = [ci, ci, i32p, i32p, i32p, i32p, i32p]
        lib.dualkv_build_index.restype = ci
        lib.dualkv_rho.argtypes = [ci, ci, i32p]
        lib.dualkv_rho.restype = ctypes.c_double
        lib.dualkv_pairs.argtypes = [ci, ci, i32p, ci]
        lib.dualkv_pairs.restype = ctypes.c_int64
        lib.dualkv_check_status.argtypes = [vp]
        lib.dualkv_check_status.restype = ci
        lib.dualkv_error_string.argtypes = [ci]
        lib.dualkv_error_string.restype = ctypes.c_char_p
        lib.dualkv_profile_enable.argtypes = [ci]
        lib.dualkv_profile_enable.restype = ci
        lib.dualkv_profile_read.argtypes = [ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_int64)]
        lib.dualkv_profile_read.restype = ci
        lib.dualkv_bwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, ci, ci, i32p, ci, ci, ci, cf, ci, vp, vp, vp, vp]
        lib.dualkv_bwd_noalloc.restype = ci
        lib.dualkv_selftest_timeout.argtypes = [ctypes.c_uint64, vp]
        lib.dualkv_selftest_timeout.restype = ci
        lib.dualkv_selftest_kernel.argtypes = [ci, ctypes.c_uint64, vp]
        lib.dualkv_selftest_kernel.restype = ci
        lib.dualkv_plan_cache_info.argtypes = [ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int64)]
        lib.dualkv_plan_cache_info.restype = ci
        for name in ("dualkv_pack", "dualkv_unpack", "dualkv_fold"):
            getattr(lib, name).argtypes = [vp, vp, ci, ci, i32p, ci, vp]
            getattr(lib, name).restype = ci
        lib.dualkv_bwd_layers_workspace_bytes.argtypes = [ci, i32p, ci, ci, i32p, ci, ci, ci]
        lib.dualkv_bwd_layers_workspace_bytes.restype = ctypes.c_size_t
        lib.dualkv_fwd_layers.argtypes = [ci, vp, vp, vp, i32p, ci, ci, i32p, ci, ci, ci, cf, vp, vp, vp]
        lib.dualkv_fwd_layers.restype = ci
        lib.dualkv_bwd_layers.argtypes = [ci, vp, vp, vp, vp, vp, vp, i32p, ci, ci, i32p, ci, ci, ci, cf, vp, vp, vp,
                                          vp, ctypes.c_size_t, vp]
        lib.dualkv_bwd_layers.restype = ci
        i64 = ctypes.c_int64
        rope = [vp, vp, ci, cf, cf, vp, ci, ci, ci, ci, i32p, ci, ci, ci]
        lib.dualkv_qk_norm_rope.argtypes = [vp, i64, vp, i64] + rope + [vp, vp, vp]
        lib.dualkv_qk_norm_rope.restype = ci
        lib.dualkv_qk_norm_rope_bwd_workspace_bytes.argtypes = [ci, ci, i32p, ci, ci, ci]
        lib.dualkv_qk_norm_rope_bwd_workspace_bytes.restype = ctypes.c_size_t
        lib.dualkv_qk_norm_rope_bwd.argtypes = [vp, i64, vp, i64, vp, vp] + rope + [vp, i64, vp, i64, vp, vp, vp,
                                                                                     ctypes.c_size_t, vp]
        lib.dualkv_qk_norm_rope_bwd.restype = ci
        logp = [vp, i64, ci, ci, cf, vp, ci, ci, i32p]
        lib.dualkv_token_logprobs.argtypes = logp + [vp, vp, vp, vp]
        lib.dualkv_token_logprobs.restype = ci
        lib.dualkv_token_logprobs_bwd.argtypes = logp + [vp, vp, vp, vp, vp, i64, vp]
        lib.dualkv_token_logprobs_bwd.restype = ci
        cd = ctypes.c_double
        lib.dualkv_policy_loss_workspace_bytes.argtypes = [ci, i32p]
        lib.dualkv_policy_loss_workspace_bytes.restype = ctypes.c_size_t
        lib.dualkv_policy_loss.argtypes = [vp, vp, vp, vp, vp, ci, vp, ci, i32p, cd, cd, cd, cd, cd, ci, vp, vp, vp, vp,
                                           ctypes.c_size_t, vp]
        lib.dualkv_policy_loss.restype = ci
        lib.dualkv_policy_loss_bwd.argtypes = [vp, vp, vp, vp, ci, vp, ci, i32p, cd, cd, cd, cd, cd, vp, vp, vp, vp, vp]
        lib.dualkv_policy_loss_bwd.restype = ci
        cache = ctypes.POINTER(_CacheStruct)
        lib.dualkv_cache_append.argtypes = ([vp, i64, vp, i64, vp, i64, vp, vp, ci, cf, cf, vp, ci, ci, cache, vp, ci, vp, vp,
                                             ci, i32p, ci, ci, ci, vp, vp])
        lib.dualkv_cache_append.restype = ci
        lib.dualkv_cache_read.argtypes = [cache, vp, ci, vp, ci, i32p, ci, ci, vp, vp, vp]
        lib.dualkv_cache_read.restype = ci
        lib.dualkv_decode_workspace_bytes.argtypes = [ci, i32p, ci, ci, ci]
        lib.dualkv_decode_workspace_bytes.restype = ctypes.c_size_t
        lib.dualkv_decode.argtypes = [vp, i64, cache, vp, ci, vp, vp, ci, vp, ci, i32p, ci, ci, ci, cf, ci, vp, vp, vp,
                                      ctypes.c_size_t, vp]
        lib.dualkv_decode.restype = ci
        lib.dualkv_release.argtypes = []
        lib.dualkv_release.restype = None
        _lib = lib
        return lib


def error_string(code: int) -> str:
    return load().dualkv_error_string(int(code)).decode()


def _offsets(R_offsets: Sequence[int]):
    """R_offsets as a ctypes int32 array; one that already is such an array is passed on as it is,
    so a program with one layout for many calls can convert it once (``offsets``)."""
    if isinstance(R_offsets, ctypes.Array) and R_offsets._type_ is ctypes.c_int32:
        return R_offsets
    values = [int(x) for x in R_offsets]
    if values and not -_TOO_FAR <= min(values) <= max(values) < _TOO_FAR:
        raise ValueError(f"R_offsets must fit 32 bits, got {max(values, key=abs)}")
    return (ctypes.c_int32 * len(values))(*values)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return ctypes.c_void_p(stream.cuda_stream)
    return ctypes.c_void_p(int(stream))


def _check_dev(name, t, dtype):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_shapes(where, P, N, R_offsets, Hq, Hkv, D, **tensors):
    """Every attention tensor must have exactly its layout's shape: q, out, dout, dq
    (T, Hq, D); k, v, dk, dv (T, Hkv, D); lse (Hq, T), with T = P + R_offsets[N].  The
    library builds its TMA views from these sizes, so an undersized tensor would be read
    or written past its end; the check runs before anything reaches the C ABI."""
    N = int(N)
    if N < 1 or len(R_offsets) != N + 1:
        raise ValueError(f"{where}: R_offsets must hold N + 1 = {N + 1} entries, got {len(R_offsets)}")
    T = int(P) + int(R_offsets[N])
    want = {"q": (T, Hq, D), "out": (T, Hq, D), "dout": (T, Hq, D), "dq": (T, Hq, D),
            "k": (T, Hkv, D), "v": (T, Hkv, D), "dk": (T, Hkv, D), "dv": (T, Hkv, D), "lse": (Hq, T)}
    for name, t in tensors.items():
        shape = tuple(int(x) for x in want[name.split("[")[0]])
        if not isinstance(t, torch.Tensor):
            raise ValueError(f"{where}: {name} must be a tensor")
        if tuple(t.shape) != shape:
            raise ValueError(f"{where}: {name} must have shape {shape} for this layout, got {tuple(t.shape)}")


def _raise(code, where):
    if code != DUALKV_OK:
        raise DualKVError(code, where)


def dualkv_fwd(q, k, v, P, N, R_offsets, Hq, Hkv, D, scale, window, out, lse, stream=None) -> None:
    _check_shapes("dualkv_fwd", P, N, R_offsets, Hq, Hkv, D, q=q, k=k, v=v, out=out, lse=lse)
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("out", out, torch.bfloat16), ("lse", lse, torch.float32)):
        _check_dev(name, t, dt)
    off = _offsets(R_offsets)
    rc = load().dualkv_fwd(_ptr(q), _ptr(k), _ptr(v), int(P), int(N), off, int(Hq), int(Hkv), int(D),
                           float(scale), int(window), _ptr(out), _ptr(lse), _stream(stream))
    _raise(rc, "dualkv_fwd")


def dualkv_bwd_workspace_bytes(P, N, R_offsets, Hq, Hkv, D, window) -> int:
    return int(load().dualkv_bwd_workspace_bytes(int(P), int(N), _offsets(R_offsets), int(Hq), int(Hkv), int(D),
                                                  int(window)))


def dualkv_bwd(q, k, v, out, lse, dout, P, N, R_offsets, Hq, Hkv, D, scale, window, dq, dk, dv, workspace,
               workspace_bytes=None, stream=None) -> None:
    _check_shapes("dualkv_bwd", P, N, R_offsets, Hq, Hkv, D, q=q, k=k, v=v, out=out, lse=lse, dout=dout, dq=dq,
                  dk=dk, dv=dv)
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("out", out, torch.bfloat16), ("lse", lse, torch.float32), ("dout", dout, torch.bfloat16),
                        ("dq", dq, torch.bfloat16), ("dk", dk, torch.bfloat16), ("dv", dv, torch.bfloat16)):
        _check_dev(name, t, dt)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = load().dualkv_bwd(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), int(P), int(N),
                           _offsets(R_offsets), int(Hq), int(Hkv), int(D), float(scale), int(window), _ptr(dq),
                           _ptr(dk), _ptr(dv), _ptr(workspace), int(workspace_bytes), _stream(stream))
    _raise(rc, "dualkv_bwd")


def dualkv_fwd_heads(q, k, v, P, N, R_offsets, Hq, Hkv, D, scale, window, kv_head_begin, kv_head_end, out, lse,
                     stream=None) -> None:
    """dualkv_fwd restricted to kv-heads [kv_head_begin, kv_head_end) and their q-heads."""
    _check_shapes("dualkv_fwd_heads", P, N, R_offsets, Hq, Hkv, D, q=q, k=k, v=v, out=out, lse=lse)
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("out", out, torch.bfloat16), ("lse", lse, torch.float32)):
        _check_dev(name, t, dt)
    rc = load().dualkv_fwd_heads(_ptr(q), _ptr(k), _ptr(v), int(P), int(N), _offsets(R_offsets), int(Hq), int(Hkv),
                                 int(D), float(scale), int(window), int(kv_head_begin), int(kv_head_end), _ptr(out),
                                 _ptr(lse), _stream(stream))
    _raise(rc, "dualkv_fwd_heads")


def dualkv_bwd_heads(q, k, v, out, lse, dout, P, N, R_offsets, Hq, Hkv, D, scale, window, kv_head_begin,
                     kv_head_end, dq, dk, dv, workspace, workspace_bytes=None, stream=None) -> None:
    """dualkv_bwd restricted to kv-heads [kv_head_begin, kv_head_end) and their q-heads."""
    _check_shapes("dualkv_bwd_heads", P, N, R_offsets, Hq, Hkv, D, q=q, k=k, v=v, out=out, lse=lse, dout=dout,
                  dq=dq, dk=dk, dv=dv)
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("out", out, torch.bfloat16), ("lse", lse, torch.float32), ("dout", dout, torch.bfloat16),
                        ("dq", dq, torch.bfloat16), ("dk", dk, torch.bfloat16), ("dv", dv, torch.bfloat16)):
        _check_dev(name, t, dt)
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = load().dualkv_bwd_heads(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), int(P), int(N),
                                 _offsets(R_offsets), int(Hq), int(Hkv), int(D), float(scale), int(window),
                                 int(kv_head_begin), int(kv_head_end), _ptr(dq), _ptr(dk), _ptr(dv), _ptr(workspace),
                                 int(workspace_bytes), _stream(stream))
    _raise(rc, "dualkv_bwd_heads")


def _check_layer_shapes(where, n, P, N, R_offsets, Hq, Hkv, D, **stacks):
    for name, ts in stacks.items():
        if len(ts) != n:
            raise ValueError(f"{where}: {name}: expected {n} tensors, got {len(ts)}")
        for i, t in enumerate(ts):
            _check_shapes(where, P, N, R_offsets, Hq, Hkv, D, **{f"{name}[{i}]": t})


def _ptr_array(name, tensors, n, dtype):
    if len(tensors) != n:
        raise ValueError(f"{name}: expected {n} tensors, got {len(tensors)}")
    for i, t in enumerate(tensors):
        _check_dev(f"{name}[{i}]", t, dtype)
    return (ctypes.c_void_p * n)(*[t.data_ptr() for t in tensors])


def dualkv_bwd_layers_workspace_bytes(windows, P, N, R_offsets, Hq, Hkv, D) -> int:
    n = len(windows)
    return int(load().dualkv_bwd_layers_workspace_bytes(n, (ctypes.c_int32 * n)(*[int(x) for x in windows]), int(P),
                                                         int(N), _offsets(R_offsets), int(Hq), int(Hkv), int(D)))


def dualkv_fwd_layers(qs, ks, vs, windows, P, N, R_offsets, Hq, Hkv, D, scale, outs, lses, stream=None) -> None:
    """Forward of a layer stack: layer l uses qs[l], ks[l], vs[l] and windows[l]."""
    n = len(windows)
    _check_layer_shapes("dualkv_fwd_layers", n, P, N, R_offsets, Hq, Hkv, D, q=qs, k=ks, v=vs, out=outs, lse=lses)
    bf = torch.bfloat16
    rc = load().dualkv_fwd_layers(n, _ptr_array("q", qs, n, bf), _ptr_array("k", ks, n, bf), _ptr_array("v", vs, n, bf),
                                  (ctypes.c_int32 * n)(*[int(x) for x in windows]), int(P), int(N),
                                  _offsets(R_offsets), int(Hq), int(Hkv), int(D), float(scale),
                                  _ptr_array("out", outs, n, bf), _ptr_array("lse", lses, n, torch.float32),
                                  _stream(stream))
    _raise(rc, "dualkv_fwd_layers")


def dualkv_bwd_layers(qs, ks, vs, outs, lses, douts, windows, P, N, R_offsets, Hq, Hkv, D, scale, dqs, dks, dvs,
                      workspace, workspace_bytes=None, stream=None) -> None:
    """Backward of a layer stack, layers in the order given, one shared workspace."""
    n = len(windows)
    _check_layer_shapes("dualkv_bwd_layers", n, P, N, R_offsets, Hq, Hkv, D, q=qs, k=ks, v=vs, out=outs, lse=lses,
                        dout=douts, dq=dqs, dk=dks, dv=dvs)
    bf = torch.bfloat16
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = load().dualkv_bwd_layers(n, _ptr_array("q", qs, n, bf), _ptr_array("k", ks, n, bf), _ptr_array("v", vs, n, bf),
                                  _ptr_array("out", outs, n, bf), _ptr_array("lse", lses, n, torch.float32),
                                  _ptr_array("dout", douts, n, bf), (ctypes.c_int32 * n)(*[int(x) for x in windows]),
                                  int(P), int(N), _offsets(R_offsets), int(Hq), int(Hkv), int(D), float(scale),
                                  _ptr_array("dq", dqs, n, bf), _ptr_array("dk", dks, n, bf),
                                  _ptr_array("dv", dvs, n, bf), _ptr(workspace), int(workspace_bytes),
                                  _stream(stream))
    _raise(rc, "dualkv_bwd_layers")


def kv_head_ranges(Hkv: int, parts: int):
    """Contiguous kv-head groups [lo, hi) for `parts` ranks (sizes differ by at most one;
    a rank gets an empty range when parts > Hkv)."""
    Hkv, parts = int(Hkv), int(parts)
    if Hkv < 1 or parts < 1:
        raise ValueError("Hkv and parts must be positive")
    base, extra = divmod(Hkv, parts)
    out, lo = [], 0
    for r in range(parts):
        hi = lo + base + (1 if r < extra else 0)
        out.append((lo, hi))
        lo = hi
    return out


def dualkv_bwd_noalloc(q, k, v, out, lse, dout, P, N, R_offsets, Hq, Hkv, D, scale, window, dq, dk, dv,
                       stream=None) -> None:
    """dualkv_bwd without a workspace: for callers that cannot allocate device
    memory.  Its scratch is a fixed array inside the library (NOALLOC_SCRATCH_BYTES
    per GPU); calls overlapping on the GPU race on it.  Returns once the pass has
    finished on `stream`."""
    _check_shapes("dualkv_bwd_noalloc", P, N, R_offsets, Hq, Hkv, D, q=q, k=k, v=v, out=out, lse=lse, dout=dout,
                  dq=dq, dk=dk, dv=dv)
    for name, t, dt in (("q", q, torch.bfloat16), ("k", k, torch.bfloat16), ("v", v, torch.bfloat16),
                        ("out", out, torch.bfloat16), ("lse", lse, torch.float32), ("dout", dout, torch.bfloat16),
                        ("dq", dq, torch.bfloat16), ("dk", dk, torch.bfloat16), ("dv", dv, torch.bfloat16)):
        _check_dev(name, t, dt)
    rc = load().dualkv_bwd_noalloc(_ptr(q), _ptr(k), _ptr(v), _ptr(out), _ptr(lse), _ptr(dout), int(P), int(N),
                                   _offsets(R_offsets), int(Hq), int(Hkv), int(D), float(scale), int(window),
                                   _ptr(dq), _ptr(dk), _ptr(dv), _stream(stream))
    _raise(rc, "dualkv_bwd_noalloc")


def _pack_call(fn, name, src, dst, P, N, R_offsets, stream):
    for nm, t in (("src", src), ("dst", dst)):
        _check_dev(nm, t, torch.bfloat16)
        if t.dim() < 2:
            raise ValueError(f"{name}: {nm} must have a row dimension and at least one more")
    T = int(P) + int(R_offsets[N])
    T_rep = int(N) * int(P) + int(R_offsets[N])
    rows_src, rows_dst = (T, T_rep) if name == "dualkv_unpack" else (T_rep, T)
    if src.shape[0] != rows_src or dst.shape[0] != rows_dst:
        raise ValueError(f"{name}: expected {rows_src} source and {rows_dst} destination rows, "
                         f"got {src.shape[0]} and {dst.shape[0]}")
    row_elems = src.numel() // rows_src
    if dst.numel() // rows_dst != row_elems:
        raise ValueError(f"{name}: src and dst rows must have the same number of elements")
    rc = fn(_ptr(src), _ptr(dst), int(P), int(N), _offsets(R_offsets), int(row_elems), _stream(stream))
    _raise(rc, name)


def dualkv_pack(x_rep, x_packed, P, N, R_offsets, stream=None) -> None:
    """x_rep [N*P + R_offsets[N], ...] -> x_packed [P + R_offsets[N], ...] (prompt rows from replica 0)."""
    _pack_call(load().dualkv_pack, "dualkv_pack", x_rep, x_packed, P, N, R_offsets, stream)


def dualkv_unpack(x_packed, x_rep, P, N, R_offsets, stream=None) -> None:
    """x_packed [T, ...] -> x_rep [T_rep, ...] (prompt rows copied into every replica)."""
    _pack_call(load().dualkv_unpack, "dualkv_unpack", x_packed, x_rep, P, N, R_offsets, stream)


def dualkv_fold(g_rep, g_packed, P, N, R_offsets, stream=None) -> None:
    """g_rep [T_rep, ...] -> g_packed [T, ...]: prompt rows summed over the N replicas (fp32, in order)."""
    _pack_call(load().dualkv_fold, "dualkv_fold", g_rep, g_packed, P, N, R_offsets, stream)


def offsets(R_offsets: Sequence[int]):
    """R_offsets as a ctypes int32 array, which every call here takes in place of the sequence."""
    return _offsets(R_offsets)


# ------------------------------------------------------------------ per-token operators
_DTYPE_CODES = {torch.bfloat16: DUALKV_BF16, torch.float32: DUALKV_F32}
_BF16, _F32, _I64 = (torch.bfloat16,), (torch.float32,), (torch.int64,)
_MASK_DTYPES = (torch.bool, torch.uint8)
_Tensor = torch.Tensor


def _arg(where, name, t, shape, dtypes, device):
    """Address of a contiguous CUDA tensor on the calling thread's current device, with this shape and one of these
    dtypes.  Raises if it is none."""
    if (isinstance(t, _Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == device
            and t.is_contiguous()):
        return t.data_ptr()
    _refuse(where, name, t, shape, dtypes, device, "must be contiguous")


def _opt(where, name, t, shape, dtypes, device):
    """The same for a tensor that may be missing."""
    return None if t is None else _arg(where, name, t, shape, dtypes, device)


def _rows(where, name, t, shape, inner, dtypes, device):
    """Address and row stride (in elements) of a CUDA tensor that is contiguous within each row of its first
    dimension: `inner` are the strides behind that one.  A single row has the stride that its width gives."""
    if isinstance(t, _Tensor) and t.dtype in dtypes and t.shape == shape and t.get_device() == device:
        strides = t.stride()
        if strides[1:] == inner or all(n == 1 or a == b for n, a, b in zip(shape[1:], strides[1:], inner)):
            return t.data_ptr(), strides[0] if shape[0] > 1 else shape[1] * inner[0]
    _refuse(where, name, t, shape, dtypes, device, "must be contiguous within its rows")


def _refuse(where, name, t, shape, dtypes, device, layout):
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise ValueError(f"{where}: {name} must be a CUDA tensor")
    if t.get_device() != device:
        raise ValueError(f"{where}: {name} is on cuda:{t.get_device()}, the current device is cuda:{device}")
    if t.dtype not in dtypes:
        raise ValueError(f"{where}: {name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{where}: {name} must have shape {tuple(shape)} for this call, got {tuple(t.shape)}")
    raise ValueError(f"{where}: {name} {layout}")


# the current stream's handle without an object around it, where this PyTorch has that (1 us per call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_of(stream, device):
    """The stream's handle: the current one of the (current) device unless given."""
    if stream is None:
        return _raw_stream(device) if _raw_stream else torch.cuda.current_stream(device).cuda_stream
    return _stream(stream)


def _layout_rows(where, P, N, R_offsets):
    """Packed rows of a layout."""
    P, N = int(P), int(N)
    if N < 1 or len(R_offsets) != N + 1:
        raise ValueError(f"{where}: R_offsets must hold N + 1 = {N + 1} entries, got {len(R_offsets)}")
    if not 0 <= P < _TOO_FAR:
        raise ValueError(f"{where}: P must be a count of tokens, got {P}")
    return P + int(R_offsets[N])


def _counts(where, **counts):
    """Refuses a count that a C int would not hold."""
    for name, v in counts.items():
        if not -_TOO_FAR <= v < _TOO_FAR:
            raise ValueError(f"{where}: {name} must fit 32 bits, got {v}")


def _rope_args(where, q, k, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved, P, N, R_offsets, Hq,
               Hkv, D):
    """Checks shared by the forward and the backward; returns (rows, device, q and k as the C call takes them, the
    arguments from the weights to D)."""
    T = _layout_rows(where, P, N, R_offsets)
    dev = torch.cuda.current_device()
    if max(Hq, Hkv, D, rope_dim) >= _TOO_FAR:
        _counts(where, Hq=Hq, Hkv=Hkv, D=D, rope_dim=rope_dim)
    inner = (D, 1)
    qk = _rows(where, "q", q, (T, Hq, D), inner, _BF16, dev) + _rows(where, "k", k, (T, Hkv, D), inner, _BF16, dev)
    if (q_weight is None) != (k_weight is None):
        raise ValueError(f"{where}: q_weight and k_weight go together")
    qw = kw = None
    code = DUALKV_F32
    if q_weight is not None:
        qw = _arg(where, "q_weight", q_weight, (D,), _DTYPE_CODES, dev)
        kw = _arg(where, "k_weight", k_weight, (D,), (q_weight.dtype,), dev)
        code = _DTYPE_CODES[q_weight.dtype]
    rope_dim = int(rope_dim)
    f = _arg(where, "inv_freq", inv_freq, (rope_dim // 2,), _F32, dev) if rope_dim else None
    return T, dev, qk, (qw, kw, code, float(weight_offset), float(eps), f, rope_dim, 1 if interleaved else 0, int(P),
                        int(N), _offsets(R_offsets), int(Hq), int(Hkv), int(D))


def dualkv_qk_norm_rope(q, k, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved, P, N, R_offsets,
                        Hq, Hkv, D, q_out, k_out, stream=None) -> None:
    """Per-head RMS norm and position rotation of packed q [T, Hq, D] and k [T, Hkv, D] (rows may be strided, as
    columns of a fused projection are) into the contiguous q_out, k_out that dualkv_fwd reads."""
    where = "dualkv_qk_norm_rope"
    T, dev, qk, args = _rope_args(where, q, k, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved, P,
                                  N, R_offsets, Hq, Hkv, D)
    rc = load().dualkv_qk_norm_rope(*qk, *args, _arg(where, "q_out", q_out, (T, Hq, D), _BF16, dev),
                                    _arg(where, "k_out", k_out, (T, Hkv, D), _BF16, dev), _stream_of(stream, dev))
    _raise(rc, where)


def dualkv_qk_norm_rope_bwd_workspace_bytes(P, N, R_offsets, Hq, Hkv, D) -> int:
    _counts("dualkv_qk_norm_rope_bwd_workspace_bytes", P=P, N=N, Hq=Hq, Hkv=Hkv, D=D)
    return int(load().dualkv_qk_norm_rope_bwd_workspace_bytes(int(P), int(N), _offsets(R_offsets), int(Hq), int(Hkv),
                                                              int(D)))


def dualkv_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved,
                            P, N, R_offsets, Hq, Hkv, D, dq, dk, dq_weight, dk_weight, workspace, workspace_bytes=None,
                            stream=None) -> None:
    """Gradients of dualkv_qk_norm_rope: dq, dk (rows may be strided) and, with weights, dq_weight, dk_weight."""
    where = "dualkv_qk_norm_rope_bwd"
    T, dev, qk, args = _rope_args(where, q, k, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved, P,
                                  N, R_offsets, Hq, Hkv, D)
    up = (_arg(where, "dq_out", dq_out, (T, Hq, D), _BF16, dev), _arg(where, "dk_out", dk_out, (T, Hkv, D), _BF16, dev))
    out = (_rows(where, "dq", dq, (T, Hq, D), (D, 1), _BF16, dev)
           + _rows(where, "dk", dk, (T, Hkv, D), (D, 1), _BF16, dev))
    gw = (None, None)
    if q_weight is not None:
        gw = (_arg(where, "dq_weight", dq_weight, (D,), _F32, dev), _arg(where, "dk_weight", dk_weight, (D,), _F32, dev))
    rc = load().dualkv_qk_norm_rope_bwd(*qk, *up, *args, *out, *gw,
                                        *_workspace_args(where, workspace, workspace_bytes, dev), _stream_of(stream, dev))
    _raise(rc, where)


def _logits_args(where, logits, tokens, scale, P, N, R_offsets):
    """Checks shared by the forward and the backward; returns (rows, tokens, device, the arguments up to R_offsets)."""
    n = _layout_rows(where, P, N, R_offsets) - int(P)
    M = n + 1 if int(P) > 0 else n
    dev = torch.cuda.current_device()
    if not isinstance(logits, _Tensor) or logits.dim() != 2:
        raise ValueError(f"{where}: logits must be a tensor of rows")
    V = logits.shape[1]
    if V >= _TOO_FAR:
        _counts(where, V=V)
    return M, n, dev, (*_rows(where, "logits", logits, (M, V), (1,), _DTYPE_CODES, dev), _DTYPE_CODES[logits.dtype], V,
                       float(scale), _arg(where, "tokens", tokens, (n,), _I64, dev), int(P), int(N), _offsets(R_offsets))


def dualkv_token_logprobs(logits, tokens, scale, P, N, R_offsets, logp, entropy, lse, stream=None) -> None:
    """Log-probabilities (and, unless None, entropies) of the response tokens from the logits of packed rows
    P - 1 .. T - 1 (all rows if P = 0); lse, unless None, gets each row's log-sum-exp."""
    where = "dualkv_token_logprobs"
    M, n, dev, args = _logits_args(where, logits, tokens, scale, P, N, R_offsets)
    rc = load().dualkv_token_logprobs(*args, _arg(where, "logp", logp, (n,), _F32, dev),
                                      _opt(where, "entropy", entropy, (n,), _F32, dev),
                                      _opt(where, "lse", lse, (M,), _F32, dev), _stream_of(stream, dev))
    _raise(rc, where)


def dualkv_token_logprobs_bwd(logits, tokens, scale, P, N, R_offsets, lse, entropy, dlogp, dentropy, dlogits,
                              stream=None) -> None:
    """Gradient of the logits from dlogp (and, unless None, dentropy); dlogits may be logits itself."""
    where = "dualkv_token_logprobs_bwd"
    M, n, dev, args = _logits_args(where, logits, tokens, scale, P, N, R_offsets)
    if dentropy is not None and entropy is None:
        raise ValueError(f"{where}: dentropy needs entropy")
    rc = load().dualkv_token_logprobs_bwd(*args, _arg(where, "lse", lse, (M,), _F32, dev),
                                          _opt(where, "entropy", entropy, (n,), _F32, dev),
                                          _arg(where, "dlogp", dlogp, (n,), _F32, dev),
                                          _opt(where, "dentropy", dentropy, (n,), _F32, dev),
                                          *_rows(where, "dlogits", dlogits, logits.shape, (1,), (logits.dtype,), dev),
                                          _stream_of(stream, dev))
    _raise(rc, where)


def _policy_args(where, logp, old_logp, ref_logp, advantages, mask, N, R_offsets, clip_low, clip_high, dual_clip, kl_coef,
                 entropy_coef, reduction, per_token):
    """Checks shared by the forward and the backward; returns (tokens, device, the log-probabilities, the arguments
    from the advantages to the coefficients)."""
    n = _layout_rows(where, 0, N, R_offsets)
    dev = torch.cuda.current_device()
    if reduction not in LOSS_REDUCTIONS:
        raise ValueError(f"{where}: reduction must be one of {tuple(LOSS_REDUCTIONS)}, got {reduction!r}")
    kl_coef = float(kl_coef)
    if kl_coef != 0.0 and ref_logp is None:
        raise ValueError(f"{where}: kl_coef needs ref_logp")
    shape = (n,)
    probs = (_arg(where, "logp", logp, shape, _F32, dev), _arg(where, "old_logp", old_logp, shape, _F32, dev),
             _opt(where, "ref_logp", ref_logp, shape, _F32, dev))
    N = int(N)
    per_token = _per_token(where, advantages, N, n, R_offsets, per_token)
    adv = _arg(where, "advantages", advantages, shape if per_token else (N,), _F32, dev)
    return n, dev, probs, (adv, per_token, _opt(where, "mask", mask, shape, _MASK_DTYPES, dev), N, _offsets(R_offsets),
                           float(clip_low), float(clip_high), float(dual_clip), kl_coef, float(entropy_coef))


def _per_token(where, advantages, N, n, R_offsets, per_token):
    """Whether advantages hold one value per token rather than per segment: as the caller says, else by their length.
    A length that fits both ways in a layout where it makes a difference has to be told."""
    if per_token is not None:
        return 1 if per_token else 0
    if not isinstance(advantages, _Tensor) or advantages.dim() != 1:
        raise ValueError(f"{where}: advantages must be a tensor of one dimension")
    if n == N and any(int(R_offsets[i]) != i for i in range(n)):
        raise ValueError(f"{where}: {n} advantages for {n} segments of {n} tokens in all: pass per_token")
    return 1 if advantages.shape[0] != N else 0


def dualkv_policy_loss_workspace_bytes(N, R_offsets) -> int:
    _counts("dualkv_policy_loss_workspace_bytes", N=N)
    return int(load().dualkv_policy_loss_workspace_bytes(int(N), _offsets(R_offsets)))


def dualkv_policy_loss(logp, old_logp, ref_logp, entropy, advantages, mask, N, R_offsets, clip_low, clip_high, dual_clip,
                       kl_coef, entropy_coef, reduction, loss, stats, weights, workspace, workspace_bytes=None,
                       stream=None, per_token=None) -> None:
    """Clipped policy loss with a KL term and an entropy bonus over packed response tokens.  advantages: [N], or one
    per token (per_token, by default told from the length)."""
    where = "dualkv_policy_loss"
    n, dev, probs, args = _policy_args(where, logp, old_logp, ref_logp, advantages, mask, N, R_offsets, clip_low,
                                       clip_high, dual_clip, kl_coef, entropy_coef, reduction, per_token)
    if float(entropy_coef) != 0.0 and entropy is None:
        raise ValueError(f"{where}: entropy_coef needs entropy")
    rc = load().dualkv_policy_loss(*probs, _opt(where, "entropy", entropy, (n,), _F32, dev), *args,
                                   LOSS_REDUCTIONS[reduction], _arg(where, "loss", loss, (1,), _F32, dev),
                                   _arg(where, "stats", stats, (4,), _F32, dev),
                                   _arg(where, "weights", weights, (int(N),), _F32, dev),
                                   *_workspace_args(where, workspace, workspace_bytes, dev), _stream_of(stream, dev))
    _raise(rc, where)


def dualkv_policy_loss_bwd(logp, old_logp, ref_logp, advantages, mask, N, R_offsets, clip_low, clip_high, dual_clip,
                           kl_coef, entropy_coef, reduction, dloss, weights, dlogp, dentropy, stream=None,
                           per_token=None) -> None:
    """Gradients of dualkv_policy_loss: dlogp and, unless None, dentropy (the reduction is in weights)."""
    where = "dualkv_policy_loss_bwd"
    n, dev, probs, args = _policy_args(where, logp, old_logp, ref_logp, advantages, mask, N, R_offsets, clip_low,
                                       clip_high, dual_clip, kl_coef, entropy_coef, reduction, per_token)
    if not isinstance(dloss, _Tensor) or dloss.numel() != 1:
        raise ValueError(f"{where}: dloss must be a tensor of one value")
    rc = load().dualkv_policy_loss_bwd(*probs, *args, _arg(where, "dloss", dloss, dloss.shape, _F32, dev),
                                       _arg(where, "weights", weights, (int(N),), _F32, dev),
                                       _arg(where, "dlogp", dlogp, (n,), _F32, dev),
                                       _opt(where, "dentropy", dentropy, (n,), _F32, dev), _stream_of(stream, dev))
    _raise(rc, where)


# ------------------------------------------------------------------ paged key/value cache
CACHE_GROUP = 32  # values that share a scale in a 4-bit cache
_I32, _U8 = (torch.int32,), (torch.uint8,)


class KVCache:
    """A paged cache of keys and values: bf16 pools [pages, Hkv, page_size, D], or 4-bit codes, two to a byte
    (uint8 [pages, Hkv, page_size, D / 2]), with bf16 scales [pages, Hkv, page_size, D / 32].  It wraps tensors
    that the caller owns; ``KVCache.empty`` allocates them.  A cache keeps the tensors that it was made of, where
    they were: calls refuse it once one of them has other memory (``set_``, ``resize_`` beyond it)."""

    __slots__ = ("_pools", "_at", "_c", "_shape", "_device")

    def __init__(self, k, v, k_scale=None, v_scale=None):
        if not isinstance(k, _Tensor) or not k.is_cuda or k.dim() != 4:
            raise ValueError("KVCache: k must be a CUDA tensor [pages, heads, page size, values]")
        shape, dev = k.shape, k.get_device()
        pages, Hkv, ps, width = shape
        if k_scale is None and v_scale is None:
            at = _arg("KVCache", "k", k, shape, _BF16, dev), _arg("KVCache", "v", v, shape, _BF16, dev)
            struct = _CacheStruct(*at, None, None, pages, ps, 16)
        elif k_scale is None or v_scale is None:
            raise ValueError("KVCache: k_scale and v_scale go together")
        else:
            width *= 2
            groups = (pages, Hkv, ps, width // CACHE_GROUP)
            at = (_arg("KVCache", "k", k, shape, _U8, dev), _arg("KVCache", "v", v, shape, _U8, dev),
                  _arg("KVCache", "k_scale", k_scale, groups, _BF16, dev),
                  _arg("KVCache", "v_scale", v_scale, groups, _BF16, dev))
            struct = _CacheStruct(*at, pages, ps, 4)
        self._pools, self._at, self._c = (k, v, k_scale, v_scale), at, struct
        self._shape, self._device = (pages, Hkv, ps, width), dev

    k, v, k_scale, v_scale = (property(lambda self, i=i: self._pools[i]) for i in range(4))
    pages, Hkv, page_size, D = (property(lambda self, i=i: self._shape[i]) for i in range(4))
    device = property(lambda self: self._device)
    bits = property(lambda self: self._c.bits)

    @classmethod
    def empty(cls, pages, Hkv, page_size, D, bits=16, device="cuda"):
        """A cache of uninitialised pages."""
        if bits not in (16, 4):
            raise ValueError(f"KVCache: bits must be 16 or 4, got {bits}")
        shape = (pages, Hkv, page_size)
        if bits == 16:
            return cls(*(torch.empty(*shape, D, dtype=torch.bfloat16, device=device) for _ in range(2)))
        if D % CACHE_GROUP:
            raise ValueError(f"KVCache: D must be a multiple of {CACHE_GROUP}, got {D}")
        return cls(*(torch.empty(*shape, D // 2, dtype=torch.uint8, device=device) for _ in range(2)),
                   *(torch.empty(*shape, D // CACHE_GROUP, dtype=torch.bfloat16, device=device) for _ in range(2)))


def _cache_arg(where, cache, Hkv, D, device):
    if not isinstance(cache, KVCache):
        raise ValueError(f"{where}: cache must be a KVCache")
    _, heads, _, width = cache._shape
    if heads != Hkv or width != D:
        raise ValueError(f"{where}: cache holds {heads} heads of {width}, not {Hkv} of {D}")
    if cache._device != device:
        raise ValueError(f"{where}: cache is on cuda:{cache._device}, the current device is cuda:{device}")
    k, v, ks, vs = cache._pools
    at = (k.data_ptr(), v.data_ptr()) if ks is None else (k.data_ptr(), v.data_ptr(), ks.data_ptr(), vs.data_ptr())
    if at != cache._at:
        raise ValueError(f"{where}: cache: its tensors have other memory by now, wrap them in a new KVCache")
    return cache._c


def _table(where, name, pages, streams, device):
    """Address and width of a page table."""
    if isinstance(pages, _Tensor) and pages.dtype == torch.int32 and pages.is_contiguous() and pages.get_device() == device:
        shape = pages.shape
        if len(shape) == 2 and shape[0] == streams and shape[1] < _TOO_FAR:
            return pages.data_ptr(), shape[1]
    if not isinstance(pages, _Tensor) or pages.dim() != 2 or pages.shape[1] >= _TOO_FAR:
        raise ValueError(f"{where}: {name} must be a tensor [streams, most pages]")
    _refuse(where, name, pages, torch.Size((streams, pages.shape[1])), _I32, device, "must be contiguous")


def _last_offset(where, name, n, offsets):
    """Rows that `offsets` (n + 1 entries) describe."""
    if n < 1 or len(offsets) != n + 1:
        raise ValueError(f"{where}: {name} must hold {n + 1} entries, got {len(offsets)}")
    last = int(offsets[n])
    if last < 0:
        raise ValueError(f"{where}: {name} must not decrease, got {last} as the last")
    return last


def dualkv_cache_append(q, k, v, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved, cache, pages, lens,
                        starts, S, row_offsets, Hq, Hkv, D, q_out, stream=None) -> None:
    """Norm and rotation of new rows q [T, Hq, D], k [T, Hkv, D] of S streams (rows may be strided, as columns of a
    fused projection are): q into q_out, k and v into the pages that `pages` [S, most pages] names.  lens: tokens of each
    stream after this call; starts: position of its token 0."""
    where = "dualkv_cache_append"
    S, rope_dim = int(S), int(rope_dim)
    T = _last_offset(where, "row_offsets", S, row_offsets)
    dev = torch.cuda.current_device()
    if Hq >= _TOO_FAR or Hkv >= _TOO_FAR or D >= _TOO_FAR or rope_dim >= _TOO_FAR:
        _counts(where, Hq=Hq, Hkv=Hkv, D=D, rope_dim=rope_dim)
    inner = (D, 1)
    qkv = (_rows(where, "q", q, (T, Hq, D), inner, _BF16, dev) + _rows(where, "k", k, (T, Hkv, D), inner, _BF16, dev)
           + _rows(where, "v", v, (T, Hkv, D), inner, _BF16, dev))
    if (q_weight is None) != (k_weight is None):
        raise ValueError(f"{where}: q_weight and k_weight go together")
    qw = kw = None
    code = DUALKV_F32
    if q_weight is not None:
        qw = _arg(where, "q_weight", q_weight, (D,), _DTYPE_CODES, dev)
        kw = _arg(where, "k_weight", k_weight, (D,), (q_weight.dtype,), dev)
        code = _DTYPE_CODES[q_weight.dtype]
    f = _arg(where, "inv_freq", inv_freq, (rope_dim // 2,), _F32, dev) if rope_dim else None
    table, width = _table(where, "pages", pages, S, dev)
    rc = load().dualkv_cache_append(*qkv, qw, kw, code, float(weight_offset), float(eps), f, rope_dim,
                                    1 if interleaved else 0, _cache_arg(where, cache, Hkv, D, dev), table, width,
                                    _arg(where, "lens", lens, (S,), _I32, dev),
                                    _arg(where, "starts", starts, (S,), _I32, dev), S, _offsets(row_offsets), int(Hq),
                                    int(Hkv), int(D), _arg(where, "q_out", q_out, (T, Hq, D), _BF16, dev),
                                    _stream_of(stream, dev))
    _raise(rc, where)


def dualkv_cache_read(cache, pages, lens, S, row_offsets, Hkv, D, k_out, v_out, stream=None) -> None:
    """The last rows of each stream (as many as row_offsets gives it) back as dense keys and values [T, Hkv, D]."""
    where = "dualkv_cache_read"
    S = int(S)
    T = _last_offset(where, "row_offsets", S, row_offsets)
    dev = torch.cuda.current_device()
    table, width = _table(where, "pages", pages, S, dev)
    shape = (T, Hkv, D)
    rc = load().dualkv_cache_read(_cache_arg(where, cache, Hkv, D, dev), table, width,
                                  _arg(where, "lens", lens, (S,), _I32, dev), S, _offsets(row_offsets), int(Hkv), int(D),
                                  _arg(where, "k_out", k_out, shape, _BF16, dev),
                                  _arg(where, "v_out", v_out, shape, _BF16, dev), _stream_of(stream, dev))
    _raise(rc, where)


def dualkv_decode_workspace_bytes(G, groups, Hq, Hkv, D) -> int:
    _counts("dualkv_decode_workspace_bytes", G=G, Hq=Hq, Hkv=Hkv, D=D)
    _last_offset("dualkv_decode_workspace_bytes", "groups", int(G), groups)
    return int(load().dualkv_decode_workspace_bytes(int(G), _offsets(groups), int(Hq), int(Hkv), int(D)))


def dualkv_decode(q, cache, prompt_pages, prompt_lens, pages, lens, G, groups, Hq, Hkv, D, scale, window, out, lse, workspace,
                  workspace_bytes=None, stream=None) -> None:
    """Attention of one new token per response, q [B, Hq, D] (rows may be strided), over the prompt that its group
    shares and its own tokens.  groups: responses before each group's first, B in all; prompt_pages and prompt_lens may
    be None (no prompts), lse may be."""
    where = "dualkv_decode"
    G = int(G)
    B = _last_offset(where, "groups", G, groups)
    dev = torch.cuda.current_device()
    if Hq >= _TOO_FAR or Hkv >= _TOO_FAR or D >= _TOO_FAR or not -_TOO_FAR <= window < _TOO_FAR:
        _counts(where, Hq=Hq, Hkv=Hkv, D=D, window=window)
    if (prompt_pages is None) != (prompt_lens is None):
        raise ValueError(f"{where}: prompt_pages and prompt_lens go together")
    prompts = (None, 0, None)
    if prompt_pages is not None:
        prompts = (*_table(where, "prompt_pages", prompt_pages, G, dev),
                   _arg(where, "prompt_lens", prompt_lens, (G,), _I32, dev))
    table, width = _table(where, "pages", pages, B, dev)
    rc = load().dualkv_decode(*_rows(where, "q", q, (B, Hq, D), (D, 1), _BF16, dev),
                              _cache_arg(where, cache, Hkv, D, dev), *prompts, table, width,
                              _arg(where, "lens", lens, (B,), _I32, dev), G, _offsets(groups), int(Hq), int(Hkv), int(D),
                              float(scale), int(window), _arg(where, "out", out, (B, Hq, D), _BF16, dev),
                              _opt(where, "lse", lse, (Hq, B), _F32, dev),
                              *_workspace_args(where, workspace, workspace_bytes, dev), _stream_of(stream, dev))
    _raise(rc, where)


def _workspace_args(where, workspace, workspace_bytes, device):
    """(address, bytes) of a workspace tensor, (None, 0) for None; no more than it holds may be claimed."""
    if workspace is None:
        return None, 0
    if not isinstance(workspace, _Tensor) or not workspace.is_cuda or not workspace.is_contiguous():
        raise ValueError(f"{where}: workspace must be a contiguous CUDA tensor")
    if workspace.get_device() != device:
        raise ValueError(f"{where}: workspace is on cuda:{workspace.get_device()}, the current device is cuda:{device}")
    held = workspace.numel() * workspace.element_size()
    if workspace_bytes is not None and int(workspace_bytes) > held:
        raise ValueError(f"{where}: workspace holds {held} bytes, not {workspace_bytes}")
    return workspace.data_ptr(), held if workspace_bytes is None else int(workspace_bytes)


def dualkv_build_index(P, N, R_offsets):
    """Host index builder: returns (seg_id, pos_id, cu_seqlens_rep, rep2pack) as int32 CPU tensors."""
    T = int(P) + int(R_offsets[N])
    n_rep = int(N) * int(P) + int(R_offsets[N])
    seg = torch.empty(T, dtype=torch.int32)
    pos = torch.empty(T, dtype=torch.int32)
    cu = torch.empty(int(N) + 1, dtype=torch.int32)
    r2p = torch.empty(max(n_rep, 1), dtype=torch.int32)
    i32p = ctypes.POINTER(ctypes.c_int32)
    rc = load().dualkv_build_index(int(P), int(N), _offsets(R_offsets),
                                   ctypes.cast(seg.data_ptr(), i32p), ctypes.cast(pos.data_ptr(), i32p),
                                   ctypes.cast(cu.data_ptr(), i32p), ctypes.cast(r2p.data_ptr(), i32p))
    _raise(rc, "dualkv_build_index")
    return seg, pos, cu, r2p[:n_rep]


def dualkv_rho(P, N, R_offsets) -> float:
    return float(load().dualkv_rho(int(P), int(N), _offsets(R_offsets)))


def dualkv_pairs(P, N, R_offsets, window=0) -> int:
    return int(load().dualkv_pairs(int(P), int(N), _offsets(R_offsets), int(window)))


def dualkv_check_status(stream=None) -> None:
    _raise(load().dualkv_check_status(_stream(stream)), "dualkv_check_status")


def dualkv_profile_enable(on: bool) -> None:
    _raise(load().dualkv_profile_enable(1 if on else 0), "dualkv_profile_enable")


def dualkv_profile_read():
    """{kernel kind: (total ms, launches)} of the launches timed since the last read."""
    n = len(KERNEL_KINDS)
    ms = (ctypes.c_double * n)()
    cnt = (ctypes.c_int64 * n)()
    _raise(load().dualkv_profile_read(ms, cnt), "dualkv_profile_read")
    return {KERNEL_KINDS[i]: (float(ms[i]), int(cnt[i])) for i in range(n)}


def dualkv_selftest_timeout(limit_ns: int, stream=None) -> None:
    _raise(load().dualkv_selftest_timeout(int(limit_ns), _stream(stream)), "dualkv_selftest_timeout")


def dualkv_selftest_kernel(which: int, limit_ns: int, stream=None) -> None:
    """Runs a production kernel on a tiny internal layout with its failure path
    forced (0: forward, a K/V tile never loaded; 1: dK/dV, a query block one
    barrier arrival short; 2: forward, a work item past the last row; 3: dQ, a
    work item past the last row; 4: the D = 512 P / dS pass, a K/V tile never
    loaded; 6 and 7: the decode's prompts over a bf16 and a 4-bit cache, a key tile never loaded) and every wait limited to limit_ns.  dualkv_check_status() then raises DUALKV_ERR_DEVICE."""
    _raise(load().dualkv_selftest_kernel(int(which), int(limit_ns), _stream(stream)), "dualkv_selftest_kernel")


def dualkv_plan_cache_info():
    """(resident plans, device bytes held by the plan cache, resident and pooled)."""
    n = ctypes.c_int(0)
    b = ctypes.c_int64(0)
    _raise(load().dualkv_plan_cache_info(ctypes.byref(n), ctypes.byref(b)), "dualkv_plan_cache_info")
    return int(n.value), int(b.value)


def dualkv_release() -> None:
    load().dualkv_release()


# ------------------------------------------------------------------ convenience
def forward(q, k, v, P, R_offsets, window=0, scale=None, stream=None):
    """Allocate out/lse and run dualkv_fwd. q [T,Hq,D], k/v [T,Hkv,D] bf16 CUDA."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    N = len(R_offsets) - 1
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    out = torch.empty_like(q)
    lse = torch.empty(Hq, T, dtype=torch.float32, device=q.device)
    dualkv_fwd(q, k, v, P, N, R_offsets, Hq, Hkv, D, scale, window, out, lse, stream)
    return out, lse


def workspace_for(P, R_offsets, Hq, Hkv, D, window=0, device="cuda"):
    nbytes = dualkv_bwd_workspace_bytes(P, len(R_offsets) - 1, R_offsets, Hq, Hkv, D, window)
    if nbytes == 0:
        raise DualKVError(DUALKV_ERR_INVALID, "dualkv_bwd_workspace_bytes")
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def backward(q, k, v, out, lse, dout, P, R_offsets, window=0, scale=None, workspace=None, stream=None):
    """Allocate dq/dk/dv (and workspace if not given) and run dualkv_bwd."""
    T, Hq, D = q.shape
    Hkv = k.shape[1]
    N = len(R_offsets) - 1
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    if workspace is None:
        workspace = workspace_for(P, R_offsets, Hq, Hkv, D, window, q.device)
    dq = torch.empty_like(q)
    dk = torch.empty_like(k)
    dv = torch.empty_like(v)
    dualkv_bwd(q, k, v, out, lse, dout, P, N, R_offsets, Hq, Hkv, D, scale, window, dq, dk, dv, workspace,
               None, stream)
    return dq, dk, dv


def _allocating_on(stream):
    """Context in which tensors are allocated for use on `stream` (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream))
    return torch.cuda.stream(stream)


def qk_norm_rope(q, k, P, R_offsets, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, weight_offset=0.0,
                 interleaved=False, stream=None):
    """Allocate q_out, k_out and run dualkv_qk_norm_rope; rope_dim is twice the length of inv_freq (None: no rotation)."""
    (T, Hq, D), Hkv = q.shape, k.shape[1]
    rope_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
    with _allocating_on(stream):
        q_out = torch.empty(T, Hq, D, dtype=q.dtype, device=q.device)
        k_out = torch.empty(T, Hkv, D, dtype=k.dtype, device=k.device)
        dualkv_qk_norm_rope(q, k, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved, P,
                            len(R_offsets) - 1, R_offsets, Hq, Hkv, D, q_out, k_out)
    return q_out, k_out


def qk_norm_rope_backward(q, k, dq_out, dk_out, P, R_offsets, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                          weight_offset=0.0, interleaved=False, stream=None):
    """Allocate the gradients (and the workspace) and run dualkv_qk_norm_rope_bwd.
    Returns (dq, dk, dq_weight, dk_weight), the last two None without weights."""
    (T, Hq, D), Hkv, N = q.shape, k.shape[1], len(R_offsets) - 1
    rope_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
    dqw = dkw = ws = None
    with _allocating_on(stream):
        dq = torch.empty(T, Hq, D, dtype=q.dtype, device=q.device)
        dk = torch.empty(T, Hkv, D, dtype=k.dtype, device=k.device)
        if q_weight is not None:
            dqw, dkw = (torch.empty(D, dtype=torch.float32, device=q.device) for _ in range(2))
            nbytes = dualkv_qk_norm_rope_bwd_workspace_bytes(P, N, R_offsets, Hq, Hkv, D)
            ws = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        dualkv_qk_norm_rope_bwd(q, k, dq_out, dk_out, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim,
                                interleaved, P, N, R_offsets, Hq, Hkv, D, dq, dk, dqw, dkw, ws)
    return dq, dk, dqw, dkw


def token_logprobs(logits, tokens, P, R_offsets, scale=1.0, entropy=False, stream=None):
    """Allocate the outputs and run dualkv_token_logprobs: (logp, entropy or None, lse)."""
    n, f32 = int(tokens.shape[0]), dict(dtype=torch.float32, device=logits.device)
    with _allocating_on(stream):
        logp, lse = torch.empty(n, **f32), torch.empty(logits.shape[0], **f32)
        ent = torch.empty(n, **f32) if entropy else None
        dualkv_token_logprobs(logits, tokens, scale, P, len(R_offsets) - 1, R_offsets, logp, ent, lse)
    return logp, ent, lse


def token_logprobs_backward(logits, tokens, lse, dlogp, P, R_offsets, scale=1.0, entropy=None, dentropy=None,
                            inplace=False, stream=None):
    """Allocate dlogits (or, inplace, write it over logits) and run dualkv_token_logprobs_bwd."""
    with _allocating_on(stream):
        dlogits = logits if inplace else torch.empty_like(logits)
        dualkv_token_logprobs_bwd(logits, tokens, scale, P, len(R_offsets) - 1, R_offsets, lse, entropy, dlogp, dentropy,
                                  dlogits)
    return dlogits


def policy_loss(logp, old_logp, advantages, R_offsets, ref_logp=None, entropy=None, mask=None, clip_low=0.2,
                clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0, reduction="token_mean", stream=None,
                per_token=None):
    """Allocate the outputs and the workspace and run dualkv_policy_loss: (loss [1], stats [4], weights [N])."""
    N, f32 = len(R_offsets) - 1, dict(dtype=torch.float32, device=logp.device)
    with _allocating_on(stream):
        loss, stats, weights = torch.empty(1, **f32), torch.empty(4, **f32), torch.empty(N, **f32)
        ws = torch.empty(dualkv_policy_loss_workspace_bytes(N, R_offsets), dtype=torch.uint8, device=logp.device)
        dualkv_policy_loss(logp, old_logp, ref_logp, entropy, advantages, mask, N, R_offsets, clip_low, clip_high,
                           dual_clip, kl_coef, entropy_coef, reduction, loss, stats, weights, ws, per_token=per_token)
    return loss, stats, weights


def policy_loss_backward(logp, old_logp, advantages, R_offsets, dloss, weights, ref_logp=None, mask=None, clip_low=0.2,
                         clip_high=0.2, dual_clip=0.0, kl_coef=0.0, entropy_coef=0.0, stream=None, per_token=None):
    """Allocate the gradients and run dualkv_policy_loss_bwd: (dlogp, dentropy or None without entropy_coef)."""
    N, f32 = len(R_offsets) - 1, dict(dtype=torch.float32, device=logp.device)
    with _allocating_on(stream):
        dlogp = torch.empty(logp.shape[0], **f32)
        dentropy = torch.empty(logp.shape[0], **f32) if entropy_coef else None
        dualkv_policy_loss_bwd(logp, old_logp, ref_logp, advantages, mask, N, R_offsets, clip_low, clip_high, dual_clip,
                               kl_coef, entropy_coef, "token_mean", dloss, weights, dlogp, dentropy,
                               per_token=per_token)
    return dlogp, dentropy


def cache_append(q, k, v, cache, pages, lens, starts, row_offsets, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                 weight_offset=0.0, interleaved=False, stream=None):
    """Allocate q_out and run dualkv_cache_append; rope_dim is twice the length of inv_freq (None: no rotation)."""
    (T, Hq, D), Hkv = q.shape, k.shape[1]
    rope_dim = 0 if inv_freq is None else 2 * inv_freq.numel()
    with _allocating_on(stream):
        q_out = torch.empty(T, Hq, D, dtype=q.dtype, device=q.device)
        dualkv_cache_append(q, k, v, q_weight, k_weight, weight_offset, eps, inv_freq, rope_dim, interleaved, cache, pages,
                            lens, starts, len(row_offsets) - 1, row_offsets, Hq, Hkv, D, q_out)
    return q_out


def cache_read(cache, pages, lens, row_offsets, stream=None):
    """Allocate k and v and run dualkv_cache_read: (k, v), as dualkv.forward takes them."""
    S = len(row_offsets) - 1
    with _allocating_on(stream):
        k, v = (torch.empty(int(row_offsets[S]), cache.Hkv, cache.D, dtype=torch.bfloat16, device=cache.k.device)
                for _ in range(2))
        dualkv_cache_read(cache, pages, lens, S, row_offsets, cache.Hkv, cache.D, k, v)
    return k, v


def decode(q, cache, prompt_pages, prompt_lens, pages, lens, groups, window=0, scale=None, workspace=None, stream=None):
    """Allocate out, lse (and the workspace if not given) and run dualkv_decode: (out [B, Hq, D], lse [Hq, B])."""
    (B, Hq, D), G = q.shape, len(groups) - 1
    scale = 1.0 / math.sqrt(D) if scale is None else scale
    with _allocating_on(stream):
        out = torch.empty(B, Hq, D, dtype=q.dtype, device=q.device)
        lse = torch.empty(Hq, B, dtype=torch.float32, device=q.device)
        if workspace is None:
            nbytes = dualkv_decode_workspace_bytes(G, groups, Hq, cache.Hkv, D)
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=q.device)
        dualkv_decode(q, cache, prompt_pages, prompt_lens, pages, lens, G, groups, Hq, cache.Hkv, D, scale, window, out, lse,
                      workspace)
    return out, lse
