"""Python binding of libkda, the KDA operator for MI355X (gfx950).

The functions here carry the C entry points' names and only marshal arguments:
they check torch tensors (device, dtype, shape, contiguity), allocate outputs
and workspace with torch (device memory is plumbing), pass raw pointers and
the current HIP stream to libkda, and raise on a non-OK status.  Every step of
the operator runs in libkda's HIP kernels; there is no fallback.  If libkda.so
has not been built, every call raises.

    o, S_T = kda_chunk_fwd(q, k, v, theta, beta, S0=None)
    o      = kda_decode_step(q, k, v, theta, beta, S)        # S updated in place
    o, S_T = kda_chunk_fwd_gated(q, k, v, theta, beta, z)    # o * sigmoid(z)
    o, S_T = kda_chunk_fwd_noalloc(q, k, v, theta, beta, S0=None, o=o, S_T=S_T)
    o      = kda_decode_step_gated(q, k, v, theta, beta, S, z)
    g, gc  = kda_gate(theta)

Beside KDA, the gated delta rule with one decay a head, and the norms around a block:

    o, S_T = kda_gdr_chunk_fwd(q, k, v, g, beta, S0, cu_seqlens=cu_seqlens)
    grads  = kda_gdr_chunk_bwd(q, k, v, g, beta, do, S0, dS_T, cu_seqlens=cu_seqlens)
    o      = kda_gdr_step(q, k, v, g, beta, S, slots=slots)  # S updated in place
    r, h   = kda_block_norm_fwd(y, x=x, z=z, w_post=w_post, s=s, w_pre=w_pre)
    grads  = kda_block_norm_bwd(y, dr, dh, x=x, z=z, w_post=w_post, s=s, w_pre=w_pre)
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkda.so")
HEADER_PATH = os.path.join(_HERE, "..", "include", "kda.h")

KDA_BF16, KDA_F32 = 0, 1
KDA_ACT_SIGMOID, KDA_ACT_SILU = 0, 1
KDA_CHUNK = 16
KDA_G_MIN = -5.0

_lib = None


class KdaError(RuntimeError):
    def __init__(self, fn, status, msg):
        super().__init__(f"{fn} failed with status {status}: {msg}")
        self.status = status


def load_library(path: str = LIB_PATH):
    """Load libkda.so (raises if it is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} not found: build it first "
                           "(python -m chunked_gated_delta_12_amd.build)")
    lib = ctypes.CDLL(path)
    c_int, c_size, vp, fp = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p, ctypes.c_void_p
    lib.kda_chunk_fwd.argtypes = [c_int] * 7 + [vp] * 3 + [fp] * 3 + [vp, fp, vp, c_size, vp]
    lib.kda_chunk_fwd.restype = c_int
    lib.kda_chunk_fwd_workspace_size.argtypes = [c_int] * 6 + [ctypes.POINTER(c_size)]
    lib.kda_chunk_fwd_workspace_size.restype = c_int
    lib.kda_chunk_fwd_auto_segments.argtypes = [c_int] * 5
    lib.kda_chunk_fwd_auto_segments.restype = c_int
    lib.kda_decode_step.argtypes = [c_int] * 5 + [vp] * 3 + [fp] * 3 + [vp, vp]
    lib.kda_decode_step.restype = c_int
    lib.kda_chunk_fwd_noalloc.argtypes = [c_int] * 7 + [vp] * 3 + [fp] * 3 + [vp, fp, vp]
    lib.kda_chunk_fwd_noalloc.restype = c_int
    lib.kda_chunk_fwd_gated.argtypes = [c_int] * 7 + [vp] * 3 + [fp] * 3 + [vp, vp, fp, vp, c_size, vp]
    lib.kda_chunk_fwd_gated.restype = c_int
    lib.kda_chunk_bwd.argtypes = [c_int] * 6 + [vp] * 3 + [fp] * 3 + [vp, fp] + [fp] * 6 + [vp, c_size, vp]
    lib.kda_chunk_bwd.restype = c_int
    lib.kda_chunk_bwd_workspace_size.argtypes = [c_int] * 5 + [ctypes.POINTER(c_size)]
    lib.kda_chunk_bwd_workspace_size.restype = c_int
    lib.kda_chunk_fwd_unbounded.argtypes = [c_int] * 6 + [vp] * 3 + [fp] * 3 + [vp, fp, vp]
    lib.kda_chunk_fwd_unbounded.restype = c_int
    lib.kda_decode_step_gated.argtypes = [c_int] * 5 + [vp] * 3 + [fp] * 3 + [vp, vp, vp]
    lib.kda_decode_step_gated.restype = c_int
    lib.kda_gate.argtypes = [c_int] * 4 + [fp, fp, fp, vp]
    lib.kda_gate.restype = c_int
    lib.kda_status_string.argtypes = [c_int]
    lib.kda_status_string.restype = ctypes.c_char_p
    lib.kda_last_error.argtypes = []
    lib.kda_last_error.restype = ctypes.c_char_p
    lib.kda_abi_version.argtypes = []
    lib.kda_abi_version.restype = c_int
    lib.kda_gdr_chunk_fwd.argtypes = [c_int] * 7 + [ctypes.c_float] + [vp] * 9 + [vp, c_size, vp]
    lib.kda_gdr_chunk_fwd.restype = c_int
    lib.kda_gdr_chunk_bwd.argtypes = [c_int] * 7 + [ctypes.c_float] + [vp] * 15 + [vp, c_size, vp]
    lib.kda_gdr_chunk_bwd.restype = c_int
    for fn in (lib.kda_gdr_chunk_fwd_workspace_size, lib.kda_gdr_chunk_bwd_workspace_size):
        fn.argtypes = [c_int] * 6 + [ctypes.POINTER(c_size)]
        fn.restype = c_int
    lib.kda_gdr_clear_rows.argtypes = [c_int, c_int, vp, c_int, ctypes.POINTER(vp), ctypes.POINTER(c_size), vp]
    lib.kda_gdr_clear_rows.restype = c_int
    lib.kda_gdr_step.argtypes = [c_int] * 8 + [ctypes.c_float] + [vp] * 3 + [fp] * 3 + [vp, vp, vp, vp]
    lib.kda_gdr_step.restype = c_int
    lib.kda_block_norm_fwd.argtypes = [c_int, c_int, ctypes.c_longlong, c_int, ctypes.c_float] + [vp] * 9
    lib.kda_block_norm_fwd.restype = c_int
    lib.kda_block_norm_bwd.argtypes = ([c_int, c_int, ctypes.c_longlong, c_int, ctypes.c_float] + [vp] * 15
                                       + [c_size, vp])
    lib.kda_block_norm_bwd.restype = c_int
    lib.kda_block_norm_bwd_workspace_size.argtypes = [ctypes.c_longlong, c_int, ctypes.POINTER(c_size)]
    lib.kda_block_norm_bwd_workspace_size.restype = c_int
    _lib = lib
    return lib


def header_functions(path: str = HEADER_PATH):
    """Names of the functions include/kda.h declares."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kda_\w+)\s*\(", text)))


def _check(fn, status):
    if status != 0:
        lib = load_library()
        raise KdaError(fn, status, lib.kda_last_error().decode() or lib.kda_status_string(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(t, stream):
    if stream is None:
        stream = torch.cuda.current_stream(t.device)
    return ctypes.c_void_p(stream.cuda_stream)


def _dtype_code(t):
    if t.dtype == torch.bfloat16:
        return KDA_BF16
    if t.dtype == torch.float32:
        return KDA_F32
    raise TypeError(f"q/k/v must be bfloat16 or float32, got {t.dtype}")


def _need(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def kda_chunk_fwd_auto_segments(B, T, H, dk, dv) -> int:
    return int(load_library().kda_chunk_fwd_auto_segments(B, T, H, dk, dv))


def kda_chunk_fwd_workspace_size(B, T, H, dk, dv, segments=0) -> int:
    n = ctypes.c_size_t(0)
    _check("kda_chunk_fwd_workspace_size",
           load_library().kda_chunk_fwd_workspace_size(B, T, H, dk, dv, segments, ctypes.byref(n)))
    return int(n.value)


def kda_chunk_fwd(q, k, v, theta, beta, S0=None, *, segments=0, o=None, S_T=None,
                  want_state=True, workspace=None, stream=None):
    """Chunked prefill.  q, k [B,T,H,dk], v [B,T,H,dv] (bf16 or fp32), theta
    [B,T,H,dk] fp32, beta [B,T,H] fp32, S0 [B,H,dk,dv] fp32 or None.
    Returns (o, S_T); S_T is None when want_state is False."""
    return _chunk_fwd(q, k, v, theta, beta, S0, None, segments, o, S_T, want_state, workspace, stream)


def kda_chunk_fwd_gated(q, k, v, theta, beta, z, S0=None, *, segments=0, o=None, S_T=None,
                        want_state=True, workspace=None, stream=None):
    """kda_chunk_fwd with the output gate: o * sigmoid(z), z [B,T,H,dv] of q's dtype."""
    return _chunk_fwd(q, k, v, theta, beta, S0, z, segments, o, S_T, want_state, workspace, stream)


def kda_chunk_fwd_noalloc(q, k, v, theta, beta, S0=None, *, segments=0, o=None, S_T=None,
                          want_state=True, stream=None):
    """kda_chunk_fwd without a workspace: libkda uses its static per-device scratch
    (KDA_NOALLOC_SCRATCH_BYTES).  Pass o and S_T to make the call allocate nothing."""
    return _chunk_fwd(q, k, v, theta, beta, S0, None, segments, o, S_T, want_state, None, stream,
                      noalloc=True)


def kda_chunk_fwd_unbounded(q, k, v, theta, beta, S0=None, *, o=None, S_T=None, want_state=True,
                            stream=None):
    """The ablation of the bound: the recurrence with the unbounded gate
    g = -softplus(theta) and position-wise fp32 diagonal tiles (one segment)."""
    return _chunk_fwd(q, k, v, theta, beta, S0, None, 1, o, S_T, want_state, None, stream, unbounded=True)


def _chunk_fwd(q, k, v, theta, beta, S0, z, segments, o, S_T, want_state, workspace, stream,
               unbounded=False, noalloc=False):
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    _need(q, "q", dt, (B, T, H, dk), dev)
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    _need(theta, "theta", torch.float32, (B, T, H, dk), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dk, dv), dev)
    if z is not None:
        _need(z, "z", dt, (B, T, H, dv), dev)
    if o is None:
        o = torch.empty((B, T, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (B, T, H, dv), dev)
    if S_T is None and want_state:
        S_T = torch.empty((B, H, dk, dv), dtype=torch.float32, device=dev)
    if S_T is not None:
        _need(S_T, "S_T", torch.float32, (B, H, dk, dv), dev)
    nbytes = 0 if (unbounded or noalloc) else kda_chunk_fwd_workspace_size(B, T, H, dk, dv, segments)
    if workspace is None and nbytes > 0:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    if unbounded:
        st = lib.kda_chunk_fwd_unbounded(code, B, T, H, dk, dv, _ptr(q), _ptr(k), _ptr(v), _ptr(theta),
                                         _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T), _stream(q, stream))
        _check("kda_chunk_fwd_unbounded", st)
    elif noalloc:
        st = lib.kda_chunk_fwd_noalloc(code, B, T, H, dk, dv, segments, _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(theta), _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T),
                                       _stream(q, stream))
        _check("kda_chunk_fwd_noalloc", st)
    elif z is None:
        st = lib.kda_chunk_fwd(code, B, T, H, dk, dv, segments, _ptr(q), _ptr(k), _ptr(v), _ptr(theta),
                               _ptr(beta), _ptr(S0), _ptr(o), _ptr(S_T), _ptr(workspace), ws_bytes,
                               _stream(q, stream))
        _check("kda_chunk_fwd", st)
    else:
        st = lib.kda_chunk_fwd_gated(code, B, T, H, dk, dv, segments, _ptr(q), _ptr(k), _ptr(v),
                                     _ptr(theta), _ptr(beta), _ptr(S0), _ptr(z), _ptr(o), _ptr(S_T),
                                     _ptr(workspace), ws_bytes, _stream(q, stream))
        _check("kda_chunk_fwd_gated", st)
    return o, S_T


def kda_chunk_bwd_workspace_size(B, T, H, dk, dv) -> int:
    n = ctypes.c_size_t(0)
    _check("kda_chunk_bwd_workspace_size",
           load_library().kda_chunk_bwd_workspace_size(B, T, H, dk, dv, ctypes.byref(n)))
    return int(n.value)


def kda_chunk_bwd(q, k, v, theta, beta, do, S0=None, dS_T=None, *, want_dS0=True, workspace=None,
                  stream=None):
    """Backward pass of kda_chunk_fwd for L = sum <do, o> + <dS_T, S_T>.  Inputs as
    kda_chunk_fwd plus do [B,T,H,dv] (q's dtype) and dS_T [B,H,dk,dv] fp32 or None.
    Returns a dict of fp32 tensors dq, dk, dv, dtheta, dbeta and dS0 (None unless
    want_dS0)."""
    lib = load_library()
    B, T, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    _need(q, "q", dt, (B, T, H, dk), dev)
    _need(k, "k", dt, (B, T, H, dk), dev)
    _need(v, "v", dt, (B, T, H, dv), dev)
    _need(theta, "theta", torch.float32, (B, T, H, dk), dev)
    _need(beta, "beta", torch.float32, (B, T, H), dev)
    _need(do, "do", dt, (B, T, H, dv), dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (B, H, dk, dv), dev)
    if dS_T is not None:
        _need(dS_T, "dS_T", torch.float32, (B, H, dk, dv), dev)
    f32 = dict(dtype=torch.float32, device=dev)
    g = {"dq": torch.empty((B, T, H, dk), **f32), "dk": torch.empty((B, T, H, dk), **f32),
         "dv": torch.empty((B, T, H, dv), **f32), "dtheta": torch.empty((B, T, H, dk), **f32),
         "dbeta": torch.empty((B, T, H), **f32),
         "dS0": torch.empty((B, H, dk, dv), **f32) if want_dS0 else None}
    nbytes = kda_chunk_bwd_workspace_size(B, T, H, dk, dv)
    if workspace is None:
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.kda_chunk_bwd(code, B, T, H, dk, dv, _ptr(q), _ptr(k), _ptr(v), _ptr(theta), _ptr(beta), _ptr(S0),
                           _ptr(do), _ptr(dS_T), _ptr(g["dq"]), _ptr(g["dk"]), _ptr(g["dv"]), _ptr(g["dtheta"]),
                           _ptr(g["dbeta"]), _ptr(g["dS0"]), _ptr(workspace), ws_bytes, _stream(q, stream))
    _check("kda_chunk_bwd", st)
    return g


def kda_decode_step(q, k, v, theta, beta, S, *, o=None, stream=None):
    """One decode step.  q, k [B,H,dk], v [B,H,dv] (bf16 or fp32), theta [B,H,dk]
    fp32, beta [B,H] fp32, S [B,H,dk,dv] fp32 (updated in place).  Returns o."""
    return _decode_step(q, k, v, theta, beta, S, None, o, stream)


def kda_decode_step_gated(q, k, v, theta, beta, S, z, *, o=None, stream=None):
    """kda_decode_step with the output gate: o * sigmoid(z), z [B,H,dv] of q's dtype."""
    return _decode_step(q, k, v, theta, beta, S, z, o, stream)


def _decode_step(q, k, v, theta, beta, S, z, o, stream):
    lib = load_library()
    B, H, dk = q.shape
    dv = v.shape[-1]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    _need(q, "q", dt, (B, H, dk), dev)
    _need(k, "k", dt, (B, H, dk), dev)
    _need(v, "v", dt, (B, H, dv), dev)
    _need(theta, "theta", torch.float32, (B, H, dk), dev)
    _need(beta, "beta", torch.float32, (B, H), dev)
    _need(S, "S", torch.float32, (B, H, dk, dv), dev)
    if z is not None:
        _need(z, "z", dt, (B, H, dv), dev)
    if o is None:
        o = torch.empty((B, H, dv), dtype=dt, device=dev)
    _need(o, "o", dt, (B, H, dv), dev)
    if z is None:
        st = lib.kda_decode_step(code, B, H, dk, dv, _ptr(q), _ptr(k), _ptr(v), _ptr(theta), _ptr(beta),
                                 _ptr(S), _ptr(o), _stream(q, stream))
        _check("kda_decode_step", st)
    else:
        st = lib.kda_decode_step_gated(code, B, H, dk, dv, _ptr(q), _ptr(k), _ptr(v), _ptr(theta),
                                       _ptr(beta), _ptr(S), _ptr(z), _ptr(o), _stream(q, stream))
        _check("kda_decode_step_gated", st)
    return o


def kda_gate(theta, *, g=True, g_cum=True, stream=None):
    """Bounded gate. theta [B,T,H,dk] fp32 -> (g, g_cum) fp32 (either may be skipped
    by passing False).  Pre-allocated tensors may be passed instead of True."""
    lib = load_library()
    B, T, H, dk = theta.shape
    dev = theta.device
    _need(theta, "theta", torch.float32, (B, T, H, dk), dev)
    if g is True:
        g = torch.empty_like(theta)
    if g_cum is True:
        g_cum = torch.empty_like(theta)
    g = g if isinstance(g, torch.Tensor) else None
    g_cum = g_cum if isinstance(g_cum, torch.Tensor) else None
    for name, t in (("g", g), ("g_cum", g_cum)):
        if t is not None:
            _need(t, name, torch.float32, (B, T, H, dk), dev)
    st = lib.kda_gate(B, T, H, dk, _ptr(theta), _ptr(g), _ptr(g_cum), _stream(theta, stream))
    _check("kda_gate", st)
    return g, g_cum


# ----------------------------------------------------------------------------- one decay a head
class _On:
    """Makes the tensors' device and the work's stream current for one call: launches go to
    the device, and what the call allocates belongs to the stream that uses it.  Where both
    are current already there is nothing to do (a decode step's call is mostly host time)."""

    __slots__ = ("raw", "ctx")

    def __init__(self, t, stream):
        if not t.is_cuda:
            raise ValueError("tensors must be on the GPU")
        if stream is None:
            if t.device.index == torch.cuda.current_device():
                self.raw, self.ctx = torch._C._cuda_getCurrentRawStream(t.device.index), None
                return
            stream = torch.cuda.current_stream(t.device)
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, tensors on {t.device}")
        self.raw, self.ctx = stream.cuda_stream, torch.cuda.stream(stream)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self.raw

    def __exit__(self, *exc):
        if self.ctx is not None:
            return self.ctx.__exit__(*exc)


def _at(t):
    return None if t is None else t.data_ptr()


def _check_workspace(t, device):
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError("workspace must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"workspace is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")


def _dims(t, name, n):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != n:
        raise ValueError(f"{name} has {t.dim()} dimensions, expected {n}")
    return t.shape


def _gdr_inputs(q, k, v, g, beta, scale):
    """Checks what the calls of the rule share: (B, T, Hk, Hv, dk, dv, dtype code, scale)."""
    B, T, Hk, dk = _dims(q, "q", 4)
    Hv, dv = _dims(v, "v", 4)[2:]
    dev, dt = q.device, q.dtype
    code = _dtype_code(q)
    _need(q, "q", dt, (B, T, Hk, dk), dev)
    _need(k, "k", dt, (B, T, Hk, dk), dev)
    _need(v, "v", dt, (B, T, Hv, dv), dev)
    _need(g, "g", torch.float32, (B, T, Hv), dev)
    _need(beta, "beta", torch.float32, (B, T, Hv), dev)
    return B, T, Hk, Hv, dk, dv, code, float(dk ** -0.5 if scale is None else scale)


def _gdr_sequences(B, T, cu_seqlens, dev):
    """(sequences, tokens of each or rows of all) and the shape of a state's leading axis."""
    if cu_seqlens is None:
        return B, T
    if B != 1:
        raise ValueError(f"packed sequences have a leading axis of 1, got {B}")
    n = _dims(cu_seqlens, "cu_seqlens", 1)[0] - 1
    _need(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), dev)
    return n, T


def kda_gdr_chunk_fwd_workspace_size(nseq, T, Hv, dk, dv, packed=False) -> int:
    n = ctypes.c_size_t(0)
    _check("kda_gdr_chunk_fwd_workspace_size",
           load_library().kda_gdr_chunk_fwd_workspace_size(nseq, T, Hv, dk, dv, int(packed), ctypes.byref(n)))
    return int(n.value)


def kda_gdr_chunk_bwd_workspace_size(nseq, T, Hv, dk, dv, packed=False) -> int:
    n = ctypes.c_size_t(0)
    _check("kda_gdr_chunk_bwd_workspace_size",
           load_library().kda_gdr_chunk_bwd_workspace_size(nseq, T, Hv, dk, dv, int(packed), ctypes.byref(n)))
    return int(n.value)


def kda_gdr_clear_rows(cu_seqlens, *tensors, stream=None):
    """Zeros in the rows of no sequence of packed tensors [1,T,..], one to eight, of one T: those
    before cu_seqlens[0] and from cu_seqlens[-1] on.  Nothing else is touched."""
    if not tensors:
        raise ValueError("no tensors")
    n = _dims(cu_seqlens, "cu_seqlens", 1)[0] - 1
    for t in tensors:
        if not isinstance(t, torch.Tensor):
            raise TypeError("tensors must be torch.Tensors")
        if t.dim() < 2 or t.shape[0] != 1:
            raise ValueError(f"packed tensors are [1,T,..], got {tuple(t.shape)}")
    dev, T = tensors[0].device, tensors[0].shape[1]
    _need(cu_seqlens, "cu_seqlens", torch.int32, (n + 1,), dev)
    for t in tensors:
        _need(t, "tensor", t.dtype, (1, T) + tuple(t.shape[2:]), dev)
    with _On(tensors[0], stream) as st:
        _clear_rows(n, T, cu_seqlens, tensors, st)


def _clear_rows(n, T, cu_seqlens, tensors, st):
    k = len(tensors)
    ptrs = (ctypes.c_void_p * k)(*[t.data_ptr() for t in tensors])
    # from the shape: the stride of an axis of one is not the size of its row
    sizes = (ctypes.c_size_t * k)(*[t.numel() // max(1, T) * t.element_size() for t in tensors])
    _check("kda_gdr_clear_rows", load_library().kda_gdr_clear_rows(n, T, _at(cu_seqlens), k, ptrs, sizes, st))


def kda_gdr_chunk_fwd(q, k, v, g, beta, S0=None, *, cu_seqlens=None, scale=None, o=None, S_T=None, want_state=True,
                      workspace=None, stream=None):
    """The gated delta rule with one decay a head over whole sequences.  q, k [B,T,Hk,dk],
    v [B,T,Hv,dv] (bf16 or fp32), g (log-decay), beta [B,T,Hv] fp32, S0 [N,Hv,dk,dv] fp32 or
    None; N = B, or with cu_seqlens [N+1] int32 (then B = 1) the packed sequences.  scale
    defaults to dk ** -0.5.  Returns (o, S_T); S_T is None when want_state is False.  Rows of
    no sequence are left as they were in o (zero where o is made here)."""
    lib = load_library()
    B, T, Hk, Hv, dk, dv, code, scale = _gdr_inputs(q, k, v, g, beta, scale)
    dev = q.device
    nseq, T = _gdr_sequences(B, T, cu_seqlens, dev)
    if S0 is not None:
        _need(S0, "S0", torch.float32, (nseq, Hv, dk, dv), dev)
    _check_workspace(workspace, dev)
    nbytes = kda_gdr_chunk_fwd_workspace_size(nseq, T, Hv, dk, dv, cu_seqlens is not None)
    with _On(q, stream) as st:
        if o is None:
            o = torch.empty((B, T, Hv, dv), dtype=q.dtype, device=dev)
            if cu_seqlens is not None:
                _clear_rows(nseq, T, cu_seqlens, (o,), st)
        _need(o, "o", q.dtype, (B, T, Hv, dv), dev)
        if S_T is None and want_state:
            S_T = torch.empty((nseq, Hv, dk, dv), dtype=torch.float32, device=dev)
        if S_T is not None:
            _need(S_T, "S_T", torch.float32, (nseq, Hv, dk, dv), dev)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check("kda_gdr_chunk_fwd",
               lib.kda_gdr_chunk_fwd(code, nseq, T, Hk, Hv, dk, dv, scale, _at(cu_seqlens), _at(q), _at(k), _at(v), _at(g),
                                     _at(beta), _at(S0), _at(o), _at(S_T), _at(workspace),
                                     workspace.numel() * workspace.element_size(), st))
    return o, S_T


def kda_gdr_chunk_bwd(q, k, v, g, beta, do, S0=None, dS_T=None, *, cu_seqlens=None, scale=None, want_dS0=True,
                      workspace=None, stream=None):
    """Backward of kda_gdr_chunk_fwd for L = sum <do, o> + <dS_T, S_T>, from its inputs alone.
    Returns a dict of dq, dk, dv (q's dtype), dg, dbeta and dS0 (fp32; dS0 None unless
    want_dS0).  The gradients of rows of no sequence are zero."""
    lib = load_library()
    B, T, Hk, Hv, dk, dv, code, scale = _gdr_inputs(q, k, v, g, beta, scale)
    dev = q.device
    nseq, T = _gdr_sequences(B, T, cu_seqlens, dev)
    _need(do, "do", q.dtype, (B, T, Hv, dv), dev)
    for name, t in (("S0", S0), ("dS_T", dS_T)):
        if t is not None:
            _need(t, name, torch.float32, (nseq, Hv, dk, dv), dev)
    _check_workspace(workspace, dev)
    nbytes = kda_gdr_chunk_bwd_workspace_size(nseq, T, Hv, dk, dv, cu_seqlens is not None)
    with _On(q, stream) as st:
        d = {"dq": torch.empty_like(q), "dk": torch.empty_like(k), "dv": torch.empty_like(v),
             "dg": torch.empty_like(g), "dbeta": torch.empty_like(beta),
             "dS0": torch.empty((nseq, Hv, dk, dv), dtype=torch.float32, device=dev) if want_dS0 else None}
        if cu_seqlens is not None:
            _clear_rows(nseq, T, cu_seqlens, [d[name] for name in ("dq", "dk", "dv", "dg", "dbeta")], st)
        if workspace is None:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=dev)
        _check("kda_gdr_chunk_bwd",
               lib.kda_gdr_chunk_bwd(code, nseq, T, Hk, Hv, dk, dv, scale, _at(cu_seqlens), _at(q), _at(k), _at(v), _at(g),
                                     _at(beta), _at(S0), _at(do), _at(dS_T), _at(d["dq"]), _at(d["dk"]), _at(d["dv"]),
                                     _at(d["dg"]), _at(d["dbeta"]), _at(d["dS0"]), _at(workspace),
                                     workspace.numel() * workspace.element_size(), st))
    return d


def kda_gdr_step(q, k, v, g, beta, S, *, slots=None, ntok=None, scale=None, o=None, stream=None):
    """T tokens of the gated delta rule (one decay a head) for each of B rows, the states in
    a pool updated in place.  q, k [B,T,Hk,dk], v [B,T,Hv,dv] (bf16 or fp32), g, beta
    [B,T,Hv] fp32, S [nslot,Hv,dk,dv] fp32; slots [B] int32 names each row's state (None:
    row b has state b; outside the pool: a padded row), ntok [B] int32 how many of its
    tokens are real (None: all).  scale defaults to dk ** -0.5.  Returns o [B,T,Hv,dv]; what
    belongs to padded rows and tokens is left as it was (zero where o is made here)."""
    lib = load_library()
    B, T, Hk, Hv, dk, dv, code, scale = _gdr_inputs(q, k, v, g, beta, scale)
    dev = q.device
    nslot = _dims(S, "S", 4)[0]
    _need(S, "S", torch.float32, (nslot, Hv, dk, dv), dev)
    for name, t in (("slots", slots), ("ntok", ntok)):
        if t is not None:
            _need(t, name, torch.int32, (B,), dev)
    with _On(q, stream) as st:
        if o is None:
            make = torch.empty if slots is None and ntok is None else torch.zeros
            o = make((B, T, Hv, dv), dtype=q.dtype, device=dev)
        _need(o, "o", q.dtype, (B, T, Hv, dv), dev)
        _check("kda_gdr_step",
               lib.kda_gdr_step(code, B, T, Hk, Hv, dk, dv, nslot, scale, _at(q), _at(k), _at(v), _at(g), _at(beta),
                                _at(S), _at(slots), _at(ntok), _at(o), st))
    return o


# ----------------------------------------------------------------------------- block norm
_ACTS = {"sigmoid": KDA_ACT_SIGMOID, "silu": KDA_ACT_SILU}


def _norm_inputs(y, x, z, w_post, s, w_pre, act):
    if not isinstance(y, torch.Tensor) or y.dim() < 1:
        raise TypeError("y must be a torch.Tensor with at least one dimension")
    if act not in _ACTS:
        raise ValueError(f"act must be one of {sorted(_ACTS)}, got {act!r}")
    code = _dtype_code(y)
    D = y.shape[-1]
    for name, t in (("y", y), ("x", x), ("z", z)):
        if t is not None:
            _need(t, name, y.dtype, y.shape, y.device)
    for name, t in (("w_post", w_post), ("s", s), ("w_pre", w_pre)):
        if t is not None:
            _need(t, name, torch.float32, (D,), y.device)
    return code, _ACTS[act], y.numel() // max(1, D), D


def kda_block_norm_fwd(y, *, x=None, z=None, w_post=None, s=None, w_pre=None, act="sigmoid", eps=1e-6, r=None, h=None,
                       stream=None):
    """The norms around a block with its gate and residual: with n = rmsnorm(y) w_post,
    r = x + n act(z) s and h = rmsnorm(r) w_pre over the last dimension, every part but y
    optional.  y, x, z [..., D] (bf16 or fp32), w_post, s, w_pre [D] fp32; act "sigmoid"
    or "silu".  r may be x itself.  Returns (r, h); h is None without w_pre."""
    lib = load_library()
    code, a, rows, D = _norm_inputs(y, x, z, w_post, s, w_pre, act)
    if h is not None and w_pre is None:
        raise ValueError("h without w_pre")
    with _On(y, stream) as st:
        r = torch.empty_like(y) if r is None else r
        _need(r, "r", y.dtype, y.shape, y.device)
        if w_pre is not None:
            h = torch.empty_like(y) if h is None else h
            _need(h, "h", y.dtype, y.shape, y.device)
        _check("kda_block_norm_fwd",
               lib.kda_block_norm_fwd(code, a, rows, D, eps, _at(y), _at(x), _at(z), _at(w_post), _at(s), _at(w_pre),
                                      _at(r), _at(h), st))
    return r, h


def kda_block_norm_bwd_workspace_size(rows, D) -> int:
    n = ctypes.c_size_t(0)
    _check("kda_block_norm_bwd_workspace_size",
           load_library().kda_block_norm_bwd_workspace_size(rows, D, ctypes.byref(n)))
    return int(n.value)


def kda_block_norm_bwd(y, dr, dh=None, *, x=None, z=None, w_post=None, s=None, w_pre=None, act="sigmoid", eps=1e-6,
                       workspace=None, stream=None):
    """Backward of kda_block_norm_fwd for L = sum <dr, r> + <dh, h>, from its inputs alone
    (dr may be None; dh goes with w_pre).  Returns a dict of dy, dx, dz (y's dtype) and
    dw_post, ds, dw_pre (fp32); None for parts that were not given."""
    lib = load_library()
    code, a, rows, D = _norm_inputs(y, x, z, w_post, s, w_pre, act)
    for name, t in (("dr", dr), ("dh", dh)):
        if t is not None:
            _need(t, name, y.dtype, y.shape, y.device)
    _check_workspace(workspace, y.device)
    with _On(y, stream) as st:
        d = {name: None if t is None else torch.empty_like(t)
             for name, t in (("dy", y), ("dx", x), ("dz", z), ("dw_post", w_post), ("ds", s), ("dw_pre", w_pre))}
        if workspace is None and not (w_post is None and s is None and w_pre is None):
            workspace = torch.empty(kda_block_norm_bwd_workspace_size(rows, D), dtype=torch.uint8, device=y.device)
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check("kda_block_norm_bwd",
               lib.kda_block_norm_bwd(code, a, rows, D, eps, _at(y), _at(x), _at(z), _at(w_post), _at(s), _at(w_pre),
                                      _at(dr), _at(dh), _at(d["dy"]), _at(d["dx"]), _at(d["dz"]), _at(d["dw_post"]),
                                      _at(d["ds"]), _at(d["dw_pre"]), _at(workspace), ws_bytes, st))
    return d


__all__ = ["kda_gdr_chunk_fwd", "kda_gdr_chunk_bwd", "kda_gdr_chunk_fwd_workspace_size",
           "kda_gdr_chunk_bwd_workspace_size", "kda_gdr_clear_rows", "kda_gdr_step", "kda_block_norm_fwd", "kda_block_norm_bwd", "kda_block_norm_bwd_workspace_size",
           "KDA_ACT_SIGMOID", "KDA_ACT_SILU", "kda_chunk_fwd", "kda_chunk_fwd_noalloc", "kda_chunk_fwd_gated", "kda_chunk_fwd_unbounded", "kda_chunk_bwd",
           "kda_chunk_bwd_workspace_size", "kda_decode_step",
           "kda_decode_step_gated", "kda_gate", "kda_chunk_fwd_workspace_size",
           "kda_chunk_fwd_auto_segments", "load_library", "header_functions", "KdaError",
           "KDA_BF16", "KDA_F32", "KDA_CHUNK", "KDA_G_MIN"]
